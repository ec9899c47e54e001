"""The sampler (qurl_sample) against the definition in 64 bits, row by row.

Tokens are equal, but where a border is undecided: every weight carries a relative
error below 2^-29, so the running sum and the sum it is compared with differ from
the exact ones by at most that each, and a choice is the exact one for a u and a
top_p within 2^-28 of those given.  The reference says how near the nearest border
is; in a row nearer than 2^-28 (a nucleus that ends among tens of thousands of
tokens of weight 1e-9 has to be) the token is one that such a u and top_p give.
logp: weights' error 2^-29 and one fp32 rounding, 2^-24 |logp|, taken as 2^-26 +
2^-23 |logp|; in a row with top-k, min-p or temperature 0 the whole row's sum (only
logp has it) is of fp32 exponentials: 2^-22 each, their arguments' rounding (p |a|
2^-23 <= 2^-24), and at most V / 256 + 32 additions of 2^-24 in a row."""
import math

import pytest
import torch

import w8a8_precision_gemm_gb300 as q

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(autouse=True)
def _status():
    yield
    q.qurl_check_device_status()


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def logits(B, V, dtype=torch.bfloat16, seed=0, sigma=2.5, peaks=8, pad=None):
    g = _gen(seed)
    per = 8 if dtype == torch.bfloat16 else 4
    ld = -(-V // per) * per if pad is None else pad
    x = torch.full((B, ld), 1e4, device="cuda")  # what lies behind a row is never drawn
    x[:, :V] = torch.randn((B, V), device="cuda", generator=g) * sigma
    if peaks:
        at = torch.randint(0, V, (B, peaks), device="cuda", generator=g)
        x.scatter_add_(1, at, torch.rand((B, peaks), device="cuda", generator=g) * 12)
    return x.to(dtype)[:, :V]


def reference(x, u, t=None, k=None, p=None, m=None):
    """(token, logp, logp_kept, distance to the nearest border) of each row."""
    out = []
    for b in range(x.shape[0]):
        l = x[b].double()
        l = torch.where(torch.isnan(l), -INF, l).clamp(max=float(torch.finfo(torch.float32).max))
        T = 1.0 if t is None else float(t[b])
        top = l.max()
        if float(top) == -INF:
            out.append((-1, -INF, -INF, 1.0))
            continue
        z = (l - top) / (T or 1.0)
        w = torch.exp(z)
        order = torch.sort(l, descending=True, stable=True).indices
        ws, n, near = w[order], len(l), 1.0
        if T == 0:
            n = 1
        else:
            if k is not None and 0 < int(k[b]) < n:
                n = int(k[b])
            if m is not None and float(m[b]) > 0:
                n = min(n, int((ws >= float(m[b])).sum()))
                if float(m[b]) < 1:
                    near = min(near, float((ws / float(m[b]) - 1).abs().min()))
            if p is not None and float(p[b]) < 1:
                before = torch.cumsum(ws[:n], 0) - ws[:n]
                edge = float(p[b]) * float(ws[:n].sum())
                near = min(near, float((before[1:] - edge).abs().min()) / edge) if n > 1 and edge > 0 else near
                n = max(1, int((before < edge).sum()))
        kept = torch.zeros_like(w)
        kept[order[:n]] = ws[:n]
        cum = torch.cumsum(kept, 0)
        goal = float(u[b]) * float(cum[-1])
        i = int((cum <= goal).sum())
        if goal > 0:
            near = min(near, float((cum - goal).abs().min()) / float(cum[-1]))
        out.append((i, float(z[i] - torch.log(w.sum())), float(z[i] - torch.log(cum[-1])), near))
    return out


def check(x, u, t=None, k=None, p=None, m=None):
    token, logp, kept = q.sample(x, u, t, k, p, m, want_kept=True)
    token, logp, kept = token.tolist(), logp.tolist(), kept.tolist()
    for b, (i, lp, lk, near) in enumerate(reference(x, u, t, k, p, m)):
        if token[b] != i:
            assert 0 < near <= 2.0 ** -28, (b, token[b], i, near)
            row = slice(b, b + 1)
            some = [reference(x[row], u[row].double() * (1 + du), *(None if v is None else v[row] for v in (t, k)),
                              None if p is None else p[row].double() * (1 + dp), None if m is None else m[row])[0]
                    for du in (0, 2.0 ** -28, -2.0 ** -28) for dp in (0, 2.0 ** -28, -2.0 ** -28)]
            assert token[b] in [r[0] for r in some], (b, token[b], i, near)
            lp, lk = next((r[1], r[2]) for r in some if r[0] == token[b])
        plain = (k is not None and 0 < int(k[b]) < x.shape[1]) or (m is not None and float(m[b]) > 0) or \
            (t is not None and float(t[b]) == 0)
        sum32 = 2.0 ** -21 + (x.shape[1] / 256 + 32) * 2.0 ** -24 if plain else 0.0
        for got, want, more in ((logp[b], lp, sum32), (kept[b], lk, 0.0)):
            tol = 2.0 ** -26 + 2.0 ** -23 * abs(want) + more
            assert got == want if math.isinf(want) else abs(got - want) <= tol, (b, got, want)
    return token


def f32(*v):
    return torch.tensor(v, dtype=torch.float32, device="cuda")


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [1, 2, 3, 7, 8, 9, 255, 1000, 1024, 1025, 8192, 8193, 32000, 50257, 131072, 200001])
def test_vocabularies(V, dtype):
    B = 5
    x, u = logits(B, V, dtype, seed=V), torch.rand(B, device="cuda", generator=_gen(V))
    check(x, u)
    check(x, u, f32(.7, 1., 0., 1.4, .2), i32(0, 50, 5, 1, 7), f32(.9, 1., .5, .95, .3), f32(0., .01, .1, .3, 0.))


@pytest.mark.parametrize("B", [1, 2, 7, 64, 151, 153, 304, 700])
def test_batches(B):
    g = _gen(B)
    r = torch.rand((5, B), device="cuda", generator=g)
    x = logits(B, 5000, seed=B)
    check(x, r[0], 0.3 + r[1], torch.where(r[2] < .5, 0, (r[2] * 200).int()).int(),
          torch.where(r[3] < .3, torch.ones_like(r[3]), r[3]), torch.where(r[4] < .5, torch.zeros_like(r[4]), r[4] * .2))


@pytest.mark.parametrize("sigma,peaks", [(0.01, 0), (1.0, 0), (4.0, 0), (0.5, 3), (20.0, 0)])
@pytest.mark.parametrize("p", [0.0, 0.01, 0.5, 0.99, 0.99999])
def test_flat_and_peaked_rows(sigma, peaks, p):
    """Nuclei of one token to nearly the whole vocabulary."""
    x = logits(3, 60000, seed=17, sigma=sigma, peaks=peaks)
    check(x, torch.rand(3, device="cuda", generator=_gen(3)), p=f32(p, p, p))
    check(x.float(), torch.rand(3, device="cuda", generator=_gen(4)), p=f32(p, p, p))


@pytest.mark.parametrize("k", [1, 2, 100, 1000, 5000, 59999, 60000, 10 ** 9, -1])
def test_top_k(k):
    x = logits(3, 60000, torch.float32, seed=k & 1023, sigma=1.5)
    u = torch.rand(3, device="cuda", generator=_gen(5))
    check(x, u, k=i32(k, k, k))
    check(x, u, k=i32(k, k, k), p=f32(.9, .5, .999))


@pytest.mark.parametrize("m", [0.0, 1e-30, 1e-6, 0.01, 0.5, 1.0])
def test_min_p(m):
    x = logits(3, 30000, seed=2)
    u = torch.rand(3, device="cuda", generator=_gen(6))
    check(x, u, m=f32(m, m, m))
    check(x, u, t=f32(.5, 2., 5.), k=i32(40, 4000, 0), p=f32(1., .9, .99), m=f32(m, m, m))


def test_min_p_that_cuts_nothing_behind_a_large_top_k():
    """The min-p step then has nothing to do in any CTA of the row's cluster, and the next
    step follows at once."""
    x = logits(3, 60000, seed=21, sigma=1.5)
    u = torch.rand(3, device="cuda", generator=_gen(21))
    k, m = i32(1000, 4000, 9000), f32(1e-30, 1e-30, 1e-30)
    token = check(x, u, k=k, m=m)
    for _ in range(50):
        assert q.sample(x, u, top_k=k, min_p=m)[0].tolist() == token
    check(x, u, k=k, p=f32(.9, .99, .999), m=m)


def test_ties_go_to_the_lowest_index():
    """Equal logits: the order is by index, the kept weights are exact, so is every border."""
    x = torch.zeros((4, 4096), device="cuda")
    assert check(x, f32(0., .25, .5, 1 - 2.0 ** -24)) == [0, 1024, 2048, 4095]
    assert check(x, f32(0., .5, .5, .75), k=i32(10, 10, 3, 4)) == [0, 5, 1, 3]
    assert check(x, f32(.999, .999, 0., .5), p=f32(.25, 1 / 4096, .5, 0.)) == [1022, 0, 0, 0]
    assert check(x, f32(.9, .9, .9, .9), t=f32(0., 0., 0., 0.)) == [0, 0, 0, 0]
    x[:, 3000] = 1.0
    x[:, 700] = 1.0
    assert check(x, f32(0., .9, .4, .6), t=f32(0., 0., 1., 1.), k=i32(0, 0, 2, 2)) == [700, 700, 700, 3000]
    x = torch.zeros((2, 100000), device="cuda", dtype=torch.bfloat16)  # one value in all of a large row
    # (.999 in fp32 is .99900001287: of 50000 equal weights 49950.0006 lie below it, so the 49951st is drawn)
    assert check(x, f32(.5, .999), k=i32(60001, 0), p=f32(1., .5)) == [30000, 49950]


def test_negative_and_signed_zero_logits():
    x = -logits(3, 3000, torch.float32, seed=9).abs() - 3
    x[1, ::2] = -0.0
    x[1, 1::2] = 0.0
    check(x, f32(.1, .7, .99), k=i32(5, 6, 0), p=f32(.9, .9, .9))


def test_masked_infinite_and_nan_logits():
    low = float(torch.finfo(torch.bfloat16).min)
    x = logits(8, 1000, seed=11)
    x[0] = -INF                      # nothing left
    x[1] = -INF
    x[1, 777] = -3.0                 # one token left
    x[2, :990] = low                 # masked by the lowest value
    x[3] = low                       # all of it: a uniform row
    x[4, 5] = float("nan")
    x[5, 400] = INF
    x[5, 500] = INF                  # the largest float, twice
    x[6] = float("nan")
    x[7, ::2] = -INF
    u = torch.rand(8, device="cuda", generator=_gen(12))
    for kw in (dict(), dict(k=i32(*[7] * 8)), dict(p=f32(*[.8] * 8)), dict(m=f32(*[.05] * 8)), dict(t=f32(*[0.] * 8)),
               dict(t=f32(*[2.] * 8), k=i32(*[900] * 8), p=f32(*[.99] * 8))):
        token = check(x, u, **kw)
        assert token[0] == -1 and token[6] == -1 and token[1] == 777 and token[7] % 2 == 1 and token[5] in (400, 500)


def test_extreme_temperatures_and_magnitudes():
    x = logits(4, 20000, torch.float32, seed=13)
    u = torch.rand(4, device="cuda", generator=_gen(13))
    check(x, u, f32(1e-6, 1e6, 1e-3, 50.), p=f32(.9, .9, .9, .9))
    check(x * 1e30, u, f32(1., 1e6, 1e-6, .1))
    check(x * 1e-20, u, f32(1., 1e-6, 2., .1), k=i32(10, 10, 0, 0))
    check(x + 1e6, u, p=f32(.9, .9, 1., 1.))


def test_bad_parameters_are_reported():
    x, u = logits(9, 100, seed=1), f32(*[.5] * 9)
    nan = float("nan")
    t, k = f32(-1., nan, 1e7, 1., 1., 1., 1., 1., 1.), None
    p = f32(1., 1., 1., -.1, nan, 1., 1., 1., 1.)
    m = f32(0., 0., 0., 0., 0., 1.5, nan, 0., 0.)
    u[7] = 1.0
    token, logp, kept = q.sample(x, u, t, k, p, m, want_kept=True)
    with pytest.raises(q.QurlError):
        q.qurl_check_device_status()
    assert token[:8].tolist() == [-1] * 8 and bool((logp[:8] == -INF).all()) and bool((kept[:8] == -INF).all())
    assert int(token[8]) == reference(x[8:], u[8:])[0][0]


def test_repeats_streams_and_graphs():
    x, u = logits(20, 40000, seed=3), torch.rand(20, device="cuda", generator=_gen(3))
    p = torch.full((20,), .9, device="cuda")
    a = q.sample(x, u, top_p=p)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = q.sample(x, u, top_p=p)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c = q.sample(x, u, top_p=p)
    u.copy_(torch.rand(20, device="cuda", generator=_gen(4)))
    g.replay()
    assert c[0].tolist() == [r[0] for r in reference(x, u, p=p)]


def test_rows_behind_the_batch_and_optional_outputs():
    x, u = logits(3, 50, seed=5), f32(.1, .5, .9)
    token = torch.full((5,), -7, dtype=torch.int64, device="cuda")
    q.qurl_sample(x, u, token[:3])
    assert token.tolist() == [r[0] for r in reference(x, u)] + [-7, -7]
    with pytest.raises(ValueError):
        q.sample(x, u.double())
    with pytest.raises(ValueError):
        q.sample(x, u, top_k=f32(1., 1., 1.))
    with pytest.raises(ValueError):
        q.sample(x, u[:2])
    with pytest.raises(ValueError):
        q.sample(x.half(), u)


@pytest.mark.parametrize("B", [4096, 4097])
def test_large_batches_of_differing_rows(B):
    """Batches of several waves, whose rows are taken in an order of their own up to 4096 rows."""
    g = _gen(B)
    r = torch.rand((4, B), device="cuda", generator=g)
    x = logits(B, 700, seed=B)
    u, t = r[0], torch.where(r[1] < .1, torch.zeros_like(r[1]), 0.5 + r[1])
    k = torch.where(r[2] < .4, 0, (r[2] * 600).int()).int()
    p, m = torch.where(r[3] < .3, torch.ones_like(r[3]), r[3]), torch.where(r[0] < .5, torch.zeros_like(u), r[1] * .01)
    token, logp, kept = q.sample(x, u, t, k, p, m, want_kept=True)
    some = torch.randperm(B, generator=torch.Generator().manual_seed(B))[:200].cuda()
    y = torch.empty((200, 704), dtype=x.dtype, device="cuda")[:, :700]
    y.copy_(x[some])
    got = q.sample(y, u[some], t[some], k[some], p[some], m[some], want_kept=True)  # (one wave)
    for a, b in zip((token, logp, kept), got):
        assert torch.equal(a[some], b)
    check(y, u[some], t[some], k[some], p[some], m[some])


@pytest.mark.parametrize("V", [7, 600, 5000, 60000])
def test_negative_zero_parameters(V):
    """-0 lies in every parameter's range and is 0."""
    z, n = f32(0., 0., 0.), f32(-0., -0., -0.)
    x = logits(3, V, seed=V)
    for kw in (dict(u=n), dict(u=n, p=n), dict(u=f32(.5, .9, .1), p=n), dict(u=n, t=n), dict(u=n, m=n, k=i32(0, 3, 900))):
        token = check(x, **kw)
        assert token == check(x, **{a: z if b is n else b for a, b in kw.items()})


@pytest.mark.parametrize("V", [262144, 262145, 300001, (1 << 20) + 3, 1 << 24])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_vocabularies_of_longer_segments(V, dtype):
    """Past 2^18 logits a segment holds more than 512; 2^24 is the most."""
    B = 2 if V < 1 << 24 else 1
    x, u = logits(B, V, dtype, seed=V & 1023), torch.rand(B, device="cuda", generator=_gen(V & 1023))
    check(x, u)
    check(x, u, k=i32(50, 7)[:B], p=f32(.9, .5)[:B])
    check(x, u, t=f32(.8, 1.1)[:B], p=f32(.95, .999)[:B])
    check(x, u, k=i32(5000, 100000)[:B], m=f32(1e-4, 0.)[:B], p=f32(.99, .9)[:B])
