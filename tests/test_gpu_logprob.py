"""Token log-probabilities and the logits' gradient (qurl_token_logprob,
qurl_token_logprob_grad) against the formulas in 64 bits and, for the gradient,
against differences of the forward call.

Tolerances, from the arithmetic.  Forward: each exp carries 2^-22 (the
approximate instruction) and its argument a few roundings, worth p |a| 2^-22 <=
2^-23 of the sum; the sum itself at most n additions of 2^-24 in a row, n = V /
512 + 24; then fp32 roundings of logp and lse.  Gradient: exp(z - lse) with z and
lse in fp32, so relative (|z| + |lse| + 4) 2^-23, times the row's factor, and
half a step of the output type."""
import pytest
import torch

import w8a8_precision_gemm_gb300 as q

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(autouse=True)
def _status():
    yield
    q.qurl_check_device_status()


def make(T, V, dtype, seed=0, sigma=3.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    per = 8 if dtype == torch.bfloat16 else 4
    ld = -(-V // per) * per + per
    x = torch.full((T, ld), 1e4, device="cuda")  # never part of a row
    x[:, :V] = torch.randn((T, V), device="cuda", generator=g) * sigma
    t = torch.randint(0, V, (T,), device="cuda", generator=g)
    return x.to(dtype)[:, :V], t, torch.randn(T, device="cuda", generator=g)


def check(x, targets, g, temperature=1.0, scale=1.0, denom=None, inplace=False):
    T, V = x.shape
    z = x.double() / temperature
    ok = (targets >= 0) & (targets < V)
    at = torch.where(ok, targets, 0)
    lse_r = torch.logsumexp(z, -1)
    logp_r = torch.gather(z, 1, at[:, None])[:, 0] - lse_r
    logp, lse = q.token_logprob(x, targets, temperature)
    live = ok & torch.isfinite(lse_r)
    assert bool((logp[~ok] == 0).all()) and bool((lse[~ok] == 0).all())
    empty = ok & ~torch.isfinite(lse_r)
    assert bool((lse[empty] == -INF).all()) and bool((logp[empty] == -INF).all())
    tol = (V / 512 + 24) * 2.0 ** -24 + 2.0 ** -21
    fin = live & torch.isfinite(logp_r)
    assert bool((logp[live & ~fin] == -INF).all())
    zero = torch.zeros_like(logp_r)
    d = torch.where(fin, logp.double() - logp_r, zero).abs()
    assert bool(d.le(tol + 2.0 ** -22 * torch.where(fin, logp_r, zero).abs()).all()), float(d.max())
    d = torch.where(live, lse.double() - lse_r, zero).abs()
    assert bool(d.le(tol + 2.0 ** -22 * torch.where(live, lse_r, zero).abs()).all()), float(d.max())

    n = 1.0 if denom is None else float(denom)
    w = torch.where(live, g.double() * scale / (n * temperature), zero)[:, None] if n > 0 else zero[:, None]
    lz = torch.where(live, lse.double(), zero)[:, None]
    p = torch.where(live[:, None], torch.exp(z - lz), 0.0)
    want = -w * p
    want.scatter_add_(1, at[:, None], w * live[:, None])
    size = torch.where(torch.isfinite(z), z, 0.0).abs()
    half = 2.0 ** -8 if x.dtype == torch.bfloat16 else 2.0 ** -24  # half of finfo.eps: 8 and 24 significant bits
    bound = w.abs() * (p * (size + lz.abs() + 4) * 2.0 ** -23) + want.abs() * (half + 2.0 ** -22) + 1e-38
    src = x.clone() if inplace else x
    if inplace:
        src = torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device="cuda").copy_(x)
    got = q.token_logprob_grad(src, targets, lse, g, temperature, scale, denom, inplace)
    assert got.dtype == x.dtype and (got.data_ptr() == src.data_ptr()) == inplace
    e = (got.double() - want).abs()
    assert bool(e.le(bound).all()), (float(e.max()), float((e / bound).max()))
    return logp, lse, got


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,V", [(1, 1), (3, 2), (5, 7), (4, 8), (2, 9), (6, 255), (3, 4096), (7, 4097), (1, 131072),
                                 (2, 131073), (40, 32000), (700, 1003), (310, 16384)])
def test_sizes(T, V, dtype):
    x, t, g = make(T, V, dtype, seed=V + T)
    check(x, t, g)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("temperature", [0.05, 0.7, 3.0])
def test_temperature_scale_and_denominator(temperature, dtype):
    x, t, g = make(9, 5000, dtype, seed=1)
    n = torch.tensor([7.0], dtype=torch.float64, device="cuda")
    check(x, t, g, temperature, -1.5, n)
    check(x, t, g, temperature, inplace=True)
    n.zero_()
    check(x, t, g, temperature, 1.0, n)


def test_padding_and_bad_targets():
    x, t, g = make(8, 3000, torch.float32, seed=2)
    t[1], t[4], t[7] = -1, -100, -2 ** 40
    x[4] = float("nan")  # a padded row's values are not used
    g[4] = float("nan")
    xs, gs = x.clone(), g.clone()
    xs[4], gs[4] = 0, 0
    logp, lse, d = (o.clone() for o in check(xs, t, gs))
    l2, s2 = q.token_logprob(x, t)
    d2 = q.token_logprob_grad(x, t, torch.where(t < 0, float("nan"), s2), g)
    assert torch.equal(l2, logp) and torch.equal(s2, lse) and torch.equal(d2, d) and not bool(d2[4].any())
    q.qurl_check_device_status()
    t[2] = 3000
    logp, lse = q.token_logprob(x, t)
    with pytest.raises(q.QurlError):
        q.qurl_check_device_status()
    assert float(logp[2]) == 0 and float(lse[2]) == 0
    d = q.token_logprob_grad(x, t, lse, g)
    with pytest.raises(q.QurlError):
        q.qurl_check_device_status()
    assert not bool(d[2].any())


def test_masked_logits():
    low = float(torch.finfo(torch.bfloat16).min)
    x, t, g = make(6, 2000, torch.bfloat16, seed=3)
    x[0] = -INF                      # nothing in the row
    x[1, :1990] = -INF
    t[1] = 1995
    x[2, 5:] = -INF
    t[2] = 1000                      # the target itself is masked
    x[3, 100:] = low
    t[3] = 50
    x[4, ::2] = low
    t[4] = 2                         # a target at the lowest value
    logp, lse, d = check(x[[0, 1, 2, 3, 5]], t[[0, 1, 2, 3, 5]], g[[0, 1, 2, 3, 5]])
    assert not bool(d[0].any())
    logp, lse = q.token_logprob(x[4:5], t[4:5])
    assert float(logp[0]) < -1e38 and bool(torch.isfinite(lse).all())
    x[4] = low                       # a uniform row at the lowest value
    logp, _ = q.token_logprob(x[4:5], t[4:5])
    assert abs(float(logp[0]) + torch.log(torch.tensor(2000.0)).item()) < 1e-5


def test_large_logits():
    x, t, g = make(4, 1000, torch.float32, seed=4)
    check(x * 20, t, g)
    check(x + 500, t, g)
    check(x - 500, t, g)


@pytest.mark.parametrize("dtype,h", [(torch.float32, 2.0 ** -5)])
def test_gradient_against_differences(dtype, h):
    """Central differences of the forward call: h^2 / 6 times the third derivative (at most 1 / 8 per unit of
    weight and temperature^-3) and the forward call's error, at most 2^-19 by the bound above, over h."""
    temperature, scale = 0.8, 2.0
    x, t, g = make(3, 40, dtype, seed=5, sigma=1.5)
    _, lse = q.token_logprob(x, t, temperature)
    d = q.token_logprob_grad(x, t, lse, g, temperature, scale)
    for v in range(40):
        up, down = x.clone(), x.clone()
        up[:, v] += h
        down[:, v] -= h
        diff = (q.token_logprob(up, t, temperature)[0] - q.token_logprob(down, t, temperature)[0]).double() * g * scale / (2 * h)
        tol = (scale * g.abs()) * (h * h / 48 / temperature ** 3 + 2.0 ** -18 / h)
        assert bool((diff - d[:, v].double()).abs().le(tol).all())


def test_gradient_rows_sum_to_zero_and_match_autograd():
    x, t, g = make(16, 777, torch.float32, seed=6)
    leaf = x.double().detach().clone().requires_grad_(True)
    (torch.log_softmax(leaf / 1.3, -1).gather(1, t[:, None])[:, 0] * g.double()).sum().backward()
    _, lse = q.token_logprob(x, t, 1.3)
    d = q.token_logprob_grad(x, t, lse, g, 1.3)
    assert bool((d.double() - leaf.grad).abs().le(g.abs().double()[:, None] * 2.0 ** -17).all())
    assert bool(d.double().sum(-1).abs().le(g.abs().double() * 777 * 2.0 ** -20).all())


def test_offsets_past_32_bits():
    """Rows whose elements lie past 2^31: the last rows of a 2.4 G-element batch."""
    T, V = 18400, 131072
    x = torch.zeros((T, V), dtype=torch.bfloat16, device="cuda")
    x[-3:].normal_(generator=torch.Generator(device="cuda").manual_seed(1))
    t = torch.full((T,), -1, dtype=torch.int64, device="cuda")
    t[-3:] = torch.tensor([0, 131071, 77], device="cuda")
    g = torch.ones(T, device="cuda")
    a = q.token_logprob(x, t)
    b = q.token_logprob(x[-3:].clone(), t[-3:].clone())
    assert torch.equal(a[0][-3:], b[0]) and torch.equal(a[1][-3:], b[1])
    want = q.token_logprob_grad(x[-3:].clone(), t[-3:].clone(), b[1], g[-3:].clone())
    d = q.token_logprob_grad(x, t, a[1], g, inplace=True)
    assert torch.equal(d[-3:], want) and not bool(d[-4].any())


def test_repeats_streams_and_graphs():
    x, t, g = make(30, 20000, torch.bfloat16, seed=7)
    logp, lse = q.token_logprob(x, t)
    d = q.token_logprob_grad(x, t, lse, g)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        l2, s2 = q.token_logprob(x, t)
        d2 = q.token_logprob_grad(x, t, s2, g)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(logp, l2) and torch.equal(lse, s2) and torch.equal(d, d2)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        l3, s3 = q.token_logprob(x, t)
        d3 = q.token_logprob_grad(x, t, s3, g)
    x2, t2, g2 = make(30, 20000, torch.bfloat16, seed=8)
    x.copy_(x2), t.copy_(t2), g.copy_(g2)
    gr.replay()
    l4, s4 = q.token_logprob(x, t)
    assert torch.equal(l3, l4) and torch.equal(d3, q.token_logprob_grad(x, t, s4, g))


def test_columns_behind_a_row_stay():
    x, t, g = make(5, 30, torch.bfloat16, seed=9)
    wide = torch.full((5, 48), 3.0, dtype=torch.bfloat16, device="cuda")
    _, lse = q.token_logprob(x, t)
    q.qurl_token_logprob_grad(x, t, lse, g, wide[:, :30])
    assert bool((wide[:, 30:] == 3).all())
    with pytest.raises(ValueError):
        q.token_logprob(x, t.int())
    with pytest.raises(ValueError):
        q.token_logprob(x, t[:3])
    with pytest.raises(ValueError):
        q.token_logprob_grad(x, t, lse, g, denom=torch.ones(1, device="cuda"))


def test_rows_split_over_clusters():
    """Few rows of every length that is split over 2, 4 or 8 CTAs, padding rows (whose CTAs leave at once) beside
    them, again and again."""
    for T, V in ((1, 8192), (2, 16384), (3, 40000), (7, 32768), (19, 65536), (38, 33000), (150, 8200)):
        x, t, g = make(T, V, torch.bfloat16, seed=T)
        t[1::3] = -1
        logp, lse, _ = check(x, t, g)
        for _ in range(20):
            again = q.token_logprob(x, t)
            assert torch.equal(again[0], logp) and torch.equal(again[1], lse)


def test_denominator_that_counts_nothing():
    """No valid token: zeros, whatever the derivative holds."""
    x, t, g = make(4, 1000, torch.bfloat16, seed=12)
    _, lse = q.token_logprob(x, t)
    g[0], g[1] = INF, float("nan")
    for n in (0.0, -1.0, float("nan")):
        d = q.token_logprob_grad(x, t, lse, g, denom=torch.tensor([n], dtype=torch.float64, device="cuda"))
        assert not bool(d.any())
