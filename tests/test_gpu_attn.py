"""Attention of one new token over the paged FP8 cache (qurl_kv_attn_decode)
against the formula in 64 bits on the cache's own codes and scales.

Tolerances, from the arithmetic.  Scores: the products of a query value and a
code are summed in fp32, so s is within e = (head_dim + 8) 2^-24 sum_d |q_d k_d|
scale of its value, which is the relative error of exp(s) above and below the
fraction.  The weights that multiply the values keep 12 significant bits at
least (2^-12 relative, doubled for the fp32 roundings around them).  So before
its rounding to bf16 (8 significant bits, half a step: 2^-8 of the value) an output is within
(2 e + 2^-11) sum_j p_j |v_j| of the formula's, and lse within e plus a few fp32
roundings."""
import pytest
import torch

import w8a8_precision_gemm_gb300 as q

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _status():
    yield
    q.qurl_check_device_status()


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def make(lens, q_heads, kv_heads, hd, block, seed=0, spare=3, extra=0, peak=1.0, pages=None):
    """Inputs: every sequence's pages scattered over the cache, all slots filled."""
    g = _gen(seed)
    B, longest = len(lens), max(max(lens), 1)
    per = -(-longest // block)
    pages = max(per * B + spare, pages or 0)
    slots = pages * block
    c = {}
    for n in "kv":
        x = torch.randn((slots, kv_heads, hd), device="cuda", generator=g)
        c[n] = (x / x.abs().amax(-1, keepdim=True) * 448).to(torch.float8_e4m3fn)
        c[n + "s"] = (0.5 + torch.rand((slots, kv_heads), device="cuda", generator=g)) * (3.0 / 448)
    table = torch.randperm(pages, device="cuda", generator=g)[:per * B].view(B, per).to(torch.int32)
    qkv = (torch.randn((B, q_heads * hd + extra), device="cuda", generator=g) * peak).to(torch.bfloat16)
    return dict(q=qkv, q_heads=q_heads, k=c["k"], ks=c["ks"], v=c["v"], vs=c["vs"], table=table, block=block,
                lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), scale=hd ** -0.5, window=0)


def run(a, **kw):
    return q.kv_attn_decode(a["q"], a["q_heads"], a["k"], a["ks"], a["v"], a["vs"], a["table"], a["block"], a["lens"],
                            a["scale"], window=a["window"], want_lse=True, **kw)


def reference(a, keep=None):
    """(out, lse, bound of out, bound of lse) in 64 bits; keep(b, positions) -> those that count."""
    B, hq = a["q"].shape[0], a["q_heads"]
    _, kvh, hd = a["k"].shape
    out = torch.zeros((B, hq, hd), dtype=torch.float64, device="cuda")
    mag, lse = torch.zeros_like(out), torch.full((B, hq), float("-inf"), dtype=torch.float64, device="cuda")
    serr = torch.zeros_like(lse)
    for b in range(B):
        n = max(0, min(int(a["lens"][b]), a["table"].shape[1] * a["block"]))
        j = torch.arange(max(0, n - a["window"]) if a["window"] else 0, n, device="cuda")
        if keep is not None:
            j = j[keep(b, j)]
        if not len(j):
            continue
        slot = a["table"][b].long()[j // a["block"]] * a["block"] + j % a["block"]
        k = a["k"].view(torch.uint8)[slot].view(torch.float8_e4m3fn).double() * a["ks"][slot].double()[..., None]
        v = a["v"].view(torch.uint8)[slot].view(torch.float8_e4m3fn).double() * a["vs"][slot].double()[..., None]
        x = a["q"][b, :hq * hd].double().view(kvh, -1, hd)
        s = torch.einsum("hgd,lhd->hgl", x, k) * a["scale"]
        p = torch.softmax(s, -1)
        out[b] = torch.einsum("hgl,lhd->hgd", p, v).reshape(hq, hd)
        mag[b] = torch.einsum("hgl,lhd->hgd", p, v.abs()).reshape(hq, hd)
        lse[b] = torch.logsumexp(s, -1).reshape(hq)
        serr[b] = (torch.einsum("hgd,lhd->hgl", x.abs(), k.abs()) * abs(a["scale"])).amax(-1).reshape(hq)
    serr = (hd + 8) * 2.0 ** -24 * serr
    assert float(serr.max()) < 2.0 ** -6, "inputs outside what the bounds were derived for"
    tol = out.abs() * 2.0 ** -8 + mag * (2 * serr + 2.0 ** -11)[..., None] + 1e-30
    fin = torch.where(torch.isfinite(lse), lse, 0.0)
    return out.reshape(B, -1), lse, tol.reshape(B, -1), serr + 2.0 ** -21 * (1 + fin.abs())


def check(a, got=None, keep=None):
    o, l = run(a) if got is None else got
    ro, rl, to, tl = reference(a, keep)
    assert bool((o.double() - ro).abs().le(to).all()), float(((o.double() - ro).abs() / to).max())
    empty = torch.isinf(rl)
    assert torch.equal(torch.isinf(l), empty) and bool((l[empty] < 0).all())
    d = torch.where(empty, 0.0, l.double() - rl).abs()
    assert bool(d.le(tl).all()), float((d / tl).max())


@pytest.mark.parametrize("q_heads,kv_heads", [(1, 1), (4, 4), (28, 4), (40, 8), (16, 1), (17, 1), (33, 1), (12, 2), (30, 3)])
def test_head_groups(q_heads, kv_heads):
    check(make([1, 130, 300], q_heads, kv_heads, 128, 16, seed=q_heads))


@pytest.mark.parametrize("hd", [16, 32, 48, 64, 80, 96, 112, 128, 144, 160, 192, 240, 256])
def test_head_dims(hd):
    check(make([77, 260], 10, 2, hd, 16, seed=hd))


@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 31, 32, 33, 127, 128, 129, 255, 256, 257, 511, 513, 1000, 4097])
def test_lengths(length):
    check(make([length], 7, 1, 128, 16, seed=length))


@pytest.mark.parametrize("block", [1, 2, 3, 5, 7, 16, 24, 48, 100, 128, 129, 256, 1000])
def test_page_sizes(block):
    check(make([1, 128, 401, 640], 8, 2, 64, block, seed=block))


@pytest.mark.parametrize("lens", [[0], [0, 0, 0], [0, 5, 0, 300, 0], [-3, 17], [1] * 200, list(range(0, 600, 37))])
def test_empty_and_ragged(lens):
    check(make(lens, 10, 2, 128, 16, seed=len(lens)))


@pytest.mark.parametrize("window", [1, 2, 100, 128, 129, 1000, 5000])
def test_window(window):
    a = make([0, 1, 100, 500, 1500], 10, 2, 128, 16, seed=window)
    a["window"] = window
    check(a)


def test_long_sequences_and_batches():
    check(make([70000, 3, 20011], 5, 1, 128, 64, seed=5))
    check(make([2048 + 13 * i for i in range(48)], 40, 8, 128, 16, seed=6))


def test_sequences_over_many_ranges():
    """One KV head, sequences that begin and end inside ranges of their neighbours: partial sums joined in groups."""
    check(make([20000, 9000, 31234, 128, 17, 12345], 8, 1, 64, 32, seed=21))
    check(make([150001], 2, 1, 32, 128, seed=22))
    check(make([5000] * 9, 3, 3, 64, 16, seed=23))


def test_peaked_and_flat_scores():
    check(make([900], 10, 2, 128, 16, seed=1, peak=6.0))
    a = make([900], 10, 2, 128, 16, seed=2)
    a["q"].zero_()  # every token alike
    check(a)
    # a running maximum that grows along the sequence, and one token far above the rest
    a = make([1500], 4, 1, 64, 16, seed=3)
    slot = a["table"][0].long().repeat_interleave(16)[:1500] * 16 + torch.arange(1500, device="cuda") % 16
    a["ks"][slot] *= torch.linspace(0.1, 2.0, 1500, device="cuda")[:, None]
    check(a)


def test_scales_of_every_size():
    """Value scales that span 2^40 between tokens, key scales of zero, codes at both ends of e4m3."""
    a = make([700, 260], 8, 2, 128, 16, seed=8)
    g = _gen(9)
    a["vs"].copy_(torch.exp2(torch.randint(-30, 11, a["vs"].shape, device="cuda", generator=g).float()))
    a["ks"][::3] = 0.0
    a["v"].view(torch.uint8)[::5] = 0x7E   # 448
    a["v"].view(torch.uint8)[1::5] = 0x01  # 2^-9
    a["v"].view(torch.uint8)[2::5] = 0x80  # -0
    check(a)


def test_query_values_of_every_size():
    a = make([300], 8, 2, 128, 16, seed=12)
    e = torch.randint(-40, 1, a["q"].shape, device="cuda", generator=_gen(1)).float()
    a["q"].copy_((a["q"].float() * torch.exp2(e)).to(torch.bfloat16))
    check(a)
    a["q"].mul_(2.0 ** 60)
    a["scale"] = a["scale"] * 2.0 ** -60
    check(a)
    a["scale"] = 0.0
    check(a)
    a["scale"] = -0.1
    a["q"].mul_(2.0 ** -60)
    check(a)


def test_unused_slots_and_pages_are_not_read():
    """NaN codes and scales in every slot no sequence sees, table entries past a sequence's pages out of range."""
    a = make([0, 40, 130, 257], 10, 2, 128, 16, seed=4)
    used = torch.zeros(a["k"].shape[0], dtype=torch.bool, device="cuda")
    for b in range(4):
        n = int(a["lens"][b])
        j = torch.arange(n, device="cuda")
        used[a["table"][b].long()[j // 16] * 16 + j % 16] = True
        a["table"][b, -(-n // 16):] = 2 ** 30 if b % 2 else -7
    for n in "kv":
        a[n].view(torch.uint8)[~used] = 0x7F  # NaN
        a[n + "s"][~used] = float("nan")
    check(a)


def test_strides_and_neighbours():
    """The fused qkv output as q, a wide output, a table that is a slice: what lies beside the rows stays."""
    a = make([33, 200, 5], 6, 2, 64, 16, seed=3, extra=2 * 2 * 64)
    wide = torch.full((5, 6 * 64 + 32), 7.0, dtype=torch.bfloat16, device="cuda")
    table = torch.full((3, a["table"].shape[1] + 5), -1, dtype=torch.int32, device="cuda")
    table[:, :a["table"].shape[1]] = a["table"]
    a["table"] = table[:, :a["table"].shape[1]]
    lse = torch.full((3, 6), 7.0, device="cuda")
    ws = q.kv_attn_workspace(3, 6, 2, 64, a["table"].shape[1], 16)
    q.qurl_kv_attn_decode(a["q"], 6, a["k"], a["ks"], a["v"], a["vs"], a["table"], 16, a["lens"], a["scale"],
                          wide[:3, :6 * 64], ws, lse=lse)
    check(a, (wide[:3, :6 * 64], lse))
    assert bool((wide[3:] == 7).all()) and bool((wide[:, 6 * 64:] == 7).all())
    out2 = torch.empty_like(wide)
    q.qurl_kv_attn_decode(a["q"], 6, a["k"], a["ks"], a["v"], a["vs"], a["table"], 16, a["lens"], a["scale"],
                          out2[:3, :6 * 64], ws)  # without lse
    assert torch.equal(out2[:3, :6 * 64], wide[:3, :6 * 64])


def test_bad_pages_and_lengths_are_reported_and_left_out():
    a = make([100, 64, 50], 10, 2, 128, 16, seed=7)
    a["table"][0, 2] = -1
    a["table"][1, 1] = a["k"].shape[0] // 16  # one page past the cache
    a["lens"][2] = 10 ** 6                    # longer than its table
    o, l = run(a)
    with pytest.raises(q.QurlError):
        q.qurl_check_device_status()
    bad = {0: 2, 1: 1}
    check(a, (o, l), keep=lambda b, j: (j // 16) != bad.get(b, -1))
    a = make([40], 2, 1, 64, 16, seed=7)
    a["table"].fill_(-1)
    o, l = run(a)
    with pytest.raises(q.QurlError):
        q.qurl_check_device_status()
    assert bool((o == 0).all()) and bool((l == float("-inf")).all())


def test_workspace_reuse_repeats_and_streams():
    """One workspace over calls of different shapes; identical bits on repeat, on another stream, in a graph."""
    big = make([3000, 10, 0, 777], 40, 8, 128, 16, seed=1)
    small = make([1, 129], 10, 2, 128, 16, seed=2)
    ws = q.kv_attn_workspace(4, 40, 8, 128, big["table"].shape[1], 16)
    first = run(big, ws=ws)
    check(big, first)
    check(small, run(small, ws=ws))
    again = run(big, ws=ws)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = run(big, ws=ws)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(first[0], other[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = run(big, ws=ws)
    for n in (3000, 64, 1):
        big["lens"][0] = n  # the lengths are read at replay
        g.replay()
        check(big, captured)


def test_small_workspace_is_refused():
    a = make([5], 2, 1, 64, 16)
    need = q.qurl_kv_attn_workspace_size(1, 2, 1, 64, 1, 16)
    with pytest.raises(q.QurlError, match="WORKSPACE"):
        run(a, ws=torch.zeros(need - 1, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("e", [-18, -20, -24, -30, -60])
@pytest.mark.parametrize("q_heads,kv_heads,hd", [(10, 2, 128), (7, 1, 128), (5, 1, 256), (8, 1, 192)])
def test_attended_tokens_of_small_value_scale(q_heads, kv_heads, hd, e):
    """Each query head attends one token whose value scale is 2^e of its neighbours' (the heads of a group
    attend different tokens of one tile, each of another scale): what the others weigh, 2^-40 and less, leaves
    the output to that token where its scale is not below theirs by as much, and to all of them where it is."""
    a = make([300, 128, 700], q_heads, kv_heads, hd, 16, seed=q_heads)
    group, part = q_heads // kv_heads, 16 * (hd // 16 // (q_heads // kv_heads))
    x = torch.zeros((3, kv_heads, group, hd), device="cuda")
    for b in range(3):
        for h in range(group):
            j = int(a["lens"][b]) - 1 - 3 * h
            slot = int(a["table"][b, j // 16]) * 16 + j % 16
            x[b, :, h, part * h:part * (h + 1)] = 40.0 * hd ** 0.5 / part / 3.0
            a["k"][slot] = torch.zeros((kv_heads, hd), device="cuda").to(torch.float8_e4m3fn)
            a["k"][slot, :, part * h:part * (h + 1)] = torch.full((kv_heads, part), 448.0, device="cuda").to(torch.float8_e4m3fn)
            a["ks"][slot] = 3.0 / 448
            a["vs"][slot] *= 2.0 ** (e - h)
    a["q"] = x.reshape(3, -1).to(torch.bfloat16)
    check(a)


def test_workspace_of_another_head_layout():
    """A workspace serves any layout it is large enough for, whatever layouts ran on it before: sequences over
    many ranges leave partial sums everywhere, then a layout whose counters lie elsewhere joins in groups."""
    big = make([1664, 8064], 32, 32, 128, 16, seed=41)
    others = [make([40000, 1], 4, 1, 64, 64, seed=42), make([9000], 2, 1, 256, 64, seed=43),
              make([6000, 300], 28, 4, 128, 16, seed=44)]
    sizes = [q.qurl_kv_attn_workspace_size(a["q"].shape[0], a["q_heads"], a["k"].shape[1], a["k"].shape[2],
                                           a["table"].shape[1], a["block"]) for a in [big] + others]
    ws = torch.zeros(max(sizes), dtype=torch.uint8, device="cuda")
    for a in others:
        check(a, run(a, ws=ws))
        check(big, run(big, ws=ws))
        check(a, run(a, ws=ws))


def test_scores_of_any_size():
    """Scores far below any that a mask would have: a softmax takes only their differences."""
    a = make([1, 2, 200], 5, 1, 64, 16, seed=31)
    a["k"].copy_(torch.full(a["k"].shape, 448.0, device="cuda").to(torch.float8_e4m3fn))
    a["ks"].fill_(1.0 / 448)
    a["q"].fill_(2.0 ** 100)
    a["scale"] = -1.0
    o, l = run(a)
    # eight roundings of 2^-24: the key's scale, log2(e) and ln(2) as constants, and the four products and the sum
    # between the raw score and lse
    assert bool((l.double() / (-64 * 2.0 ** 100) - 1).abs().le(2.0 ** -21).all())
    for b, n in enumerate((1, 2, 200)):
        j = torch.arange(n, device="cuda")
        slot = a["table"][b].long()[j // 16] * 16 + j % 16
        v = a["v"].view(torch.uint8)[slot, 0].view(torch.float8_e4m3fn).double() * a["vs"][slot].double()
        want, mag = v.mean(0), v.abs().mean(0)
        d = (o[b].double().view(5, 64) - want).abs()
        assert bool(d.le(want.abs() * 2.0 ** -8 + mag * 2.0 ** -11).all()), b


def test_behind_a_timeout_of_another_kernel():
    """A GEMM's wait has run out and is not looked at yet: the attention behind it may give up, but what it stores
    is right; with the status read and the workspace zeroed it runs as ever."""
    a = make([3000, 10, 0, 777], 10, 2, 128, 16, seed=51)
    ws = q.kv_attn_workspace(4, 10, 2, 128, a["table"].shape[1], 16)
    want = run(a, ws=ws)
    X, W = torch.randn((16, 256), device="cuda").to(torch.bfloat16), torch.randn((512, 256), device="cuda")
    Wq, sw, _, _ = q.prepare_weights(W, q.FP8_E4M3, keep_scaled=False)
    Xq, sx = q.quant_act(X, q.FP8_E4M3)
    gws = q.workspace(16, 512, 256, q.FP8_E4M3)
    out, lse = torch.full_like(want[0], 7.0), torch.full_like(want[1], 7.0)
    q.qurl_check_device_status()
    q.qurl_debug_inject_timeout()
    q.linear(Xq, sx, Wq, sw, q.FP8_E4M3, gws)
    q.qurl_kv_attn_decode(a["q"], 10, a["k"], a["ks"], a["v"], a["vs"], a["table"], 16, a["lens"], a["scale"], out, ws,
                          lse=lse)
    with pytest.raises(q.QurlError) as e:
        q.qurl_check_device_status()
    assert e.value.status == 6  # QURL_ERR_TIMEOUT
    per_head = out.view(4, 10, 128)
    left = (per_head == 7.0).all(-1)
    assert bool((left | (per_head == want[0].view(4, 10, 128)).all(-1)).all())
    assert bool(((lse == 7.0) | (lse == want[1])).all())
    ws.zero_()
    got = run(a, ws=ws)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("q_heads,kv_heads,hd", [(7, 1, 144), (8, 1, 256), (16, 1, 192), (20, 1, 256), (12, 2, 240), (5, 1, 160)])
def test_wide_heads_over_many_ranges(q_heads, kv_heads, hd):
    """Heads of two panels, up to eight query heads a unit, sequences joined from two ranges and from groups of
    them."""
    check(make([5000, 1, 700, 0, 333], q_heads, kv_heads, hd, 16, seed=hd))
    check(make([15000, 9000, 20011], q_heads, kv_heads, hd, 64, seed=hd + 1))


def test_offsets_past_32_bits():
    """Pages at both ends of caches of more than 2^32 bytes."""
    block, kvh, hd = 16, 8, 256
    pages = (2 ** 32 // (kvh * hd * block)) + 40
    g = _gen(61)
    kc, ks, vc, vs = q.kv_cache(pages * block, kvh, hd)
    small = make([300, 77], 16, kvh, hd, block, seed=61, pages=60)
    per = small["table"].shape[1]
    table = torch.stack([pages - 1 - torch.arange(per), pages - 1 - per - torch.arange(per)]).int().cuda()
    table[1, :2] = torch.tensor([3, 1])
    slot = lambda t: (t.long()[..., None] * block + torch.arange(block, device="cuda")).reshape(-1)  # noqa: E731
    for big, name in ((kc, "k"), (vc, "v")):
        big.view(torch.uint8)[slot(table)] = small[name].view(torch.uint8)[slot(small["table"])]
    for big, name in ((ks, "ks"), (vs, "vs")):
        big[slot(table)] = small[name][slot(small["table"])]
    want = run(small)
    check(small, want)
    got = run(small | dict(k=kc, ks=ks, v=vc, vs=vs, table=table))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("peak", [0.0, 1.0, 4.0, 12.0])
def test_attended_tokens_without_a_value(peak):
    """The tokens that every head attends have a value scale of 0, as have others at random: what is left comes
    from weights far below the largest."""
    a = make([300, 128, 5, 700], 10, 2, 128, 16, seed=71)
    g = _gen(72)
    a["vs"].masked_fill_(torch.rand(a["vs"].shape, device="cuda", generator=g) < 0.3, 0.0)
    a["q"].fill_(peak / 8)
    for b in range(4):
        for j in (0, int(a["lens"][b]) // 2):
            slot = int(a["table"][b, j // 16]) * 16 + j % 16
            a["k"][slot] = torch.full((2, 128), 448.0, device="cuda").to(torch.float8_e4m3fn)
            a["vs"][slot] = 0.0
    check(a)
