"""Causal attention of several new tokens per sequence over the paged FP8 cache
(qurl_kv_attn_chunk) against the formula in 64 bits on the cache's own codes and scales.

Tolerances, from the arithmetic.  A query row is scaled so that its largest value is in [2^7, 2^8) and enters as e4m3
(4 significant bits, steps of 2^-9 below 2^-6) and the rest as e5m2 (3 bits, steps of 2^-16 below 2^-14).  A bf16 value has
8 bits: from 2^-6 on the rest is at most 8 units of its last place, whole ones of 2^-13 at least, and exact; below, the rest is at
most 2^-10 and off by at most half a step there, 2^-14: 2^-21 of the row's largest.  Products with a code are
exact and summed in fp32, so s is within e = ((head_dim + 8) 2^-24 sum_d |q_d k_d| + 2^-21 max |q| sum_d |k_d|) scale of
its value, which is the relative error of exp(s) above and below the fraction.  A weight is rounded to fp16, half a step: 2^-11 of
the value (with the fp32 roundings around it 2^-10.9), or 2^-27 of the row's largest weight
(of exp(s) times the value's scale) where that is more; a tensor-core sum in fp32 adds 2^-20
of the magnitudes.  So before its rounding to bf16 (half a step: 2^-8 of the value) an output is
within (2 e + 2^-10.9 + 2^-20) sum_j p_j |v_j| + 2^-27 448 n max_j p_j |vs_j| of the formula's (n tokens, the
codes' largest), and lse within e plus a few fp32 roundings."""
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


def make(spans, q_heads, kv_heads, hd, block, seed=0, spare=3, extra=0, peak=1.0, pages=None, pad=0):
    """Inputs for sequences of (cached, new) tokens: pages scattered over the cache, all slots filled."""
    g = _gen(seed)
    B, lens = len(spans), [max(c + n, 0) for c, n in spans]
    per = -(-max(max(lens), 1) // block)
    pages = max(per * B + spare, pages or 0)
    slots = pages * block
    c = {}
    for n in "kv":
        x = torch.randn((slots, kv_heads, hd), device="cuda", generator=g)
        c[n] = (x / x.abs().amax(-1, keepdim=True) * 448).to(torch.float8_e4m3fn)
        c[n + "s"] = (0.5 + torch.rand((slots, kv_heads), device="cuda", generator=g)) * (3.0 / 448)
    table = torch.randperm(pages, device="cuda", generator=g)[:per * B].view(B, per).to(torch.int32)
    new = [n for _, n in spans]
    x = (torch.randn((sum(new) + pad, q_heads * hd + extra), device="cuda", generator=g) * peak).to(torch.bfloat16)
    cu = torch.tensor([0] + new).cumsum(0).to(torch.int32).cuda()
    return dict(q=x, q_heads=q_heads, k=c["k"], ks=c["ks"], v=c["v"], vs=c["vs"], table=table, block=block, cu=cu,
                lens=torch.tensor([a + b for a, b in spans], dtype=torch.int32, device="cuda"), scale=hd ** -0.5, window=0)


def run(a, **kw):
    return q.kv_attn_chunk(a["q"], a["q_heads"], a["k"], a["ks"], a["v"], a["vs"], a["table"], a["block"], a["cu"], a["lens"],
                           a["scale"], window=a["window"], want_lse=True, **kw)


def reference(a, keep=None):
    """(out, lse, bound of out, bound of lse) in 64 bits; keep(b, positions) -> those that count."""
    M, hq = a["q"].shape[0], a["q_heads"]
    _, kvh, hd = a["k"].shape
    out = torch.zeros((M, hq, hd), dtype=torch.float64, device="cuda")
    tol, lse = torch.zeros_like(out), torch.full((M, hq), float("-inf"), dtype=torch.float64, device="cuda")
    serr = torch.zeros_like(lse)
    for b in range(len(a["lens"])):
        r0, r1 = int(a["cu"][b]), int(a["cu"][b + 1])
        n = max(0, min(int(a["lens"][b]), a["table"].shape[1] * a["block"]))
        j = torch.arange(n, device="cuda")
        if keep is not None:
            j = j[keep(b, j)]
        if r1 <= r0 or not len(j):
            continue
        slot = a["table"][b].long()[j // a["block"]] * a["block"] + j % a["block"]
        k = a["k"].view(torch.uint8)[slot].view(torch.float8_e4m3fn).double() * a["ks"][slot].double()[..., None]
        v = a["v"].view(torch.uint8)[slot].view(torch.float8_e4m3fn).double() * a["vs"][slot].double()[..., None]
        vs = a["vs"][slot].double().abs().T[:, None, None]                                    # [kvh, 1, 1, l]
        step = max(1, (1 << 26) // (hq * len(j)))
        for i in range(r0, r1, step):
            rows = torch.arange(i, min(i + step, r1), device="cuda")
            pos = n - (r1 - r0) + rows - r0
            hide = j[None] > pos[:, None]
            if a["window"]:
                hide = hide | (j[None] <= pos[:, None] - a["window"])
            x = a["q"][rows, :hq * hd].double().view(len(rows), kvh, -1, hd)
            s = (torch.einsum("mhgd,lhd->hgml", x, k) * a["scale"]).masked_fill(hide, float("-inf"))
            some = (~hide).any(-1)
            p = torch.nan_to_num(torch.softmax(s, -1))
            o = torch.einsum("hgml,lhd->mhgd", p, v).reshape(len(rows), hq, hd)
            mag = torch.einsum("hgml,lhd->mhgd", p, v.abs()).reshape(len(rows), hq, hd)
            out[rows] = o
            lse[rows] = torch.logsumexp(s, -1).permute(2, 0, 1).reshape(len(rows), hq)
            e = torch.einsum("mhgd,lhd->hgml", x.abs(), k.abs()) * abs(a["scale"])
            small = torch.einsum("mhg,lh->hgml", x.abs().amax(-1), k.abs().sum(-1)) * abs(a["scale"])
            e = ((hd + 8) * 2.0 ** -24 * e + 2.0 ** -21 * small).masked_fill(hide, 0.0).amax(-1).permute(2, 0, 1).reshape(len(rows), hq)
            serr[rows] = e
            top = (p * vs).amax(-1).permute(2, 0, 1).reshape(len(rows), hq)
            low = 2.0 ** -27 * 448 * len(j) * top
            tol[rows] = o.abs() * 2.0 ** -8 * 1.002 + mag * (2 * e + 2.0 ** -10.9 + 2.0 ** -20)[..., None] + low[..., None] + 1e-30
            assert bool((torch.isinf(lse[rows]) == ~some[:, None]).all())
    assert M == 0 or float(serr.max()) < 2.0 ** -6, "inputs outside what the bounds were derived for"
    fin = torch.where(torch.isfinite(lse), lse, 0.0)
    return out.reshape(M, hq * hd), lse, tol.reshape(M, hq * hd), serr + 2.0 ** -20 * (1 + fin.abs())


def check(a, got=None, keep=None):
    o, l = run(a) if got is None else got
    rows = slice(int(a["cu"][0]), int(a["cu"][-1]))
    ro, rl, to, tl = (t[rows] for t in reference(a, keep))
    o, l = o[rows], l[rows]
    d = (o.double() - ro).abs()
    assert bool(d.le(to).all()), (float((d / to).max()), (d / to).nan_to_num(1e9).amax(-1).argmax().item())
    empty = torch.isinf(rl)
    assert torch.equal(torch.isinf(l), empty) and bool((l[empty] < 0).all())
    d = torch.where(empty, 0.0, l.double() - rl).abs()
    assert bool(d.le(tl).all()), float((d / tl).max())


def test_one_tile():
    check(make([(0, 16)], 1, 1, 64, 16))
    check(make([(0, 128)], 1, 1, 64, 16))
    check(make([(0, 100)], 1, 1, 128, 16))


@pytest.mark.parametrize("hd", [16, 32, 48, 64, 80, 96, 112, 128, 144, 160, 192, 208, 240, 256])
def test_head_dims(hd):
    check(make([(0, 77), (260, 40), (5, 1)], 10, 2, hd, 16, seed=hd))


@pytest.mark.parametrize("q_heads,kv_heads", [(1, 1), (4, 4), (28, 4), (40, 8), (16, 1), (17, 1), (12, 2), (30, 3), (129, 1), (300, 1),
                                              (257, 1)])
def test_head_groups(q_heads, kv_heads):
    check(make([(0, 130), (300, 3), (0, 1)], q_heads, kv_heads, 128, 16, seed=q_heads))
    check(make([(7, 50)], q_heads, kv_heads, 192, 16, seed=q_heads))


@pytest.mark.parametrize("new", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 513, 1000])
def test_lengths(new):
    check(make([(0, new)], 3, 1, 128, 16, seed=new))
    check(make([(new, 5), (3, new), (1000 - new, new)], 2, 1, 64, 16, seed=new))
    check(make([(130, new)], 2, 2, 256, 16, seed=new))


@pytest.mark.parametrize("block", [1, 2, 3, 5, 7, 16, 24, 48, 100, 128, 129, 256, 1000])
def test_page_sizes(block):
    check(make([(0, 1), (128, 20), (0, 401), (600, 40)], 8, 2, 64, block, seed=block))
    check(make([(0, 90), (300, 20)], 4, 2, 160, block, seed=block))


@pytest.mark.parametrize("spans", [[(0, 0)], [(0, 0), (5, 0), (0, 3)], [(300, 0), (0, 300), (0, 0), (7, 1), (0, 0)],
                                   [(i, 1) for i in range(200)], [(37 * i, 5 * i) for i in range(20)],
                                   [(3 * i % 200, i % 4) for i in range(1500)]])
def test_empty_and_ragged(spans):
    check(make(spans, 10, 2, 128, 16, seed=len(spans)))


def test_single_tokens_are_decode():
    """A batch of single tokens is what qurl_kv_attn_decode computes, to both kernels' tolerances."""
    a = make([(n, 1) for n in (0, 17, 300, 1000, 4095)], 40, 8, 128, 16, seed=4)
    o, l = run(a)
    check(a, (o, l))
    od, ld = q.kv_attn_decode(a["q"], 40, a["k"], a["ks"], a["v"], a["vs"], a["table"], 16, a["lens"], a["scale"], want_lse=True)
    _, _, to, tl = reference(a)
    assert bool((o.double() - od.double()).abs().le(2 * to).all()) and bool((l - ld).abs().le(2 * tl).all())


@pytest.mark.parametrize("window", [1, 2, 100, 128, 129, 1000, 5000])
def test_window(window):
    a = make([(0, 0), (0, 1), (100, 30), (0, 500), (1500, 200), (900, 1)], 10, 2, 128, 16, seed=window)
    a["window"] = window
    check(a)
    a = make([(100, 300), (700, 5)], 2, 1, 192, 16, seed=window)
    a["window"] = window
    check(a)


def test_long_prompts_and_caches():
    check(make([(0, 3000)], 8, 2, 128, 64, seed=5))
    check(make([(70000, 3), (20011, 70), (3, 2)], 5, 1, 128, 64, seed=6))
    check(make([(2048 + 13 * i, 4) for i in range(48)], 40, 8, 128, 16, seed=7))
    check(make([(30000, 300)], 4, 1, 256, 64, seed=8))


def test_units_over_many_ranges():
    """Units cut into two and into many parts, next to whole ones."""
    check(make([(20000, 9), (9000, 100), (31234, 1), (128, 60), (17, 17), (12345, 30)], 8, 1, 64, 32, seed=21))
    check(make([(150001, 2)], 2, 1, 32, 128, seed=22))
    check(make([(5000, 64)] * 9, 3, 3, 64, 16, seed=23))
    check(make([(9000, 33), (100, 1000)], 6, 2, 160, 16, seed=24))


def test_units_of_one_and_two_row_tiles_in_turn():
    """Sequences whose last unit has one row tile, with many tiles of tokens, before and between units of two."""
    check(make([(n, 210 + n % 3) for n in range(0, 1800, 60)], 10, 2, 128, 16, seed=41))
    check(make([(1500, 65 + i % 2) for i in range(60)], 12, 3, 64, 16, seed=42))
    check(make([(3000 * (i % 3), 33) for i in range(40)], 16, 2, 80, 16, seed=43))
    check(make([(2000, 1), (0, 300)] * 40, 10, 2, 128, 16, seed=44))


def test_many_units_of_a_sequence():
    """More units than a warp looks at together, the ranges' borders anywhere among them."""
    check(make([(0, 12000), (50, 700)], 2, 1, 16, 64, seed=31))
    check(make([(10, 4500)], 16, 1, 32, 64, seed=32))


def test_peaked_and_flat_scores():
    check(make([(500, 100)], 10, 2, 128, 16, seed=1, peak=6.0))
    a = make([(500, 400)], 10, 2, 128, 16, seed=2)
    a["q"].zero_()  # every token alike
    check(a)
    # a running maximum that grows along the sequence
    a = make([(1200, 300)], 4, 1, 64, 16, seed=3)
    slot = a["table"][0].long().repeat_interleave(16)[:1500] * 16 + torch.arange(1500, device="cuda") % 16
    a["ks"][slot] *= torch.linspace(0.1, 2.0, 1500, device="cuda")[:, None]
    check(a)
    a["q"].mul_(8)
    check(a)


def test_scales_of_every_size():
    """Value scales that span 2^40 between tokens, key scales of zero, codes at both ends of e4m3."""
    a = make([(500, 200), (0, 260), (90, 1)], 8, 2, 128, 16, seed=8)
    g = _gen(9)
    a["vs"].copy_(torch.exp2(torch.randint(-30, 11, a["vs"].shape, device="cuda", generator=g).float()))
    a["ks"][::3] = 0.0
    a["v"].view(torch.uint8)[::5] = 0x7E   # 448
    a["v"].view(torch.uint8)[1::5] = 0x01  # 2^-9
    a["v"].view(torch.uint8)[2::5] = 0x80  # -0
    check(a)
    a["vs"].mul_(2.0 ** -60)
    check(a)
    a["vs"].mul_(-2.0 ** 120)
    check(a)


@pytest.mark.parametrize("e", [-6, -12, -18, -24, -30, -60])
@pytest.mark.parametrize("q_heads,kv_heads,hd", [(10, 2, 128), (7, 1, 64), (4, 1, 256)])
def test_attended_tokens_of_small_value_scale(q_heads, kv_heads, hd, e):
    """Each query head attends one token whose value scale is 2^e of its neighbours'."""
    a = make([(299, 1), (100, 28), (690, 10)], q_heads, kv_heads, hd, 16, seed=q_heads)
    group, part = q_heads // kv_heads, 16 * (hd // 16 // (q_heads // kv_heads)) or 8
    x = torch.zeros((a["q"].shape[0], kv_heads, group, hd), device="cuda")
    for b in range(3):
        first = int(a["lens"][b]) - (int(a["cu"][b + 1]) - int(a["cu"][b]))
        for h in range(group):
            j = first - 3 * h
            slot = int(a["table"][b, j // 16]) * 16 + j % 16
            x[int(a["cu"][b]):int(a["cu"][b + 1]), :, h, part * h:part * (h + 1)] = 40.0 * hd ** 0.5 / part / 3.0
            a["k"][slot] = torch.zeros((kv_heads, hd), device="cuda").to(torch.float8_e4m3fn)
            a["k"][slot, :, part * h:part * (h + 1)] = torch.full((kv_heads, part), 448.0, device="cuda").to(torch.float8_e4m3fn)
            a["ks"][slot] = 3.0 / 448
            a["vs"][slot] *= 2.0 ** (e - h)
    a["q"] = x.reshape(x.shape[0], -1).to(torch.bfloat16)
    check(a)


@pytest.mark.parametrize("peak", [0.0, 1.0, 4.0, 12.0])
def test_attended_tokens_without_a_value(peak):
    """The tokens that every head attends have a value scale of 0, as have others at random."""
    a = make([(200, 100), (100, 28), (0, 5), (640, 60)], 10, 2, 128, 16, seed=71)
    g = _gen(72)
    a["vs"].masked_fill_(torch.rand(a["vs"].shape, device="cuda", generator=g) < 0.3, 0.0)
    a["q"].fill_(peak / 8)
    for b in range(4):
        for j in (0, int(a["lens"][b]) // 2):
            slot = int(a["table"][b, j // 16]) * 16 + j % 16
            a["k"][slot] = torch.full((2, 128), 448.0, device="cuda").to(torch.float8_e4m3fn)
            a["vs"][slot] = 0.0
    check(a)
    a["vs"].zero_()
    assert bool((run(a)[0] == 0).all())


def test_query_values_of_every_size():
    a = make([(200, 100)], 8, 2, 128, 16, seed=12)
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


def test_scores_of_any_size():
    """Scores far below any that a mask would have: a softmax takes only their differences."""
    a = make([(0, 1), (0, 2), (150, 50)], 5, 1, 64, 16, seed=31)
    a["k"].copy_(torch.full(a["k"].shape, 448.0, device="cuda").to(torch.float8_e4m3fn))
    a["ks"].fill_(1.0 / 448)
    for big in (2.0 ** 20, 2.0 ** 100):
        a["q"].fill_(big)
        a["scale"] = -1.0
        o, l = run(a)
        # eight roundings of 2^-24: the key's scale, log2(e) and ln(2) as constants, and the four products and the sum
        # between the raw score and lse
        assert bool((l.double() / (-64 * big) - 1).abs().le(2.0 ** -21).all())
        for b in range(3):
            r0, r1, n = int(a["cu"][b]), int(a["cu"][b + 1]), int(a["lens"][b])
            for r in range(r0, r1):
                j = torch.arange(n - (r1 - 1 - r), device="cuda")
                slot = a["table"][b].long()[j // 16] * 16 + j % 16
                v = a["v"].view(torch.uint8)[slot, 0].view(torch.float8_e4m3fn).double() * a["vs"][slot].double()
                want, mag = v.mean(0), v.abs().mean(0)
                d = (o[r].double().view(5, 64) - want).abs()
                assert bool(d.le(want.abs() * 2.0 ** -8 * 1.002 + mag * 2.0 ** -10).all()), (b, r)


def test_later_tokens_do_not_reach_earlier_queries():
    """Scales of infinity and NaN, and other codes, in the tokens behind a query leave its result as it is, to the bit;
    what is not in any sequence is not read at all."""
    a = make([(100, 60), (0, 200), (0, 40)], 10, 2, 128, 16, seed=9)
    want = run(a)
    used = torch.zeros(a["k"].shape[0], dtype=torch.bool, device="cuda")
    late = []
    for b in range(3):
        n, cut = int(a["lens"][b]), int(a["lens"][b]) - 25
        j = torch.arange(n, device="cuda")
        slot = a["table"][b].long()[j // 16] * 16 + j % 16
        used[slot] = True
        late.append(slot[cut:])
        a["table"][b, -(-n // 16):] = 2 ** 30 if b % 2 else -7
    late = torch.cat(late)
    for n in "kv":
        a[n].view(torch.uint8)[~used] = 0x7F
        a[n + "s"][~used] = float("nan")
    got = run(a)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    a["k"].view(torch.uint8)[late] ^= 0x15
    a["ks"][late] = float("inf")
    a["vs"][late[::2]] = float("inf")
    a["vs"][late[1::2]] = float("nan")
    got = run(a)
    rows = torch.cat([torch.arange(int(a["cu"][b]), int(a["cu"][b + 1]) - 25, device="cuda") for b in range(3)])
    # (a tile with such scales takes its references another way: the same to the rounding of the weights)
    plain = a["k"].clone()
    plain.view(torch.uint8)[late] = 0
    ro, rl, to, tl = reference(a | dict(k=plain, ks=torch.where(torch.isfinite(a["ks"]), a["ks"], 0.0),
                                        vs=torch.where(torch.isfinite(a["vs"]), a["vs"], 0.0)))
    assert bool((got[0].double() - ro).abs().le(to)[rows].all()) and bool((got[1].double() - rl).abs().le(tl)[rows].all())


def test_strides_and_neighbours():
    """The fused qkv output as q, a wide output, a table that is a slice, rows of padding: what lies beside stays."""
    a = make([(33, 3), (150, 50), (0, 5)], 6, 2, 64, 16, seed=3, extra=2 * 2 * 64, pad=9)
    M = a["q"].shape[0]
    wide = torch.full((M + 2, 6 * 64 + 32), 7.0, dtype=torch.bfloat16, device="cuda")
    table = torch.full((3, a["table"].shape[1] + 5), -1, dtype=torch.int32, device="cuda")
    table[:, :a["table"].shape[1]] = a["table"]
    a["table"] = table[:, :a["table"].shape[1]]
    a["q"][58:] = float("nan")
    lse = torch.full((M, 6), 7.0, device="cuda")
    ws = q.kv_attn_chunk_workspace(6, 2, 64)
    args = (a["q"], 6, a["k"], a["ks"], a["v"], a["vs"], a["table"], 16, a["cu"], a["lens"], a["scale"])
    q.qurl_kv_attn_chunk(*args, wide[:M, :6 * 64], ws, lse=lse)
    a["q"][58:] = 0.0
    check(a, (wide[:M, :6 * 64], lse))
    assert bool((wide[58:] == 7).all()) and bool((wide[:, 6 * 64:] == 7).all()) and bool((lse[58:] == 7).all())
    out2 = torch.full_like(wide, 7.0)
    q.qurl_kv_attn_chunk(*args, out2[:M, :6 * 64], ws)  # without lse
    assert torch.equal(out2, wide)


def test_bad_pages_lengths_and_rows_are_reported_and_left_out():
    def reported():
        with pytest.raises(q.QurlError) as e:
            q.qurl_check_device_status()
        assert e.value.status == 1

    a = make([(60, 40), (0, 64), (40, 10)], 10, 2, 128, 16, seed=7)
    a["table"][0, 2] = -1
    a["table"][1, 1] = a["k"].shape[0] // 16  # one page past the cache
    o, l = run(a)
    reported()
    bad = {0: 2, 1: 1}
    check(a, (o, l), keep=lambda b, j: (j // 16) != bad.get(b, -1))
    a = make([(60, 40), (0, 64)], 10, 2, 128, 16, seed=7)
    a["lens"][1] = 10 ** 6  # longer than its table: cut to 112
    o, l = run(a)
    reported()
    check(a, (o, l))
    a = make([(40, 4)], 2, 1, 64, 16, seed=7)
    a["table"].fill_(-1)
    o, l = run(a)
    reported()
    assert bool((o == 0).all()) and bool((l == float("-inf")).all())
    # rows past M, and in decreasing order
    a = make([(60, 40), (0, 64), (5, 20)], 4, 2, 64, 16, seed=8)
    cu = a["cu"].clone()
    for change in ((1, 300), (2, 10), (3, 1000), (1, -5)):
        a["cu"].copy_(cu)
        a["cu"][change[0]] = change[1]
        run(a)
        reported()


def test_more_new_tokens_than_the_length():
    """Rows that stand before the first token see nothing: zeros and -inf."""
    a = make([(0, 40), (10, 30), (0, 3)], 6, 2, 64, 16, seed=9)
    a["lens"].copy_(torch.tensor([15, 0, -4]))
    o, l = run(a)
    check(a, (o, l))
    assert bool((o[:25] == 0).all()) and bool((l[:25] == float("-inf")).all()) and bool((o[40:] == 0).all())
    a["lens"].copy_(torch.tensor([39, 29, 3]))
    check(a)
    a = make([(0, 600)], 2, 1, 64, 16, seed=9)
    a["lens"].fill_(70)
    check(a)


def test_workspace_reuse_repeats_streams_and_graphs():
    """One workspace over calls of different shapes and head layouts; identical bits on repeat, on another stream, in a
    graph whose lengths change."""
    big = make([(3000, 20), (0, 10), (5, 0), (777, 100)], 40, 8, 128, 16, seed=1)
    small = make([(0, 1), (100, 29)], 10, 2, 64, 16, seed=2)
    other = make([(9000, 2)], 4, 1, 256, 64, seed=3)
    ws = torch.zeros(max(q.qurl_kv_attn_chunk_workspace_size(40, 8, 128), q.qurl_kv_attn_chunk_workspace_size(4, 1, 256)),
                     dtype=torch.uint8, device="cuda")
    first = run(big, ws=ws)
    check(big, first)
    check(small, run(small, ws=ws))
    check(other, run(other, ws=ws))
    again = run(big, ws=ws)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = run(big, ws=ws, stream=s)
    s.synchronize()
    assert torch.equal(first[0], got[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = run(big, ws=ws)
    for lens, cu in (([3020, 10, 5, 877], [0, 20, 30, 30, 130]), ([64, 10, 3, 877], [0, 1, 5, 8, 130]), ([1, 0, 0, 0], [0, 1, 1, 1, 1])):
        big["lens"].copy_(torch.tensor(lens))
        big["cu"].copy_(torch.tensor(cu))
        g.replay()
        check(big, captured)


def test_small_workspace_is_refused():
    a = make([(0, 5)], 2, 1, 64, 16)
    need = q.qurl_kv_attn_chunk_workspace_size(2, 1, 64)
    with pytest.raises(q.QurlError, match="WORKSPACE"):
        run(a, ws=torch.zeros(need - 1, dtype=torch.uint8, device="cuda"))


def test_offsets_past_32_bits():
    """Pages at both ends of caches of more than 2^32 bytes."""
    block, kvh, hd = 16, 8, 256
    pages = (2 ** 32 // (kvh * hd * block)) + 40
    kc, ks, vc, vs = q.kv_cache(pages * block, kvh, hd)
    small = make([(280, 20), (0, 77)], 16, kvh, hd, block, seed=61, pages=60)
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


def test_behind_a_timeout_of_another_kernel():
    """A GEMM's wait has run out and is not looked at yet: the attention behind it may give up, but what it stores
    is right; with the status read and the workspace zeroed it runs as ever."""
    a = make([(3000, 9), (0, 10), (0, 0), (700, 77)], 10, 2, 128, 16, seed=51)
    ws = q.kv_attn_chunk_workspace(10, 2, 128)
    want = run(a, ws=ws)
    X, W = torch.randn((16, 256), device="cuda").to(torch.bfloat16), torch.randn((512, 256), device="cuda")
    Wq, sw, _, _ = q.prepare_weights(W, q.FP8_E4M3, keep_scaled=False)
    Xq, sx = q.quant_act(X, q.FP8_E4M3)
    gws = q.workspace(16, 512, 256, q.FP8_E4M3)
    out, lse = torch.full_like(want[0], 7.0), torch.full_like(want[1], 7.0)
    q.qurl_check_device_status()
    q.qurl_debug_inject_timeout()
    q.linear(Xq, sx, Wq, sw, q.FP8_E4M3, gws)
    q.qurl_kv_attn_chunk(a["q"], 10, a["k"], a["ks"], a["v"], a["vs"], a["table"], 16, a["cu"], a["lens"], a["scale"], out, ws,
                         lse=lse)
    with pytest.raises(q.QurlError) as e:
        q.qurl_check_device_status()
    assert e.value.status == 6  # QURL_ERR_TIMEOUT
    per_head, M = out.view(-1, 10, 128), out.shape[0]
    left = (per_head == 7.0).all(-1)
    assert bool((left | (per_head == want[0].view(M, 10, 128)).all(-1)).all())
    assert bool(((lse == 7.0) | (lse == want[1])).all())
    ws.zero_()
    got = run(a, ws=ws)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 3, 2 ** 30, 5, 1])
def test_rows_before_the_first_token_and_windows(window):
    """More new tokens than the length says, whatever the window: zeros and -inf there, all else as ever."""
    a = make([(0, 40), (300, 30), (0, 3), (2000, 270), (10, 9)], 6, 2, 64, 16, seed=9)
    a["lens"][0], a["lens"][2], a["lens"][4] = 15, -4, 5
    a["window"] = window
    out = torch.full_like(a["q"], 7.0)
    lse = torch.full((a["q"].shape[0], 6), 7.0, device="cuda")
    q.qurl_kv_attn_chunk(a["q"], 6, a["k"], a["ks"], a["v"], a["vs"], a["table"], 16, a["cu"], a["lens"], a["scale"], out,
                         q.kv_attn_chunk_workspace(6, 2, 64), window, lse)
    check(a, (out, lse))
    assert bool((out[:25] == 0).all()) and bool((lse[:25] == float("-inf")).all()) and bool((out[70:73] == 0).all())


@pytest.mark.parametrize("first,second", [(290, 200), (290, 270), (290, 3), (100, 290), (19990, 40), (19990, 12000), (60, 19990)])
@pytest.mark.parametrize("gap", [0, 30, 60, 100])
def test_value_scales_far_apart_between_blocks(first, second, gap):
    """A token of the largest score and a value scale of 2^-100, and one whose score is `gap` less (in log2 units) and whose
    value scale is 2^100, in different blocks, tiles and parts of a unit: the outputs are the second one's values, the sum of
    exponentials is the first one's."""
    n = 20000 if max(first, second) > 300 else 300
    a = make([(n - 1, 1)], 1, 1, 64, 16, seed=81)
    at = lambda j: int(a["table"][0, j // 16]) * 16 + j % 16  # noqa: E731
    a["q"].fill_(1.0)
    a["k"].view(torch.uint8).zero_()
    for j, x, e in ((first, 110.0, -100), (second, 110.0 - gap, 100)):
        a["k"][at(j)] = torch.full((1, 64), 448.0, device="cuda").to(torch.float8_e4m3fn)
        a["ks"][at(j)] = x / 1.4426950408889634 / (448.0 * 64 * a["scale"])
        a["vs"][at(j)] = 2.0 ** e
    check(a)


@pytest.mark.parametrize("block", [16, 24, 128])
@pytest.mark.parametrize("window", [1, 100, 128, 129, 1000])
def test_pages_behind_the_window(window, block):
    """Pages that no row's window reaches have been given back: neither they nor their tokens are read."""
    a = make([(1500, 200), (900, 1), (3000, 7), (300, 40), (0, 250)], 10, 2, 128, block, seed=window)
    a["window"] = window
    want = run(a)
    check(a, want)
    for b in range(5):
        cached = int(a["lens"][b]) - int(a["cu"][b + 1] - a["cu"][b])
        a["table"][b, :max(0, cached + 1 - window) // block] = -1 if b % 2 else 2 ** 30
    got = run(a)
    q.qurl_check_device_status()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_rows_of_nearly_as_many_columns_as_an_int_counts():
    """A row that sees nothing, of 2^27 - 1 heads of 16: zeros up to its last column, and nothing behind it."""
    heads = 2 ** 27 - 1
    a = make([(0, 1)], 1, 1, 16, 16)
    x = torch.zeros(heads * 16, dtype=torch.bfloat16, device="cuda")
    out = torch.full((heads * 16 + 4096,), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((1, heads), 7.0, device="cuda")
    a["lens"].zero_()
    q.qurl_kv_attn_chunk(x.view(1, -1), heads, a["k"], a["ks"], a["v"], a["vs"], a["table"], 16, a["cu"], a["lens"], 0.25,
                         out[:heads * 16].view(1, -1), q.kv_attn_chunk_workspace(heads, 1, 16), lse=lse)
    assert bool((out[:heads * 16] == 0).all()) and bool((out[heads * 16:] == 7).all()) and bool((lse == float("-inf")).all())


def test_weights_are_rounded_once_where_a_reference_moves():
    """Pairs of tokens with the same score and opposite values, w_a v_a = - w_b v_b, in the first half of a tile, and a token that
    moves the reference in the second half: what is left of a pair is the rounding of its weights.  One rounding
    to fp16 leaves 2^-11 of each (2^-10.9 with the fp32 roundings of the product and the sum), which bf16 rounds by 2^-9; the
    magnitude itself, from scores that are off by 2^-12 at most, is within 2^-9."""
    a = make([(100, 28)], 16, 1, 128, 16, seed=91)
    g = _gen(92)
    slot = a["table"][0].long().repeat_interleave(16)[:128] * 16 + torch.arange(128, device="cuda") % 16
    k = torch.zeros((128, 128), device="cuda")
    k[:64, 1:] = torch.randn((32, 127), device="cuda", generator=g).repeat_interleave(2, 0)
    k[64, 0] = 448.0
    v = torch.zeros((128, 128), device="cuda")
    pair = torch.arange(32, device="cuda")
    v[2 * pair, pair], v[2 * pair + 1, pair] = 416.0, -448.0
    for n, x in (("k", k), ("v", v)):
        a[n].view(torch.uint8)[slot, 0] = x.to(torch.float8_e4m3fn).view(torch.uint8)
    a["ks"][slot] = 0.555
    a["ks"][slot[64]] = 12.5 / 1.4426950408889634 / (448.0 * a["scale"])
    a["vs"][slot] = 448.0 * 2.0 ** -15
    a["vs"][slot[2 * pair + 1]] = 416.0 * 2.0 ** -15
    a["q"].view(28, 16, 128)[..., 0] = 1.0
    o = run(a)[0].double().view(28, 16, 128)
    keys = k.to(torch.float8_e4m3fn).double() * a["ks"][slot].double()
    s = a["q"].double().view(28, 16, 128) @ keys.T * a["scale"]
    s = s.masked_fill(torch.arange(128, device="cuda") > torch.arange(100, 128, device="cuda")[:, None, None], float("-inf"))
    size = torch.softmax(s, -1)[..., :64:2] * 2 * 416 * 448 * 2.0 ** -15
    assert bool((o[..., 32:] == 0).all())
    worst = float((o[..., :32].abs() / size).max())
    assert worst <= 2.0 ** -10.9 * (1 + 2.0 ** -8), worst * 2 ** 10.9


@pytest.mark.parametrize("window", [0, 150])
@pytest.mark.parametrize("q_heads,kv_heads,hd", [(10, 2, 128), (2, 2, 64), (4, 2, 256)])
def test_values_that_are_no_numbers(q_heads, kv_heads, hd, window):
    """A value code that is no number makes NaN of its head's outputs in the rows that see the token, and of nothing else."""
    a = make([(0, 300), (200, 60), (20000, 3), (40, 1), (700, 90)], q_heads, kv_heads, hd, 16, seed=95)
    a["window"] = window
    a["q"].mul_(0.25)
    nans = {0: (5, 128, 131, 290), 1: (100, 215), 2: (19950, 20001) if window else (64, 11000, 20001), 3: (), 4: (650, 789)}
    slots = {b: [int(a["table"][b, j // 16]) * 16 + j % 16 for j in js] for b, js in nans.items()}
    every = [s for ss in slots.values() for s in ss]
    a["v"].view(torch.uint8)[every, 1, 7] = 0
    want = run(a)
    check(a, want)
    a["v"].view(torch.uint8)[every[::2], 1, 7] = 0x7F
    a["v"].view(torch.uint8)[every[1::2], 1, 7] = 0xFF
    o, l = run(a)
    assert torch.equal(l, want[1])
    sees = torch.zeros(o.shape[0], dtype=torch.bool, device="cuda")
    for b, js in nans.items():
        r0, r1 = int(a["cu"][b]), int(a["cu"][b + 1])
        pos = int(a["lens"][b]) - (r1 - r0) + torch.arange(r1 - r0, device="cuda")
        for j in js:
            sees[r0:r1] |= (j <= pos) & ((pos - window < j) if window else True)
    o, w = o.view(-1, kv_heads, q_heads // kv_heads * hd), want[0].view(-1, kv_heads, q_heads // kv_heads * hd)
    assert bool(sees.any()) and not bool(sees.all())
    assert bool(torch.isnan(o[sees, 1]).all())
    assert torch.equal(o[~sees, 1], w[~sees, 1]) and torch.equal(o[:, 0], w[:, 0])


def test_waits_that_run_out():
    """The keys of each CTA's first tile are never handed over: the call ends and says so, nothing of a sequence that sees a
    token is stored wrong, and with the workspace zeroed the next call gives what the one before gave, to the bit."""
    for spans, q_heads, kv_heads, hd in (([(3000, 9), (0, 300), (0, 0), (700, 77)], 10, 2, 128), ([(500, 70), (0, 5)], 2, 1, 256)):
        a = make(spans, q_heads, kv_heads, hd, 16, seed=61)
        ws = q.kv_attn_chunk_workspace(q_heads, kv_heads, hd)
        want = run(a, ws=ws)
        out, lse = torch.full_like(want[0], 7.0), torch.full_like(want[1], 7.0)
        torch.cuda.synchronize()
        q.qurl_debug_inject_timeout()
        q.qurl_kv_attn_chunk(a["q"], q_heads, a["k"], a["ks"], a["v"], a["vs"], a["table"], 16, a["cu"], a["lens"], a["scale"], out,
                             ws, lse=lse)
        with pytest.raises(q.QurlError) as e:
            q.qurl_check_device_status()
        assert e.value.status == 6  # QURL_ERR_TIMEOUT
        assert bool((out == 7.0).all()) and bool((lse == 7.0).all())
        ws.zero_()
        got = run(a, ws=ws)
        q.qurl_check_device_status()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("scale", [float("inf"), float("nan")])
def test_value_scales_that_are_no_numbers(scale):
    """A value scale of infinity or NaN reaches the outputs of the rows that see its token, not their lse, and nothing of the
    other rows."""
    a = make([(0, 300), (200, 60), (9000, 2), (40, 1)], 10, 2, 128, 16, seed=97)
    at = [int(a["table"][b, j // 16]) * 16 + j % 16 for b, j in ((0, 150), (1, 100), (2, 70))]
    a["v"].view(torch.uint8)[at] = 0x38  # 1
    plain = a | dict(vs=a["vs"].clone())
    a["vs"][at, 1] = scale
    plain["vs"][at, 1] = 1.0 / 448
    o, l = run(a)
    ro, rl, to, tl = reference(plain)
    assert bool((l.double() - rl).abs().le(tl).all()), float(((l.double() - rl).abs() / tl).max())
    sees = torch.ones(o.shape[0], dtype=torch.bool, device="cuda")
    sees[:150], sees[-1] = False, False
    o, ro, to = (t.view(-1, 2, 640) for t in (o, ro, to))
    assert not bool(torch.isfinite(o[sees, 1]).any())
    assert bool((o[:, 0].double() - ro[:, 0]).abs().le(to[:, 0]).all())
    assert bool((o[~sees, 1].double() - ro[~sees, 1]).abs().le(to[~sees, 1]).all())


@pytest.mark.parametrize("hd", [64, 128, 256])
def test_queries_that_are_no_numbers(hd):
    """Infinity or NaN in a head of a query makes NaN of its outputs and lse; other heads and rows are as ever, and a row that
    sees nothing stays a row that sees nothing."""
    a = make([(0, 300), (2000, 3), (40, 1), (0, 5)], 10, 2, hd, 16, seed=98)
    a["lens"][3] = 3
    bad = [(0, 3, float("inf")), (140, 9, float("nan")), (299, 0, -float("inf")), (301, 5, float("inf")), (303, 1, float("nan"))]
    plain = a | dict(q=a["q"].clone())
    for row, head, v in bad + [(304, 2, float("inf"))]:
        a["q"].view(-1, 10, hd)[row, head, 17 % hd] = v
        plain["q"].view(-1, 10, hd)[row, head] = 0.0
    o, l = run(a)
    ro, rl, to, tl = reference(plain)
    hit = torch.zeros(l.shape, dtype=torch.bool, device="cuda")
    for row, head, _ in bad:
        hit[row, head] = True
    o, ro, to = (t.view(-1, 10, hd) for t in (o, ro, to))
    assert bool(torch.isnan(o[hit]).all()) and bool(torch.isnan(l[hit]).all())
    assert bool((o.double() - ro).abs().le(to)[~hit].all())
    assert torch.equal(torch.isinf(l)[~hit], torch.isinf(rl)[~hit]) and bool((o[304:306] == 0).all())
    d = torch.where(torch.isinf(rl), 0.0, l.double() - rl).abs()
    assert bool(d.le(tl)[~hit].all())
