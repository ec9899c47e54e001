"""Rotary positions, alone and with the FP8 quantization into the cache, against the
formulas in 64 bits.

Tolerances, from the arithmetic.  The signed fraction of a turn is rounded to 32 bits and
to fp32 (2^-24 of at most pi: 2^-22.3 radians) and sincospi is off by an ulp or two
(2^-23): cosine and sine are within 2^-21.3.  With the factor's rounding and the two of
the sum, a rotated value is within (|a| + |b|) |factor| 2^-21 of the formula's before it is
rounded to the output's type (half a step: 2^-8 of the value in bf16, 2^-24 in fp32).  The
frequency's 2^-52 of the angle's whole turns adds |p f| 2^-52.  A code is the value
over the scale to half a step of e4m3 (2^-4 of the value, 2^-10 where it is subnormal)."""
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


def rotated(x, pos, freq, layout, factor, inverse=False):
    """x [M, heads, hd] in 64 bits -> (rotated, bound of the error before the output's rounding)."""
    rot = 2 * freq.numel()
    a = pos.double()[:, None] * freq
    c, s = torch.cos(a)[:, None], torch.sin(a)[:, None] * (-1 if inverse else 1)
    x = x.double()
    first, second = (slice(0, rot // 2), slice(rot // 2, rot)) if layout == q.ROPE_HALF else (slice(0, rot, 2), slice(1, rot, 2))
    u, v = x[..., first], x[..., second]
    y, e = x.clone(), torch.zeros_like(x)
    y[..., first], y[..., second] = factor * (u * c - v * s), factor * (u * s + v * c)
    # (the reference's own angle: a product and a reduction in 64 bits)
    bound = (u.abs() + v.abs()) * abs(factor) * (2.0 ** -21 + a.abs()[:, None] * 2.0 ** -51)
    e[..., first] = e[..., second] = bound
    return y, e


def check(got, y, e):
    half = torch.finfo(got.dtype).eps / 2
    err = (got.double().view(y.shape) - y).abs()
    tol = e + y.abs() * half * (1 + 2.0 ** -7) + torch.finfo(got.dtype).tiny * torch.finfo(got.dtype).eps
    assert bool(err.le(tol).all()), float((err / tol).max())


def inputs(M, heads, hd, dtype, seed, far=5000):
    g = _gen(seed)
    x = (torch.randn((M, heads * hd), device="cuda", generator=g) * 3).to(dtype)
    pos = torch.randint(0, far, (M,), device="cuda", generator=g, dtype=torch.int32)
    return x, pos


@pytest.mark.parametrize("layout", [q.ROPE_HALF, q.ROPE_INTERLEAVED])
@pytest.mark.parametrize("hd,rot", [(16, 16), (16, 2), (32, 20), (64, 64), (64, 32), (80, 80), (80, 32), (80, 20), (96, 48),
                                    (96, 94), (112, 112), (128, 128), (128, 64), (128, 30), (144, 144), (192, 64), (240, 120),
                                    (256, 256), (256, 64), (256, 254)])
def test_head_dims_and_parts(hd, rot, layout):
    for dtype in (torch.bfloat16, torch.float32):
        x, pos = inputs(9, 5, hd, dtype, hd + rot)
        freq, _ = q.rope_frequencies(rot)
        for inverse in (False, True):
            got = q.rope(x, 5, pos, freq, layout=layout, factor=1.3, inverse=inverse)
            check(got, *rotated(x.view(9, 5, hd), pos, freq, layout, 1.3, inverse))
            rest = got.view(9, 5, hd)[..., rot:]
            assert torch.equal(rest, x.view(9, 5, hd)[..., rot:])


@pytest.mark.parametrize("M,heads", [(1, 1), (1, 36), (2, 3), (151, 7), (152, 56), (153, 56), (1000, 17), (5, 130), (8192, 4)])
def test_tokens_and_heads(M, heads):
    x, pos = inputs(M, heads, 128, torch.bfloat16, M + heads)
    freq, factor = q.rope_frequencies(128, 500000.0, "yarn", 4.0, 8192)
    check(q.rope(x, heads, pos, freq, factor=factor), *rotated(x.view(M, heads, 128), pos, freq, q.ROPE_HALF, factor))


def test_positions_of_every_size():
    freq, _ = q.rope_frequencies(64, 1e6)
    pos = [0, 1, -1, 2, 7, 4095, 65535, 65536, 1000003, 2 ** 24 + 1, 2 ** 30 + 12345, 2 ** 31 - 1, -2 ** 31, -77777]
    x, _ = inputs(len(pos), 3, 64, torch.float32, 1)
    pos = torch.tensor(pos, dtype=torch.int32, device="cuda")
    check(q.rope(x, 3, pos, freq), *rotated(x.view(-1, 3, 64), pos, freq, q.ROPE_HALF, 1.0))
    assert torch.equal(q.rope(x, 3, pos, freq)[0], x[0])  # position 0 turns nothing
    # frequencies of more than a turn a position, of none, tiny and negative ones
    f = torch.tensor([0.0, 7.0, 100.5, -0.3, 1e-12, 1e-30, 2.0 ** -60, 6.283185307179586], dtype=torch.float64, device="cuda")
    pos = torch.tensor([0, 1, 5, 1000, 123457, -9], dtype=torch.int32, device="cuda")
    x, _ = inputs(6, 2, 16, torch.float32, 2)
    for layout in (q.ROPE_HALF, q.ROPE_INTERLEAVED):
        check(q.rope(x, 2, pos, f, layout=layout), *rotated(x.view(-1, 2, 16), pos, f, layout, 1.0))


@pytest.mark.parametrize("layout", [q.ROPE_HALF, q.ROPE_INTERLEAVED])
@pytest.mark.parametrize("rot", [64, 36])
def test_inverse_is_the_gradient(layout, rot):
    """Against the formula's gradient and against differences (the rotation is linear: a step of any size gives them)."""
    M, heads, hd = 7, 3, 64
    x, pos = inputs(M, heads, hd, torch.float32, 3)
    dy, _ = inputs(M, heads, hd, torch.float32, 4)
    freq, _ = q.rope_frequencies(rot)
    leaf = x.double().view(M, heads, hd).requires_grad_(True)
    y, _ = rotated(leaf, pos, freq, layout, 0.7)
    y.backward(dy.double().view(M, heads, hd))
    dx = q.rope(dy, heads, pos, freq, layout=layout, factor=0.7, inverse=True)
    _, e = rotated(dy.view(M, heads, hd), pos, freq, layout, 0.7)
    check(dx, leaf.grad, e)
    base = q.rope(x, heads, pos, freq, layout=layout, factor=0.7).double()
    for i in range(0, heads * hd, 17):
        step = torch.zeros_like(x)
        step[:, i] = 1.0
        diff = (q.rope(x + step, heads, pos, freq, layout=layout, factor=0.7).double() - base) * dy.double()
        # two results of magnitude up to 15, each within 2^-19 of it, times dy, over two values that change
        assert bool((diff.sum(1) - dx[:, i].double()).abs().le(64 * 2.0 ** -18).all())
    back = q.rope(q.rope(x, heads, pos, freq, layout=layout), heads, pos, freq, layout=layout, inverse=True)
    assert bool((back - x).abs().le(2.0 ** -18 * (x.view(M, heads, hd).norm(dim=-1).amax() + 1)).all())


@pytest.mark.parametrize("rot", [128, 60])
def test_in_place_and_neighbours(rot):
    """Queries and keys as one run of heads inside the fused rows, in place: the values beside them stay."""
    M, hd, heads = 77, 128, 6
    x, pos = inputs(M, heads + 3, hd, torch.bfloat16, 5)
    freq, _ = q.rope_frequencies(rot)
    want = q.rope(x[:, :heads * hd], heads, pos, freq)
    y = x.clone()
    assert q.rope(y, heads, pos, freq, head_dim=hd, inplace=True) is y
    assert torch.equal(y[:, :heads * hd], want) and torch.equal(y[:, heads * hd:], x[:, heads * hd:])
    wide = torch.full((M + 2, (heads + 1) * hd), 7.0, dtype=torch.bfloat16, device="cuda")
    q.qurl_rope(x, heads, hd, pos, freq, wide[1:-1, :heads * hd])
    assert torch.equal(wide[1:-1, :heads * hd], want)
    assert bool((wide[0] == 7).all()) and bool((wide[-1] == 7).all()) and bool((wide[:, heads * hd:] == 7).all())
    with pytest.raises(ValueError):
        q.qurl_rope(wide[:-1], heads, hd, pos[:1].repeat(M + 1), freq, wide[1:])


def test_infinities_stay_in_their_pair():
    x, pos = inputs(3, 4, 64, torch.bfloat16, 6)
    x[1, 70] = float("inf")
    x[2, 64 + 50] = float("nan")
    freq, _ = q.rope_frequencies(40)
    for layout in (q.ROPE_HALF, q.ROPE_INTERLEAVED):
        got = q.rope(x, 4, pos, freq, layout=layout)
        bad = ~torch.isfinite(got)
        pair = [70, 90] if layout == q.ROPE_HALF else [70, 71]
        assert bad[1].nonzero()[:, 0].tolist() == pair and bad[2].nonzero()[:, 0].tolist() == [114] and not bool(bad[0].any())


def cache_check(x, heads, kvh, hd, pos, freq, slot, layout, factor, got_q, caches, before):
    M = x.shape[0]
    v = x[:, :(heads + 2 * kvh) * hd].reshape(M, -1, hd)
    y, e = rotated(v[:, :heads + kvh], pos, freq, layout, factor)
    check(got_q, y[:, :heads].reshape(M, -1), e[:, :heads].reshape(M, -1))
    rows = ((slot >= 0) & (slot < len(before[0]))).nonzero()[:, 0]
    at = slot[rows]
    for vec, err, code, scale in ((y[:, heads:], e[:, heads:], caches[0], caches[1]),
                                  (v[:, heads + kvh:].double(), torch.zeros_like(y[:, heads:]), caches[2], caches[3])):
        vec, err = vec[rows], err[rows]
        top, sc = vec.abs().amax(-1), scale[at].double()
        want = torch.where(top == 0, 1.0, top / 448)
        assert bool((sc - want).abs().le(want * 2.0 ** -23 + err.amax(-1) / 448).all())
        c = code.view(torch.uint8)[at].view(torch.float8_e4m3fn).double()
        # half a step of the code, the value's error, and the scale's (of a value of up to 448 steps)
        tol = sc[..., None] * (c.abs() * 2.0 ** -4 * 1.07 + 2.0 ** -10) + err + vec.abs() * 2.0 ** -22 + err.amax(-1, keepdim=True)
        d = (c * sc[..., None] - vec).abs()
        assert bool(d.le(tol).all()), float((d / tol).max())
    left = torch.ones(len(before[0]), dtype=torch.bool, device="cuda")
    left[at] = False
    for a, b in zip(caches, before):
        assert torch.equal(a[left].view(torch.uint8), b[left].view(torch.uint8))


def new_cache(slots, kvh, hd):
    caches = q.kv_cache(slots, kvh, hd)
    for c in caches:
        c.view(torch.uint8).fill_(0x2A)
    return caches


@pytest.mark.parametrize("layout", [q.ROPE_HALF, q.ROPE_INTERLEAVED])
@pytest.mark.parametrize("M,heads,kvh,hd,rot", [(1, 28, 4, 128, 128), (1, 1, 1, 16, 16), (64, 40, 8, 128, 128), (153, 9, 3, 80, 32),
                                                (200, 9, 3, 80, 20), (1000, 10, 2, 64, 64), (333, 8, 1, 256, 128), (50, 6, 6, 192, 100),
                                                (700, 5, 5, 96, 96), (3, 130, 2, 48, 48)])
def test_cache(M, heads, kvh, hd, rot, layout):
    g = _gen(M)
    x, pos = inputs(M, heads + 2 * kvh, hd, torch.bfloat16, M + hd, far=100000)
    freq, factor = q.rope_frequencies(rot, 10000.0, "yarn", 16.0, 4096)
    slots = 2 * M + 3
    slot = torch.randperm(slots, device="cuda", generator=g)[:M]
    if M > 2:
        slot[::5] = -1
    caches = new_cache(slots, kvh, hd)
    before = [c.clone() for c in caches]
    got = q.rope_kv_cache_quant(x, heads, pos, freq, slot, *caches, layout=layout, factor=factor)
    cache_check(x, heads, kvh, hd, pos, freq, slot, layout, factor, got, caches, before)


def test_cache_without_turning_is_the_quantizer():
    """At position 0 with a factor of 1 codes and scales are those of qurl_kv_cache_quant, bit for bit; the values
    always are."""
    M, heads, kvh, hd = 300, 4, 2, 128
    x, pos = inputs(M, heads + 2 * kvh, hd, torch.bfloat16, 11)
    x[5] = 0.0
    x[6, heads * hd:] *= 2.0 ** -100
    slot = torch.arange(M, device="cuda")
    freq, _ = q.rope_frequencies(hd)
    a, b = new_cache(M, kvh, hd), new_cache(M, kvh, hd)
    q.qurl_kv_cache_quant(x, heads * hd, kvh, hd, slot, *a)
    got = q.rope_kv_cache_quant(x, heads, torch.zeros_like(pos), freq, slot, *b)
    assert torch.equal(got, x[:, :heads * hd])
    for u, v in zip(a, b):
        assert torch.equal(u.view(torch.uint8), v.view(torch.uint8))
    q.rope_kv_cache_quant(x, heads, pos, freq, slot, *b)
    for u, v in zip(a[2:], b[2:]):
        assert torch.equal(u.view(torch.uint8), v.view(torch.uint8))


def test_cache_in_place_wide_rows_and_bad_slots():
    M, heads, kvh, hd = 40, 5, 1, 80
    x, pos = inputs(M, heads + 2 * kvh + 1, hd, torch.bfloat16, 12)
    freq, _ = q.rope_frequencies(hd)
    slot = torch.arange(M, device="cuda") * 2
    slot[7], slot[9] = 90, -2 ** 40
    caches = new_cache(90, kvh, hd)
    before = [c.clone() for c in caches]
    y = x.clone()
    assert q.rope_kv_cache_quant(y, heads, pos, freq, slot, *caches, inplace=True) is y
    with pytest.raises(q.QurlError) as err:
        q.qurl_check_device_status()
    assert err.value.status == 1
    cache_check(x, heads, kvh, hd, pos, freq, slot, q.ROPE_HALF, 1.0, y[:, :heads * hd], caches, before)
    assert torch.equal(y[:, heads * hd:], x[:, heads * hd:])


def test_cache_heads_of_every_size():
    """Heads of zeros, of the smallest magnitudes, of one value, and of the largest."""
    M, heads, kvh, hd = 8, 2, 2, 64
    x, pos = inputs(M, heads + 2 * kvh, hd, torch.bfloat16, 13)
    x[0] = 0.0
    x[1] = 2.0 ** -133
    x[2] *= 2.0 ** -120
    x[3] = 0.0
    x[3, heads * hd + 5] = 3.0
    x[4] *= 2.0 ** 120
    freq, _ = q.rope_frequencies(hd)
    slot = torch.arange(M, device="cuda")
    caches = new_cache(M, kvh, hd)
    before = [c.clone() for c in caches]
    got = q.rope_kv_cache_quant(x, heads, pos, freq, slot, *caches)
    for c in (caches[0], caches[2]):
        assert not bool((c.view(torch.uint8) & 0x7F).eq(0x7F).any())
    rows = torch.tensor([0, 2, 3, 4, 5, 6, 7], device="cuda")
    keep = torch.full_like(slot, -1)
    keep[rows] = slot[rows]
    cache_check(x[rows], heads, kvh, hd, pos[rows], freq, slot[rows], q.ROPE_HALF, 1.0, got[rows], caches,
                [torch.where((keep < 0).view(-1, *[1] * (a.dim() - 1)), a.float(), b.float()).to(a.dtype) for a, b in zip(caches, before)])


def test_offsets_past_32_bits():
    """Slots at the end of caches of more than 2^32 bytes."""
    M, heads, kvh, hd = 6, 8, 8, 256
    slots = 2 ** 32 // (kvh * hd) + 10
    x, pos = inputs(M, heads + 2 * kvh, hd, torch.bfloat16, 14)
    freq, _ = q.rope_frequencies(hd)
    big, small = q.kv_cache(slots, kvh, hd), q.kv_cache(M, kvh, hd)
    at = torch.tensor([slots - 1, 0, slots - 3, 2 ** 31 // (kvh * hd), slots - 2, 5], device="cuda")
    a = q.rope_kv_cache_quant(x, heads, pos, freq, at, *big)
    b = q.rope_kv_cache_quant(x, heads, pos, freq, torch.arange(M, device="cuda"), *small)
    assert torch.equal(a, b)
    for u, v in zip(big, small):
        assert torch.equal(u[at].view(torch.uint8), v.view(torch.uint8))


def test_streams_graphs_and_empty_calls():
    M, heads, kvh, hd = 33, 4, 2, 128
    x, pos = inputs(M, heads + 2 * kvh, hd, torch.bfloat16, 15)
    freq, _ = q.rope_frequencies(hd)
    slot = torch.arange(M, device="cuda")
    caches = new_cache(M, kvh, hd)
    want = q.rope_kv_cache_quant(x, heads, pos, freq, slot, *caches)
    held = [c.clone() for c in caches]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = q.rope(x, heads, pos, freq, head_dim=hd, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = q.rope_kv_cache_quant(x, heads, pos, freq, slot, *caches)
    for c in caches:
        c.view(torch.uint8).zero_()
    pos.add_(0)
    g.replay()
    assert torch.equal(out, want)
    for a, b in zip(caches, held):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    pos.add_(1000)  # the positions are read at replay
    g.replay()
    check(out, *[t.reshape(M, -1) for t in rotated(x[:, :heads * hd].reshape(M, heads, hd), pos, freq, q.ROPE_HALF, 1.0)])
    assert q.rope(x[:0], heads, pos[:0], freq, head_dim=hd).shape == (0, heads * hd)
    assert q.rope_kv_cache_quant(x[:0], heads, pos[:0], freq, slot[:0], *caches).shape == (0, heads * hd)


@pytest.mark.parametrize("layout", [q.ROPE_HALF, q.ROPE_INTERLEAVED])
def test_fp32_angles(layout):
    """Cosines and sines themselves: the angle is taken modulo a turn in fixed point (2^-32 of a turn), what is left of the nearest
    quarter, at most an eighth of a turn, in fp32 (2^-28 of a turn): 2^-25.2 radians, and an ulp (2^-24) of a cosine or a sine
    that is at most 1: 2^-23.48."""
    M, hd = 4001, 64
    freq, _ = q.rope_frequencies(hd, 500.0)
    pos = torch.arange(M, dtype=torch.int32, device="cuda") - 2000
    x = torch.zeros((M, hd), device="cuda")
    first, second = (slice(0, 32), slice(32, 64)) if layout == q.ROPE_HALF else (slice(0, 64, 2), slice(1, 64, 2))
    x[:, first] = 1.0
    got = q.rope(x, 1, pos, freq, layout=layout).double()
    a = pos.double()[:, None] * freq
    # (2^-52 of the angle for the reference's own product, as much for the frequency in turns)
    bound = 2.0 ** -23.48 + a.abs() * 2.0 ** -51
    for part, want in ((first, torch.cos(a)), (second, torch.sin(a))):
        d = (got[:, part] - want).abs()
        assert bool(d.le(bound).all()), float((d / bound).max())
    back = q.rope(x, 1, pos, freq, layout=layout, inverse=True).double()
    assert torch.equal(back[:, first], got[:, first]) and torch.equal(back[:, second], -got[:, second])


def test_cache_of_what_is_no_number():
    """NaN in a head of keys or of values is in its codes, whatever stands beside it: of values as qurl_kv_cache_quant has it, of
    keys in both of a turned pair (at position 0 too: a NaN times a sine of 0 is one)."""
    M, heads, kvh, hd = 6, 2, 2, 64
    x, pos = inputs(M, heads + 2 * kvh, hd, torch.bfloat16, 16)
    v = x.view(M, -1, hd)
    nan = float("nan")
    v[0] = nan                                       # nothing else
    v[1] = 0.0
    v[1, :, 5] = nan                                 # beside zeros
    v[2] = 2.0 ** -133
    v[2, :, 40] = nan                                # beside the smallest values
    v[3, :, 7] = nan                                 # beside values
    slot = torch.arange(M, device="cuda")
    freq, _ = q.rope_frequencies(hd)
    a, b = new_cache(M, kvh, hd), new_cache(M, kvh, hd)
    rows = torch.tensor([0, 1, 3, 4, 5], device="cuda")  # (the quantizer's step of values that small is not compared)
    q.qurl_kv_cache_quant(x[rows], heads * hd, kvh, hd, slot[rows], *a)
    for p in (torch.zeros_like(pos), pos):
        q.rope_kv_cache_quant(x, heads, p, freq, slot, *b)
        keys, values = b[0].view(torch.uint8) & 0x7F, b[2].view(torch.uint8) & 0x7F
        assert torch.equal(values[rows], a[2].view(torch.uint8)[rows] & 0x7F) and torch.equal(b[3][rows], a[3][rows])
        assert bool((keys[0] == 0x7F).all()) and bool((values[0] == 0x7F).all())
        for row, d in ((1, 5), (2, 40), (3, 7)):
            assert (keys[row] == 0x7F).nonzero()[:, 1].view(kvh, -1).tolist() == [sorted((d, (d + 32) % 64))] * kvh
            assert (values[row] == 0x7F).nonzero()[:, 1].view(kvh, -1).tolist() == [[d]] * kvh
        for c in (keys, values):
            assert int((c[1] != 0).sum()) == int((c[1] == 0x7F).sum()) and not bool((c[4:] == 0x7F).any())
