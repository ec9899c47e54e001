"""Host-side refusals of the entry points that place tokens in pages and rotate
queries and keys: every bad argument is turned away before any launch, the binding
turns away tensors of the wrong kind, and the frequencies are those of the formulas."""
import ctypes
import math

import pytest
import torch

import w8a8_precision_gemm_gb300 as q
from w8a8_precision_gemm_gb300 import _build

FAKE = ctypes.c_void_p(0x10000)      # 16-byte aligned, never dereferenced: calls fail validation first
ODD = ctypes.c_void_p(0x10008)       # 8-byte aligned only
ODD4 = ctypes.c_void_p(0x10004)
ODD2 = ctypes.c_void_p(0x10002)
INVALID, UNSUPPORTED, ALIGNMENT = 1, 2, 3


@pytest.fixture(scope="module")
def L():
    _build.build()
    return q.load()


APPEND = dict(cached=FAKE, new=FAKE, B=4, table=FAKE, ldt=8, blocks=8, block=16, free=FAKE, pages=100, n=FAKE, n_out=FAKE,
              M=64, slots=FAKE, pos=FAKE, cu=FAKE, lens=FAKE, stream=None)
RELEASE = dict(lens=FAKE, keep=FAKE, B=4, table=FAKE, ldt=8, blocks=8, block=16, free=FAKE, pages=100, n=FAKE, n_out=FAKE,
               stream=None)
BOTH = [
    (dict(table=None), INVALID), (dict(B=-1), INVALID), (dict(ldt=7), INVALID), (dict(blocks=-1), INVALID),
    (dict(block=0), INVALID), (dict(free=None), INVALID), (dict(pages=-1), INVALID), (dict(n=None), INVALID),
    (dict(n_out=None), INVALID), (dict(B=16385), UNSUPPORTED), (dict(blocks=1 << 20, ldt=1 << 20, block=1025), UNSUPPORTED),
    (dict(B=16384, blocks=1 << 17, ldt=1 << 17), UNSUPPORTED), (dict(table=ODD2), ALIGNMENT), (dict(free=ODD2), ALIGNMENT),
    (dict(n=ODD2), ALIGNMENT), (dict(n_out=ODD2), ALIGNMENT),
]


@pytest.mark.parametrize("change,status", BOTH + [
    (dict(cached=None), INVALID), (dict(new=None), INVALID), (dict(M=-1), INVALID), (dict(slots=None), INVALID),
    (dict(pos=None), INVALID), (dict(cu=None), INVALID), (dict(lens=None), INVALID), (dict(slots=ODD4), ALIGNMENT),
    (dict(cached=ODD2), ALIGNMENT), (dict(new=ODD2), ALIGNMENT), (dict(pos=ODD2), ALIGNMENT), (dict(cu=ODD2), ALIGNMENT),
    (dict(lens=ODD2), ALIGNMENT),
])
def test_append_validation(L, change, status):
    assert L.qurl_kv_append(*(APPEND | change).values()) == status


@pytest.mark.parametrize("change,status", BOTH + [(dict(lens=None), INVALID), (dict(lens=ODD2), ALIGNMENT),
                                                   (dict(keep=ODD2), ALIGNMENT)])
def test_release_validation(L, change, status):
    assert L.qurl_kv_release(*(RELEASE | change).values()) == status


ROPE = dict(x=FAKE, type=0, M=2, ldx=512, heads=4, hd=128, pos=FAKE, freq=FAKE, rot=128, layout=0, factor=1.0, inverse=0,
            out=FAKE, ldo=512, stream=None)
CACHE = dict(x=FAKE, M=2, ldx=1024, heads=4, kv=2, hd=128, pos=FAKE, freq=FAKE, rot=128, layout=0, factor=1.0, out=FAKE,
             ldo=1024, slots=FAKE, num=64, k=FAKE, ks=FAKE, v=FAKE, vs=FAKE, stream=None)
ROTATION = [
    (dict(x=None), INVALID), (dict(M=-1), INVALID), (dict(heads=0), INVALID), (dict(hd=0, rot=0), INVALID),
    (dict(pos=None), INVALID), (dict(freq=None), INVALID), (dict(rot=0), INVALID), (dict(rot=130), INVALID),
    (dict(rot=63), INVALID), (dict(layout=2), INVALID), (dict(layout=-1), INVALID), (dict(factor=float("inf")), INVALID),
    (dict(factor=float("nan")), INVALID), (dict(out=None), INVALID), (dict(ldo=504, out=ODD), INVALID),
    (dict(ldx=504), INVALID), (dict(ldo=1536), INVALID), (dict(hd=72, rot=64), UNSUPPORTED),
    (dict(hd=272, ldx=4096, ldo=4096), UNSUPPORTED), (dict(x=ODD), ALIGNMENT), (dict(out=ODD), ALIGNMENT),
    (dict(ldx=1028, ldo=1028), ALIGNMENT), (dict(pos=ODD2), ALIGNMENT), (dict(freq=ODD4), ALIGNMENT),
]


@pytest.mark.parametrize("change,status", ROTATION + [(dict(type=2), INVALID), (dict(inverse=2), INVALID),
                                                       (dict(type=1, ldx=514, ldo=514), ALIGNMENT)])
def test_rope_validation(L, change, status):
    assert L.qurl_rope(*(ROPE | change).values()) == status
    assert L.qurl_rope(*(ROPE | dict(M=0, x=None)).values()) == 0


@pytest.mark.parametrize("change,status", ROTATION + [
    (dict(kv=0), INVALID), (dict(num=-1), INVALID), (dict(slots=None), INVALID), (dict(k=None), INVALID),
    (dict(ks=None), INVALID), (dict(v=None), INVALID), (dict(vs=None), INVALID), (dict(ldx=1016, ldo=1016), INVALID),
    (dict(slots=ODD4), ALIGNMENT), (dict(k=ODD), ALIGNMENT), (dict(v=ODD), ALIGNMENT), (dict(ks=ODD2), ALIGNMENT),
    (dict(vs=ODD2), ALIGNMENT),
])
def test_rope_cache_validation(L, change, status):
    assert L.qurl_rope_kv_cache_quant(*(CACHE | change).values()) == status
    assert L.qurl_rope_kv_cache_quant(*(CACHE | dict(M=0, x=None)).values()) == 0


def test_binding_takes_device_tensors_only():
    i4 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):
        q.kv_append(i4(2), i4(2), i4(2, 3), 16, i4(6), i4(1), 4)
    with pytest.raises(ValueError):
        q.kv_release(i4(2), i4(2, 3), 16, i4(6), i4(1))
    x, f = torch.zeros(2, 64, dtype=torch.bfloat16), torch.ones(8, dtype=torch.float64)
    with pytest.raises(ValueError):
        q.rope(x, 4, i4(2), f)
    c, s = torch.zeros(4, 1, 16, dtype=torch.uint8), torch.ones(4, 1)
    with pytest.raises(ValueError):
        q.rope_kv_cache_quant(x, 2, i4(2), f, torch.zeros(2, dtype=torch.int64), c, s, c, s)


def test_binding_refuses_what_does_not_fit(monkeypatch):
    """The checks behind the device's, with tensors that stand in for the device's."""
    monkeypatch.setattr(q, "_here", lambda *a: None)
    i4 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    x, f = torch.zeros(4, 64, dtype=torch.bfloat16), torch.ones(8, dtype=torch.float64)
    good = dict(X=x, heads=4, head_dim=16, positions=i4(4), inv_freq=f, out=torch.empty_like(x))
    for change in (dict(heads=5), dict(positions=i4(3)), dict(positions=i4(4).long()), dict(inv_freq=f.float()),
                   dict(inv_freq=torch.ones(9, dtype=torch.float64)), dict(inv_freq=f[:0]), dict(out=x.float()),
                   dict(out=x[:3]), dict(out=x[:, :48]), dict(X=x.half()), dict(X=x.t(), out=x.t())):
        with pytest.raises(ValueError):
            q.qurl_rope(**(good | change))
    wide = torch.zeros(6, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="overlaps"):
        q.qurl_rope(**(good | dict(X=wide[:4], out=wide[1:5])))
    with pytest.raises(ValueError, match="overlaps"):
        q.qurl_rope(**(good | dict(X=wide[:4, :48], heads=3, out=wide[:4, 16:])))
    cache, scale = torch.zeros(8, 2, 16, dtype=torch.uint8), torch.ones(8, 2)
    rows = torch.zeros(4, 8 * 16, dtype=torch.bfloat16)
    good = dict(qkv=rows, q_heads=4, positions=i4(4), inv_freq=f, q_out=torch.empty_like(x), slot_mapping=i4(4).long(),
                k_cache=cache, k_scale=scale, v_cache=cache, v_scale=scale)
    for change in (dict(q_heads=5), dict(slot_mapping=i4(4)), dict(k_scale=scale[:7]), dict(v_cache=cache[:7]),
                   dict(k_cache=cache.float(), v_cache=cache.float()), dict(q_out=x[:3]), dict(qkv=rows.float()),
                   dict(q_out=rows[:, 16:80])):
        with pytest.raises(ValueError):
            q.qurl_rope_kv_cache_quant(**(good | change))
    good = dict(cached_lens=i4(2), new_lens=i4(2), block_table=i4(2, 3), block_size=16, free_pages=i4(6), n_free=i4(1),
                n_free_out=i4(1), slot_mapping=i4(4).long(), positions=i4(4), cu_new=i4(3), seq_lens=i4(2))
    for change in (dict(new_lens=i4(3)), dict(block_table=i4(3, 3)), dict(block_table=i4(2, 3).long()), dict(n_free=i4(2)),
                   dict(free_pages=i4(12)[::2]), dict(slot_mapping=i4(4)), dict(positions=i4(5)), dict(cu_new=i4(2)),
                   dict(seq_lens=i4(1))):
        with pytest.raises(ValueError):
            q.qurl_kv_append(**(good | change))


def test_frequencies():
    f, scale = q.rope_frequencies(8, 10000.0, device="cpu")
    assert f.dtype == torch.float64 and scale == 1.0
    assert torch.allclose(f, torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64), rtol=1e-15)
    g, _ = q.rope_frequencies(8, 10000.0, "linear", 4.0, device="cpu")
    assert torch.equal(g, f / 4)
    g, _ = q.rope_frequencies(8, 10000.0, "base", 4.0, device="cpu")
    assert g[0] == 1.0 and abs(float(g[3] / f[3]) - 0.25) < 1e-14
    n = 4096
    g, scale = q.rope_frequencies(64, 10000.0, "ramp", 8.0, n, low_turns=1.0, high_turns=4.0, device="cpu")
    f, _ = q.rope_frequencies(64, 10000.0, device="cpu")
    for i in range(32):
        turns = n * float(f[i]) / (2 * math.pi)
        keep = min(max((turns - 1) / 3, 0), 1)
        assert abs(float(g[i]) - float(f[i]) * (keep + (1 - keep) / 8)) <= 1e-15 * float(f[i])
    assert scale == 1.0
    g, scale = q.rope_frequencies(64, 10000.0, "yarn", 8.0, n, device="cpu")
    assert scale == 1 + 0.1 * math.log(8.0)
    turns = n * f / (2 * math.pi)
    assert torch.equal(g[turns > 32], f[turns > 32]) and torch.equal(g[turns < 0.5], f[turns < 0.5] / 8)
    assert bool((g <= f).all()) and bool((g >= f / 8).all()) and bool((g[1:] < g[:-1]).all())
    for bad in (dict(rot_dim=7), dict(rot_dim=0), dict(rot_dim=8, scaling="cubic"), dict(rot_dim=8, base=0.0),
                dict(rot_dim=8, scaling="ramp"), dict(rot_dim=8, scaling="yarn", original_len=10, low_turns=3.0, high_turns=2.0)):
        with pytest.raises(ValueError):
            q.rope_frequencies(**bad, device="cpu")


def test_helpers_refuse_what_they_cannot_divide_by(monkeypatch):
    monkeypatch.setattr(q, "_here", lambda *a: None)
    x, i4 = torch.zeros(4, 64), torch.zeros(4, dtype=torch.int32)
    f = torch.ones(4, dtype=torch.float64)
    for heads in (0, -1):
        with pytest.raises(ValueError, match="heads"):
            q.rope(x, heads, i4, f)
    with pytest.raises(ValueError, match="base"):
        q.rope_frequencies(64, 1.0, "yarn", 4.0, 4096, device="cpu")
