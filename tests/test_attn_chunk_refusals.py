"""Host-side refusals of qurl_kv_attn_chunk: every bad argument is turned away before any
launch, and the binding turns away tensors of the wrong kind."""
import ctypes

import pytest
import torch

import w8a8_precision_gemm_gb300 as q
from w8a8_precision_gemm_gb300 import _build

FAKE = ctypes.c_void_p(0x10000)      # 16-byte aligned, never dereferenced: calls fail validation first
ODD = ctypes.c_void_p(0x10008)       # 8-byte aligned only
ODD2 = ctypes.c_void_p(0x10002)
INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = 1, 2, 3, 4


@pytest.fixture(scope="module")
def L():
    _build.build()
    return q.load()


ATTN = dict(q=FAKE, ldq=1024, M=9, q_heads=8, kv_heads=2, hd=64, k=FAKE, ks=FAKE, v=FAKE, vs=FAKE, slots=64, table=FAKE,
            ldt=4, blocks=4, block=16, cu=FAKE, lens=FAKE, B=2, window=0, scale=0.1, out=FAKE, ldo=512, lse=FAKE, ws=FAKE,
            bytes=1 << 30, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(ks=None), INVALID), (dict(v=None), INVALID),
    (dict(vs=None), INVALID), (dict(table=None), INVALID), (dict(lens=None), INVALID), (dict(cu=None), INVALID),
    (dict(out=None), INVALID), (dict(ws=None), INVALID), (dict(M=-1), INVALID), (dict(B=-1), INVALID),
    (dict(q_heads=0), INVALID), (dict(kv_heads=0), INVALID), (dict(kv_heads=3), INVALID), (dict(hd=0), INVALID),
    (dict(slots=-1), INVALID), (dict(blocks=-1), INVALID), (dict(block=0), INVALID), (dict(ldt=3), INVALID),
    (dict(window=-1), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(ldq=504), INVALID), (dict(ldo=504), INVALID), (dict(hd=72), UNSUPPORTED),
    (dict(hd=272, ldq=4096, ldo=4096), UNSUPPORTED), (dict(blocks=1 << 20, ldt=1 << 20, block=(1 << 10) + 1), UNSUPPORTED),
    (dict(M=1 << 28), UNSUPPORTED), (dict(B=16385), UNSUPPORTED), (dict(q=ODD), ALIGNMENT), (dict(k=ODD), ALIGNMENT),
    (dict(v=ODD), ALIGNMENT), (dict(out=ODD), ALIGNMENT), (dict(ws=ODD), ALIGNMENT), (dict(ldq=1028), ALIGNMENT),
    (dict(ldo=1028), ALIGNMENT), (dict(ks=ODD2), ALIGNMENT), (dict(vs=ODD2), ALIGNMENT), (dict(table=ODD2), ALIGNMENT),
    (dict(cu=ODD2), ALIGNMENT), (dict(lens=ODD2), ALIGNMENT), (dict(lse=ODD2), ALIGNMENT),
])
def test_validation(L, change, status):
    assert L.qurl_kv_attn_chunk(*(ATTN | change).values()) == status


def test_empty_calls_and_workspace_size(L):
    nothing = dict(q=None, out=None, lens=None, cu=None, ws=None)
    assert L.qurl_kv_attn_chunk(*(ATTN | dict(B=0) | nothing).values()) == 0
    assert L.qurl_kv_attn_chunk(*(ATTN | dict(M=0) | nothing).values()) == 0
    size = L.qurl_kv_attn_chunk_workspace_size
    assert size(0, 2, 64) == 0 and size(8, 0, 64) == 0 and size(8, 3, 64) == 0 and size(8, 2, 0) == 0 and size(8, 2, 272) == 0
    assert 0 < size(8, 2, 64) <= size(40, 8, 128) and size(40, 8, 128) % 16 == 0


def test_binding_refuses_what_does_not_fit(monkeypatch):
    h = torch.zeros(4, 64, dtype=torch.bfloat16)
    c, s = torch.zeros(8, 1, 16, dtype=torch.uint8), torch.ones(8, 1)
    i4 = lambda *n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    ws = torch.zeros(16, dtype=torch.uint8)
    good = dict(q=h, q_heads=4, k_cache=c, k_scale=s, v_cache=c, v_scale=s, block_table=i4(2, 2), block_size=2, cu_new=i4(3),
                seq_lens=i4(2), scale=1.0, out=torch.empty_like(h), workspace=ws)
    with pytest.raises(ValueError, match="device"):
        q.qurl_kv_attn_chunk(**good)
    monkeypatch.setattr(q, "_here", lambda *a: None)
    for change in (dict(q=h.float()), dict(out=h.float()), dict(out=h[:3]), dict(q_heads=5), dict(v_cache=c[:7]),
                   dict(k_cache=c.float(), v_cache=c.float()), dict(k_scale=s[:7]), dict(block_table=i4(2, 2).long()),
                   dict(cu_new=i4(2)), dict(seq_lens=i4(3)), dict(seq_lens=i4(2).long()), dict(lse=torch.zeros(4, 3)),
                   dict(q=torch.zeros(64, 4, dtype=torch.bfloat16).t()), dict(workspace=torch.zeros(8, 4, dtype=torch.uint8).t())):
        with pytest.raises(ValueError):
            q.qurl_kv_attn_chunk(**(good | change))


def test_binding_refuses_outputs_over_queries(monkeypatch):
    """Rows of q are still read where out is already written."""
    monkeypatch.setattr(q, "_here", lambda *a: None)
    h = torch.zeros(6, 128, dtype=torch.bfloat16)
    c, s = torch.zeros(8, 1, 16, dtype=torch.uint8), torch.ones(8, 1)
    i4 = lambda *n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    call = lambda x, out: q.qurl_kv_attn_chunk(x, 4, c, s, c, s, i4(2, 2), 2, i4(3), i4(2), 1.0, out,  # noqa: E731
                                               torch.zeros(16, dtype=torch.uint8))
    for x, out in ((h[:4], h[:4]), (h[:4], h[1:5]), (h[:4], h[:4, 32:]), (h[1:5, 32:], h[:4])):
        with pytest.raises(ValueError, match="overlaps"):
            call(x, out)

    class Launched(Exception):
        pass

    def load():
        raise Launched

    monkeypatch.setattr(q, "load", load)
    for x, out in ((h[:4], h[:4, 64:]), (h[:4, 64:], h[:4]), (h[:3], h[3:]), (h[:4], torch.empty_like(h[:4]))):
        with pytest.raises(Launched):  # (columns side by side, other rows, another matrix)
            call(x, out)
