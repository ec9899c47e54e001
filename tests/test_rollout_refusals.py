"""Host-side refusals of the decode-step entry points (cache attention, residual
update, sampler, token log-probabilities): every bad argument is turned away
before any launch, and the binding turns away tensors of the wrong kind."""
import ctypes

import pytest
import torch

import w8a8_precision_gemm_gb300 as q
from w8a8_precision_gemm_gb300 import _build

FAKE = ctypes.c_void_p(0x10000)      # 16-byte aligned, never dereferenced: calls fail validation first
ODD = ctypes.c_void_p(0x10008)       # 8-byte aligned only
ODD4 = ctypes.c_void_p(0x10004)
ODD2 = ctypes.c_void_p(0x10002)
INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = 1, 2, 3, 4


@pytest.fixture(scope="module")
def L():
    _build.build()
    return q.load()


ATTN = dict(q=FAKE, ldq=1024, B=2, q_heads=8, kv_heads=2, hd=64, k=FAKE, ks=FAKE, v=FAKE, vs=FAKE, slots=64, table=FAKE,
            ldt=4, blocks=4, block=16, lens=FAKE, window=0, scale=0.1, out=FAKE, ldo=512, lse=FAKE, ws=FAKE,
            bytes=1 << 30, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(ks=None), INVALID), (dict(v=None), INVALID),
    (dict(vs=None), INVALID), (dict(table=None), INVALID), (dict(lens=None), INVALID), (dict(out=None), INVALID),
    (dict(ws=None), INVALID), (dict(B=-1), INVALID), (dict(q_heads=0), INVALID), (dict(kv_heads=0), INVALID),
    (dict(kv_heads=3), INVALID), (dict(hd=0), INVALID), (dict(slots=-1), INVALID), (dict(blocks=-1), INVALID),
    (dict(block=0), INVALID), (dict(ldt=3), INVALID), (dict(window=-1), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(ldq=504), INVALID), (dict(ldo=504), INVALID),
    (dict(hd=72), UNSUPPORTED), (dict(hd=272, ldq=4096, ldo=4096), UNSUPPORTED),
    (dict(blocks=1 << 20, ldt=1 << 20, block=(1 << 10) + 1), UNSUPPORTED), (dict(B=1 << 28), UNSUPPORTED),
    (dict(q=ODD), ALIGNMENT), (dict(k=ODD), ALIGNMENT), (dict(v=ODD), ALIGNMENT), (dict(out=ODD), ALIGNMENT),
    (dict(ws=ODD), ALIGNMENT), (dict(ldq=1028), ALIGNMENT), (dict(ldo=1028), ALIGNMENT), (dict(ks=ODD2), ALIGNMENT),
    (dict(vs=ODD2), ALIGNMENT), (dict(table=ODD2), ALIGNMENT), (dict(lens=ODD2), ALIGNMENT), (dict(lse=ODD2), ALIGNMENT),
])
def test_attn_validation(L, change, status):
    assert L.qurl_kv_attn_decode(*(ATTN | change).values()) == status


def test_attn_empty_batch_and_workspace_size(L):
    assert L.qurl_kv_attn_decode(*(ATTN | dict(B=0, q=None, out=None, lens=None)).values()) == 0
    size = L.qurl_kv_attn_workspace_size
    assert size(-1, 8, 2, 64, 4, 16) == 0 and size(2, 0, 2, 64, 4, 16) == 0 and size(2, 8, 2, 64, 4, 0) == 0
    big = size(64, 40, 8, 128, 512, 16)
    assert big > 0 and big % 16 == 0
    # a workspace serves every smaller batch, table and head
    for smaller in ((1, 40, 8, 128, 512, 16), (64, 40, 8, 128, 1, 16), (64, 40, 8, 64, 512, 16), (63, 40, 8, 128, 300, 16),
                    (64, 8, 8, 128, 512, 16)):
        assert size(*smaller) <= big, smaller


RES = dict(Y=FAKE, ldy=256, post=FAKE, eps_post=1e-6, gate=FAKE, ldg=256, rs=1.0, H=FAKE, ldh=256, Ho=FAKE, ldo=256,
           gamma=FAKE, eps=1e-6, M=4, K=256, qt=0, Xq=FAKE, sx=FAKE, ms=None, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(Y=None), INVALID), (dict(H=None), INVALID), (dict(Ho=None), INVALID), (dict(gamma=None), INVALID),
    (dict(Xq=None), INVALID), (dict(sx=None), INVALID), (dict(M=0), INVALID), (dict(K=-16), INVALID),
    (dict(ldy=128), INVALID), (dict(ldh=128), INVALID), (dict(ldo=128), INVALID), (dict(ldg=128), INVALID),
    (dict(qt=2), INVALID), (dict(eps=-1.0), INVALID), (dict(eps_post=float("nan")), INVALID),
    (dict(rs=float("inf")), INVALID), (dict(ldo=512), INVALID), (dict(K=248, ldy=256), UNSUPPORTED),
    (dict(Y=ODD), ALIGNMENT), (dict(H=ODD, Ho=FAKE), ALIGNMENT), (dict(gate=ODD), ALIGNMENT), (dict(post=ODD), ALIGNMENT),
    (dict(ldg=260), ALIGNMENT), (dict(ldy=260), ALIGNMENT), (dict(Xq=ODD), ALIGNMENT),
])
def test_residual_validation(L, change, status):
    assert L.qurl_residual_rmsnorm_quant(*(RES | change).values()) == status


SAMPLE = dict(x=FAKE, type=0, B=2, V=100, ld=104, t=FAKE, k=FAKE, p=FAKE, m=FAKE, u=FAKE, token=FAKE, logp=FAKE,
              kept=FAKE, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(x=None), INVALID), (dict(type=2), INVALID), (dict(B=-1), INVALID), (dict(V=0), INVALID), (dict(ld=96), INVALID),
    (dict(u=None), INVALID), (dict(token=None), INVALID), (dict(x=ODD), ALIGNMENT), (dict(ld=100), ALIGNMENT),
    (dict(type=1, ld=102), ALIGNMENT), (dict(token=ODD4), ALIGNMENT), (dict(u=ODD2), ALIGNMENT),
    (dict(t=ODD2), ALIGNMENT), (dict(k=ODD2), ALIGNMENT), (dict(p=ODD2), ALIGNMENT), (dict(m=ODD2), ALIGNMENT),
    (dict(logp=ODD2), ALIGNMENT), (dict(kept=ODD2), ALIGNMENT), (dict(V=(1 << 24) + 1, ld=1 << 25), UNSUPPORTED),
])
def test_sample_validation(L, change, status):
    assert L.qurl_sample(*(SAMPLE | change).values()) == status
    assert L.qurl_sample(*(SAMPLE | dict(B=0, x=None)).values()) == 0


LOGP = dict(x=FAKE, type=0, T=2, V=100, ld=104, targets=FAKE, t=1.0, logp=FAKE, lse=FAKE, stream=None)
GRAD = dict(x=FAKE, type=0, T=2, V=100, ld=104, targets=FAKE, t=1.0, lse=FAKE, g=FAKE, scale=1.0, denom=None, d=FAKE,
            ldd=104, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(x=None), INVALID), (dict(type=-1), INVALID), (dict(T=-1), INVALID), (dict(V=0), INVALID), (dict(ld=96), INVALID),
    (dict(targets=None), INVALID), (dict(lse=None), INVALID), (dict(t=0.0), INVALID), (dict(t=float("nan")), INVALID),
    (dict(t=-1.0), INVALID), (dict(t=1e7), INVALID), (dict(x=ODD), ALIGNMENT), (dict(ld=100), ALIGNMENT),
    (dict(targets=ODD4), ALIGNMENT), (dict(lse=ODD2), ALIGNMENT),
    (dict(V=(1 << 30) + 1, ld=(1 << 30) + 8), UNSUPPORTED),
])
def test_logprob_validation(L, change, status):
    assert L.qurl_token_logprob(*(LOGP | change).values()) == status
    if "ld" in change:
        change = change | dict(d=ODD)  # (else the two strides of one buffer differ)
    assert L.qurl_token_logprob_grad(*(GRAD | change).values()) == status
    assert L.qurl_token_logprob(*(LOGP | dict(T=0, x=None)).values()) == 0
    assert L.qurl_token_logprob_grad(*(GRAD | dict(T=0, x=None)).values()) == 0


@pytest.mark.parametrize("change,status", [
    (dict(d=None), INVALID), (dict(g=None), INVALID), (dict(scale=float("nan")), INVALID), (dict(ldd=112), INVALID),
    (dict(ldd=96), INVALID), (dict(d=ODD), ALIGNMENT), (dict(denom=ODD4), ALIGNMENT), (dict(g=ODD2), ALIGNMENT),
])
def test_grad_validation(L, change, status):
    assert L.qurl_token_logprob_grad(*(GRAD | change).values()) == status


def test_binding_takes_device_tensors_only():
    x, u = torch.zeros(2, 16), torch.zeros(2)
    with pytest.raises(ValueError):
        q.sample(x, u)
    with pytest.raises(ValueError):
        q.token_logprob(x, torch.zeros(2, dtype=torch.int64))
    h = torch.zeros(2, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        q.residual_rmsnorm_quant(h, h, torch.ones(16), q.INT8)
    c, s = torch.zeros(4, 1, 16, dtype=torch.uint8), torch.ones(4, 1)
    with pytest.raises(ValueError):
        q.kv_attn_decode(h, 1, c, s, c, s, torch.zeros(2, 1, dtype=torch.int32), 2, torch.zeros(2, dtype=torch.int32),
                         ws=torch.zeros(16, dtype=torch.uint8))


class _Streams:
    """Stands in for torch.cuda.stream: which stream an allocation belongs to."""

    def __init__(self, monkeypatch):
        self.now, self.seen = ["current"], []
        outer = self

        class Use:
            def __init__(self, s):
                self.s = s

            def __enter__(self):
                outer.now.append(self.s)

            def __exit__(self, *exc):
                outer.now.pop()

        monkeypatch.setattr(torch.cuda, "stream", Use)
        for name in ("empty", "zeros", "empty_strided"):
            make = getattr(torch, name)
            monkeypatch.setattr(torch, name, lambda *a, make=make, **k: (self.seen.append(self.now[-1]), make(*a, **k))[1])


@pytest.mark.parametrize("positional", [False, True])
def test_allocations_belong_to_the_stream_of_the_call(monkeypatch, positional):
    """What a helper allocates is allocated for the stream that its kernel runs on."""
    bf, B, K = torch.bfloat16, 2, 16
    x, h, u, t = torch.zeros(B, 16), torch.zeros(B, K, dtype=bf), torch.zeros(B), torch.zeros(B, dtype=torch.int64)
    cache, scale = torch.zeros(4, 1, 16, dtype=torch.uint8), torch.ones(4, 1)
    table, lens, one = torch.zeros(B, 1, dtype=torch.int32), torch.zeros(B, dtype=torch.int32), torch.ones(B)
    codes, w = torch.zeros(B, K, dtype=torch.int8), torch.zeros(B, K)
    q4 = (torch.zeros(B, K // 2, dtype=torch.uint8), torch.zeros(B, 1, dtype=torch.uint8), one)
    calls = [
        (q.kv_attn_decode, (h, 1, cache, scale, cache, scale, table, 2, lens, None, 0, True, None)),
        (q.residual_rmsnorm_quant, (h, h, torch.ones(K), q.INT8, None, None, 1.0, 1e-6, 1e-6, False)),
        (q.sample, (x, u, None, None, None, None, True)),
        (q.token_logprob, (x, t, 1.0)),
        (q.token_logprob_grad, (x, t, u, u, 1.0, 1.0, None, False)),
        (q.prepare_weights, (w, q.INT8, 1.5, torch.ones(K), True)),
        (q.quant_act, (h, q.INT8, 1.0)),
        (q.rmsnorm_quant, (h, torch.ones(K), q.INT8, 1e-6, True)),
        (q.silu_mul_quant, (h, q.INT8, 1.0, True)),
        (q.linear, (codes, one, codes, one, q.INT8, None)),
        (q.gemm_acc, (codes, codes, q.INT8, None)),
        (q.count_diff, (codes, codes)),
        (q.nvfp4_quant, (h, 1.0)),
        (q.nvfp4_linear, (q4, q4, None)),
        (q.nvfp4_gemm_acc, (q4, q4, None)),
        (q.acr_objective, (one, one, one, one, torch.ones(B, dtype=torch.uint8), 0.2, 2.0, True, True, True, None)),
    ]
    for name in dir(q):  # the C ABI: nothing is launched here
        if name.startswith("qurl_") and not name.endswith("_size"):
            monkeypatch.setattr(q, name, lambda *a, **k: None)
    streams = _Streams(monkeypatch)
    for f, args in calls:
        streams.seen.clear()
        f(*args, "s") if positional else f(*args, stream="s")
        assert streams.seen and set(streams.seen) == {"s"}, f.__name__
        streams.seen.clear()
        f(*args)
        assert streams.seen and set(streams.seen) == {"current"}, f.__name__
