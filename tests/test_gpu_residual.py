"""The residual update with its norms and quantizer (qurl_residual_rmsnorm_quant):
the residual stream bit for bit against the fp32 steps written out in numpy (the
mean of squares in 64 bits), codes, scales and ms bit for bit against
qurl_rmsnorm_quant on the stored stream, and the dequantized codes against the
formula in 64 bits within half a code step."""
import numpy as np
import pytest
import torch

import w8a8_precision_gemm_gb300 as q

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _status():
    yield
    q.qurl_check_device_status()


def make(M, K, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    n = lambda *s: torch.randn(s, device="cuda", generator=g)  # noqa: E731
    h = n(M, K) * 2
    h[:, ::97] *= 20
    return h.to(torch.bfloat16), n(M, K).to(torch.bfloat16), 1 + 0.1 * n(K), (1 + 0.1 * n(K)) * 1.5, \
        (1 + 0.3 * n(M, K)).to(torch.bfloat16)


def stream(h, y, post, gate, rs, eps):
    f = np.float32
    h, y = h.float().cpu().numpy(), y.float().cpu().numpy()
    if post is not None:
        ms = (y.astype(np.float64) ** 2).mean(-1, keepdims=True).astype(f)
        y = (y * (f(1) / np.sqrt(ms + f(eps)))) * post.cpu().numpy()
    if gate is not None:
        y = y * gate.float().cpu().numpy()
    return torch.from_numpy(h + y * f(rs)).to(torch.bfloat16)


def check(M, K, qt, post=True, gate="rows", rs=0.7, eps=1e-6, seed=0, inplace=False):
    h, y, gp, gamma, gt = make(M, K, seed)
    gp = gp if post else None
    gt = {"rows": gt, "one": gt[:1], "vector": gt[0], "none": None}[gate]
    want = stream(h, y, gp, gt, rs, eps)
    ho, xq, sx = q.residual_rmsnorm_quant(h, y, gamma, qt, gamma_post=gp, gate=gt, residual_scale=rs, eps=eps,
                                          eps_post=eps, inplace=inplace)
    assert torch.equal(ho.cpu(), want)
    assert (ho.data_ptr() == h.data_ptr()) == inplace
    xr, sr = q.rmsnorm_quant(ho, gamma, qt, eps)
    assert torch.equal(xq.view(torch.uint8), xr.view(torch.uint8)) and torch.equal(sx, sr)
    x = ho.double()
    v = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * gamma.double()
    dec = xq.float().double() * sx.double()[:, None]
    # half a step: sx / 2 (INT8); 2^-4 of the value, at least 2^-10 sx (E4M3); and the fp32 roundings before
    half = sx.double()[:, None] / 2 if qt == q.INT8 else torch.maximum(v.abs() * 2.0 ** -4, sx.double()[:, None] * 2.0 ** -10)
    assert bool((dec - v).abs().le(half * 1.0001 + v.abs() * 2.0 ** -20).all())


@pytest.mark.parametrize("qt", [q.INT8, q.FP8_E4M3])
@pytest.mark.parametrize("M,K", [(1, 16), (3, 48), (64, 256), (65, 3584), (700, 5120), (5, 27648), (2, 40000), (400, 8208)])
def test_sizes(M, K, qt):
    check(M, K, qt, seed=M)


@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("gate", ["rows", "one", "vector", "none"])
def test_variants(post, gate):
    check(33, 512, q.FP8_E4M3, post, gate, rs=1.0)
    check(33, 512, q.INT8, post, gate, rs=-0.25, inplace=True)


def test_in_place_long_rows():
    check(3, 40000, q.INT8, inplace=True, seed=2)


def test_zero_rows_and_scale():
    h, y, gp, gamma, gt = make(4, 64)
    h[1] = 0
    y[1] = 0
    h[2] = 0
    ho, xq, sx = q.residual_rmsnorm_quant(h, y, gamma, q.INT8, gamma_post=gp, residual_scale=0.0, eps=0.0, eps_post=1e-6)
    assert torch.equal(ho, h)
    # eps = 0 and an empty row: 1 / 0 times 0 is no number; with eps the row quantizes to scale 1, codes 0
    ho, xq, sx = q.residual_rmsnorm_quant(h, y, gamma, q.INT8, gamma_post=gp, residual_scale=0.0)
    assert torch.equal(ho, h) and float(sx[1]) == 1.0 and not bool(xq[1].any()) and float(sx[2]) == 1.0


def test_strides_and_ms():
    h, y, gp, gamma, gt = make(7, 128, 5)
    wide = [torch.full((9, 160), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    H, Y, G, O = (w[:7, :128] for w in wide)
    H.copy_(h), Y.copy_(y), G.copy_(gt)
    xq = torch.empty((7, 128), dtype=torch.int8, device="cuda")
    sx, ms = torch.empty(7, device="cuda"), torch.empty(7, device="cuda")
    q.qurl_residual_rmsnorm_quant(H, Y, gamma, q.INT8, O, xq, sx, gp, G, 0.5, 1e-6, 1e-5, ms)
    assert torch.equal(O.cpu(), stream(h, y, gp, gt, 0.5, 1e-5))
    assert bool((wide[3][7:] == 3).all()) and bool((wide[3][:, 128:] == 3).all())
    _, _, mr = q.rmsnorm_quant(O.contiguous(), gamma, q.INT8, 1e-6, want_ms=True)
    assert torch.equal(ms, mr)


def test_feeds_the_linear():
    """The codes go into qurl_w8a8_linear as a quantizer's do."""
    h, y, gp, gamma, gt = make(64, 256, 9)
    W = torch.randn((96, 256), device="cuda") * 0.02
    Wq, sw, _, _ = q.prepare_weights(W, q.INT8, keep_scaled=False)
    ho, xq, sx = q.residual_rmsnorm_quant(h, y, gamma, q.INT8, gamma_post=gp, gate=gt)
    ws = q.workspace(64, 96, 256, q.INT8)
    Y = torch.empty((64, 96), dtype=torch.bfloat16, device="cuda")
    q.qurl_rmsnorm_quant_linear(ho, gamma, 1e-6, Wq, sw, q.INT8, Y, torch.empty_like(xq), torch.empty_like(sx), ws)
    assert torch.equal(q.linear(xq, sx, Wq, sw, q.INT8, ws), Y)


def test_wrong_tensors_are_refused():
    h, y, gp, gamma, gt = make(4, 64)
    for bad in (dict(gate=gt[:2]), dict(gate=gt.float()), dict(gamma_post=gp[:32]), dict(gamma_post=gp.double())):
        with pytest.raises(ValueError):
            q.residual_rmsnorm_quant(h, y, gamma, q.INT8, **bad)
    with pytest.raises(ValueError):
        q.residual_rmsnorm_quant(h, y[:2], gamma, q.INT8)
    with pytest.raises(ValueError):
        q.residual_rmsnorm_quant(h.float(), y, gamma, q.INT8)


@pytest.mark.parametrize("M,K", [(1, 5136), (3, 5136), (152, 8192), (153, 8192), (304, 5120), (305, 5120), (152, 5376),
                                 (400, 7168), (400, 8192), (305, 8176), (2, 8208)])
def test_widths_at_the_edges_of_the_variants(M, K):
    """Rows of one vector a thread and of four, at the widths and batches where the choice changes."""
    check(M, K, q.INT8, seed=M)
    check(M, K, q.FP8_E4M3, post=False, gate="one", seed=K, inplace=True)
