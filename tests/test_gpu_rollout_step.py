"""The operators of a rollout and training step together, as an engine runs them:
a decoder layer's decode step (RMSNorm -> qkv linear -> FP8 cache -> attention ->
output projection -> residual update and norms -> MLP -> residual update and norm
-> vocabulary projection -> sampler) for several tokens, then the trainer's side
(token log-probabilities under two policies -> ACR objective -> logits' gradient).

Each stage is checked on the stage before it as the GPU computed it, so the
tolerances are those of a single stage (see the tests of each): the attention's
output within 2^-8 of the value and 2^-10 of the weighted magnitudes, log-
probabilities within 1e-5."""
import pytest
import torch

import w8a8_precision_gemm_gb300 as q

pytestmark = pytest.mark.gpu

HID, HEADS, KV, HD, INTER, VOCAB, BLOCK = 256, 4, 2, 64, 512, 1000, 16
B, STEPS = 5, 40


class Layer:
    def __init__(self, qt, seed=0):
        self.qt = qt
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        w = lambda n, k: torch.randn((n, k), device="cuda", generator=g) * k ** -0.5  # noqa: E731
        gain = lambda: 1 + 0.1 * torch.randn(HID, device="cuda", generator=g)  # noqa: E731
        qkv_n = (HEADS + 2 * KV) * HD
        self.qkv, self.sqkv, self.g1, _ = q.prepare_weights(w(qkv_n, HID), qt, gamma=gain())
        self.o, self.so, _, _ = q.prepare_weights(w(HID, HEADS * HD), qt)
        self.gu, self.sgu, self.g2, _ = q.prepare_weights(w(2 * INTER, HID), qt, gamma=gain())
        self.down, self.sdown, _, _ = q.prepare_weights(w(HID, INTER), qt)
        self.lm, self.slm, self.g3, _ = q.prepare_weights(w(VOCAB, HID) * 6, qt, gamma=gain())
        self.post1, self.post2 = gain(), gain()
        self.emb = torch.randn((VOCAB, HID), device="cuda", generator=g).to(torch.bfloat16)
        per = -(-STEPS // BLOCK)
        pages = B * per + 2
        self.table = torch.randperm(pages, device="cuda", generator=g)[:B * per].view(B, per).to(torch.int32)
        self.cache = q.kv_cache(pages * BLOCK, KV, HD)
        self.attn_ws = q.kv_attn_workspace(B, HEADS, KV, HD, per, BLOCK)
        self.ws = max((q.workspace(B, n, k, qt) for n, k in ((qkv_n, HID), (HID, HEADS * HD), (2 * INTER, HID), (HID, INTER),
                                                               (VOCAB, HID))), key=lambda t: 0 if t is None else t.numel())
        e = lambda n, t=torch.bfloat16: torch.empty((B, n), dtype=t, device="cuda")  # noqa: E731
        c = q.code_dtype(qt)
        self.y_qkv, self.attn, self.y_o, self.y_gu, self.y_down, self.logits = (
            e(n) for n in (qkv_n, HEADS * HD, HID, 2 * INTER, HID, VOCAB))
        self.h1, self.h2, self.x1, self.x2 = e(HID), e(HID), e(HID, c), e(HID, c)
        self.xs, self.xo, self.xd = e(HID, c), e(HEADS * HD, c), e(INTER, c)
        self.s = [torch.empty(B, device="cuda") for _ in range(5)]
        self.lse = torch.empty((B, HEADS), device="cuda")
        self.h = e(HID)
        self.lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.slots = torch.zeros(B, dtype=torch.int64, device="cuda")
        self.token = torch.zeros(B, dtype=torch.int64, device="cuda")
        self.logp = torch.empty(B, device="cuda")
        self.u = torch.empty(B, device="cuda")
        self.top_p = torch.full((B,), 0.95, device="cuda")

    def step(self):
        """One new token per sequence; lens, slots and u are set before."""
        torch.index_select(self.emb, 0, self.token, out=self.h)
        q.qurl_rmsnorm_quant_linear(self.h, self.g1, 1e-6, self.qkv, self.sqkv, self.qt, self.y_qkv, self.xs, self.s[0], self.ws)
        q.qurl_kv_cache_quant(self.y_qkv, HEADS * HD, KV, HD, self.slots, *self.cache)
        q.qurl_kv_attn_decode(self.y_qkv, HEADS, *self.cache, self.table, BLOCK, self.lens, HD ** -0.5, self.attn,
                              self.attn_ws, lse=self.lse)
        q.qurl_quant_act_linear(self.attn, 1.5, self.o, self.so, self.qt, self.y_o, self.xo, self.s[1], self.ws)
        q.qurl_residual_rmsnorm_quant(self.h, self.y_o, self.g2, self.qt, self.h1, self.x1, self.s[2], self.post1)
        q.qurl_w8a8_linear(self.x1, self.s[2], self.gu, self.sgu, self.qt, self.y_gu, self.ws)
        q.qurl_silu_mul_quant_linear(self.y_gu, 1.5, self.down, self.sdown, self.qt, self.y_down, self.xd, self.s[3], self.ws)
        q.qurl_residual_rmsnorm_quant(self.h1, self.y_down, self.g3, self.qt, self.h2, self.x2, self.s[4], self.post2)
        q.qurl_w8a8_linear(self.x2, self.s[4], self.lm, self.slm, self.qt, self.logits, self.ws)
        q.qurl_sample(self.logits, self.u, self.token, top_p=self.top_p, logp=self.logp)

    def place(self, t):
        """Lengths and slots of the token at position t; sequence 3 is finished (padding) from 20 on."""
        t = torch.full((B,), t, device="cuda")
        done = torch.arange(B, device="cuda").eq(3) & (t >= 20)
        page = self.table.long().gather(1, (t // BLOCK)[:, None])[:, 0]
        self.slots.copy_(torch.where(done, -1, page * BLOCK + t % BLOCK))
        self.lens.copy_(torch.where(done, 20, t + 1).int())


def check_attention(L, keys, values):
    """The step's attention against all the step's keys and values so far (bf16, as projected)."""
    k8, ks, v8, vs = L.cache
    x = L.y_qkv[:, :HEADS * HD].double().view(B, KV, -1, HD)
    for b in range(B):
        n = int(L.lens[b])
        j = torch.arange(n, device="cuda")
        slot = L.table[b].long()[j // BLOCK] * BLOCK + j % BLOCK
        k = k8.view(torch.uint8)[slot].view(torch.float8_e4m3fn).double() * ks[slot].double()[..., None]
        v = v8.view(torch.uint8)[slot].view(torch.float8_e4m3fn).double() * vs[slot].double()[..., None]
        # the cache holds what was projected, to half a step of e4m3 (2^-4 of the value, 2^-10 of the scale)
        for got, want, sc in ((k, keys, ks[slot]), (v, values, vs[slot])):
            want = torch.stack([s[b] for s in want[:n]]).double()
            assert bool((got - want).abs().le(want.abs() * 2.0 ** -4 * 1.001 + sc.double()[..., None] * 2.0 ** -10).all())
        s = torch.einsum("hgd,lhd->hgl", x[b], k) * HD ** -0.5
        p = torch.softmax(s, -1)
        want = torch.einsum("hgl,lhd->hgd", p, v).reshape(-1)
        mag = torch.einsum("hgl,lhd->hgd", p, v.abs()).reshape(-1)
        assert bool((L.attn[b].double() - want).abs().le(want.abs() * 2.0 ** -8 + mag * 2.0 ** -10).all())
        assert bool((L.lse[b].double() - torch.logsumexp(s, -1).reshape(-1)).abs().le(1e-4).all())


@pytest.mark.parametrize("qt", [q.INT8, q.FP8_E4M3])
def test_decode_steps_then_training(qt):
    L = Layer(qt)
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    keys, values, tokens, logps, logits = [], [], [], [], []
    graph = None
    for t in range(STEPS):
        L.place(t)
        L.u.copy_(torch.rand(B, device="cuda", generator=g))
        if t == 3:  # from here on the captured step is replayed
            graph = torch.cuda.CUDAGraph()
            held = L.token.clone()
            with torch.cuda.graph(graph):
                L.step()
            L.token.copy_(held)
        L.step() if graph is None else graph.replay()
        kv = L.y_qkv[:, HEADS * HD:].clone().view(B, 2, KV, HD)
        keys.append(kv[:, 0])
        values.append(kv[:, 1])
        check_attention(L, keys, values)
        z = L.logits.double()
        ref = torch.log_softmax(z, -1).gather(1, L.token[:, None])[:, 0]
        assert bool((L.logp.double() - ref).abs().le(1e-5).all())
        # the token lies in the smallest set of 0.95
        order = torch.sort(z, dim=-1, descending=True, stable=True)
        before = torch.softmax(order.values, -1).cumsum(-1) - torch.softmax(order.values, -1)
        rank = order.indices.eq(L.token[:, None]).int().argmax(-1)
        assert bool((before.gather(1, rank[:, None])[:, 0] < 0.95 + 1e-9).all())
        tokens.append(L.token.clone())
        logps.append(L.logp.clone())
        logits.append(L.logits.clone())
    q.qurl_check_device_status()

    # ---- the trainer: the same responses under a proximal and a trained policy (the rollout's logits, moved a little)
    x = torch.cat(logits)
    T = x.shape[0]
    target = torch.cat(tokens)
    mask = torch.ones(T, dtype=torch.uint8, device="cuda")
    mask[3 + 20 * B::B] = 0  # the finished sequence's padding
    target = torch.where(mask.bool(), target, -1)
    prox = (x.float() + 0.02 * torch.randn(x.shape, device="cuda", generator=g)).to(torch.bfloat16)
    new = (prox.float() + 0.05 * torch.randn(x.shape, device="cuda", generator=g)).to(torch.bfloat16)
    adv = torch.randn(T, device="cuda", generator=g)
    logp_prox, _ = q.token_logprob(prox, target)
    logp, lse = q.token_logprob(new, target)
    behav = torch.cat(logps)
    stats, dterm, term = q.acr_objective(logp, logp_prox, behav, adv, mask, want_term=True)
    d = q.token_logprob_grad(new, target, lse, dterm, scale=-1.0, denom=stats[1:2])
    q.qurl_check_device_status()
    assert float(stats[1]) == int(mask.sum())

    leaf = new.double().requires_grad_(True)
    lp = torch.log_softmax(leaf, -1).gather(1, target.clamp(min=0)[:, None])[:, 0]
    w = torch.exp(logp_prox.double() - behav.double()).clamp(max=2.0)
    R = torch.exp(lp - logp_prox.double())
    c = torch.minimum(R.clamp(min=0.8), 1.2 / w)
    loss = -(torch.minimum(R * adv, c * adv) * w * mask).sum() / mask.sum()
    loss.backward()
    assert abs(float(stats[0]) + float(loss.detach())) < 1e-5
    near = ((R - 0.8).abs() < 1e-4) | ((R - 1.2 / w).abs() < 1e-4)  # a clip decided by the last bits
    ok = ~near.detach()
    # dterm's relative 2e-6, the exponentials' 2^-17 of p |w|, and half a step of bf16
    weight = (dterm.double().abs() / float(stats[1]))[:, None]
    err = (d.double() - leaf.grad).abs()
    assert bool(err[ok].le(leaf.grad.abs()[ok] * 2.0 ** -8 * 1.01 + (weight * 2.0 ** -15)[ok]).all())
    assert not bool(d[mask == 0].any())


def test_calls_given_a_stream_do_not_touch_the_current_one():
    """Every operator with stream=: the current stream is busy and its freed memory full of ones, the results on
    the given stream are those of the current stream alone."""
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    r = lambda *s: torch.randn(s, device="cuda", generator=g)  # noqa: E731
    n, hid, V, slots = 3, 256, 5000, 4096
    kc, ks, vc, vs = q.kv_cache(slots, 2, 64)
    q.qurl_kv_cache_quant(r(slots, 8 * 64).to(torch.bfloat16), 4 * 64, 2, 64, torch.arange(slots, device="cuda"), kc, ks, vc, vs)
    table = torch.arange(slots // 16, device="cuda", dtype=torch.int32)[None].repeat(n, 1).contiguous()
    lens = torch.tensor([4000, 17, 2500], dtype=torch.int32, device="cuda")
    query, h, y = r(n, 4 * 64).to(torch.bfloat16), r(n, hid).to(torch.bfloat16), r(n, hid).to(torch.bfloat16)
    gain, logits, u, dl = 1 + 0.1 * r(hid), r(n, V), torch.rand(n, device="cuda", generator=g), r(n)
    target, top_p = torch.tensor([5, -1, 4999], device="cuda"), torch.full_like(u, .9)

    def calls(stream):
        logp, lse = q.token_logprob(logits, target, stream=stream)
        return [*q.kv_attn_decode(query, 4, kc, ks, vc, vs, table, 16, lens, want_lse=True, stream=stream),
                *q.residual_rmsnorm_quant(h, y, gain, q.INT8, stream=stream),
                *q.sample(logits, u, top_p=top_p, want_kept=True, stream=stream), logp, lse,
                q.token_logprob_grad(logits, target, lse, dl, stream=stream)]

    want = calls(None)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        dirt = [torch.full((1 << k,), 255, dtype=torch.uint8, device="cuda") for k in range(6, 24)]
        torch.cuda.synchronize()
        del dirt
        torch.cuda._sleep(1 << 27)
        got = calls(s)
        s.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    torch.cuda.synchronize()


@pytest.mark.parametrize("mode", [0, 1, 2])
@pytest.mark.parametrize("qt", [q.INT8, q.FP8_E4M3])
def test_a_latched_parameter_leaves_later_calls_alone(qt, mode):
    """A page, a target or a parameter out of range is reported at the next look at the status; the calls between,
    each with other rows, compute what they compute without it, the linears that hand over inside their kernel
    among them."""
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    for M, N, K in ((16, 4096, 4096), (64, 4608, 3584), (64, 512, 18944)):
        W = torch.randn((N, K), device="cuda", generator=g) * 0.02
        Wq, sw, _, _ = q.prepare_weights(W, qt, keep_scaled=False)
        X = torch.randn((8, M, K), device="cuda", generator=g).to(torch.bfloat16)
        ws = q.workspace(M, N, K, qt)
        xq, sx = torch.empty((M, K), dtype=q.code_dtype(qt), device="cuda"), torch.empty(M, device="cuda")
        logits = torch.randn((4, 1024), device="cuda", generator=g)
        u = torch.tensor([.5, 1.5, .5, .5], device="cuda")
        out = torch.full((2, 8, M, N), 7.0, dtype=torch.bfloat16, device="cuda")
        before = q.qurl_set_fused_decode(mode)
        try:
            for k in (0, 1):
                if k:
                    q.sample(logits, u)  # u = 1.5 is out of range
                for x, y in zip(X, out[k]):
                    q.qurl_quant_act_linear(x, 1.5, Wq, sw, qt, y, xq, sx, ws)
                if k:
                    with pytest.raises(q.QurlError) as e:
                        q.qurl_check_device_status()
                    assert e.value.status == 1  # QURL_ERR_INVALID_ARG
                q.qurl_check_device_status()
        finally:
            q.qurl_set_fused_decode(before)
        assert torch.equal(out[0], out[1]) and not bool(ws[-256:].any())
