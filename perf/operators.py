"""The rollout-step operators around the quantized linear layer, as they are measured.

Attention of one new token per sequence over the paged FP8 key-value cache, the
residual update with its norms and the quantization behind them, the sampler,
and the log-probability of given tokens with its gradient.  `run` computes them
either in their plain form (elementary torch operations) or, where `own` is
true, through the package's entry points.
"""
import math

import torch

own = False

NEG = float("-inf")


# ---------------------------------------------------------------- cases

def listed():
    return [
        # the latency of a single request early in its response: 7B-class heads, one short sequence
        dict(name="attn 7B one request", op="attn", B=1, q_heads=28, kv_heads=4, head_dim=128, block=16, max_len=300,
             min_len=300, window=0),
        # a rollout batch in full flight: 32B-class heads, responses of every length up to 8 k tokens
        dict(name="attn 32B rollout batch", op="attn", B=64, q_heads=40, kv_heads=8, head_dim=128, block=16,
             max_len=8192, min_len=256, window=0),
        # the stragglers of a rollout: few sequences, very long
        dict(name="attn 32B long tail", op="attn", B=4, q_heads=40, kv_heads=8, head_dim=128, block=64,
             max_len=131072, min_len=98304, window=0),
        # a padded batch of a small model: odd heads, odd pages, a sliding window, empty sequences
        dict(name="attn odd heads window", op="attn", B=37, q_heads=9, kv_heads=3, head_dim=80, block=24,
             max_len=2500, min_len=0, window=1000),
        # one request's next token, nucleus sampling
        dict(name="sample one row", op="sample", B=1, V=32000, dtype="bf16", mode="top_p"),
        # the rollout batch's next tokens: every row with its own temperature, top-k, top-p, min-p, some greedy
        dict(name="sample batch mixed", op="sample", B=256, V=131072, dtype="bf16", mode="mixed"),
        # plain temperature sampling of fp32 logits over an odd vocabulary (what on-policy training asks for)
        dict(name="sample fp32 untruncated", op="sample", B=64, V=100003, dtype="fp32", mode="plain"),
        # the trainer's log-probabilities of one packed micro-batch
        dict(name="logprob 4096 tokens", op="logprob", T=4096, V=131072, dtype="bf16", temperature=1.0, part="forward"),
        # and the logits' gradient of the same micro-batch
        dict(name="logprob grad 4096 tokens", op="logprob", T=4096, V=131072, dtype="bf16", temperature=1.0,
             part="backward"),
        # a short response in fp32, odd vocabulary, temperature: both directions
        dict(name="logprob both fp32", op="logprob", T=93, V=50001, dtype="fp32", temperature=0.7, part="both"),
        # a decode batch of the 32B class between attention and MLP, INT8
        dict(name="residual 64 tokens int8", op="residual", M=64, K=5120, qtype="int8", post=True, gate="vector"),
        # a prefill batch of the 32B class, FP8
        dict(name="residual 8192 tokens fp8", op="residual", M=8192, K=5120, qtype="fp8", post=True, gate="none"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "sample", "logprob", "residual"])
    if op == "attn":
        group, kv = rng.choice([1, 2, 3, 5, 7, 8, 16, 20]), rng.choice([1, 2, 4, 8])
        hd = rng.choice([64, 128, 128, 128, 80, 256, 16, 192])
        max_len = _log_int(rng, 1, 131072)
        B = max(1, min(_log_int(rng, 1, 256), int(3.2e9 / (max_len * kv * (hd + 4) * 2 * 3))))
        return dict(op="attn", B=B, q_heads=group * kv, kv_heads=kv, head_dim=hd,
                    block=rng.choice([1, 7, 16, 16, 24, 32, 64, 128, 256]), max_len=max_len,
                    min_len=rng.choice([0, max_len // 2, max_len]), window=rng.choice([0, 0, 0, 128, 1000, 4096]))
    if op == "sample":
        V = _log_int(rng, 5, 150000)
        return dict(op="sample", B=max(1, min(_log_int(rng, 1, 512), int(3.3e7 / V))), V=V,
                    dtype=rng.choice(["bf16", "fp32"]), mode=rng.choice(["top_p", "mixed", "mixed", "plain"]))
    if op == "logprob":
        V = _log_int(rng, 5, 150000)
        return dict(op="logprob", T=max(1, min(_log_int(rng, 1, 4096), int(2.5e8 / V))), V=V,
                    dtype=rng.choice(["bf16", "fp32"]), temperature=rng.choice([1.0, 1.0, 0.6, 1.3]),
                    part=rng.choice(["forward", "backward", "both"]))
    K = 16 * _log_int(rng, 2, 512)
    return dict(op="residual", M=_log_int(rng, 1, 8192), K=K, qtype=rng.choice(["fp8", "fp8", "int8"]),
                post=rng.choice([True, False]), gate=rng.choice(["none", "vector", "rows"]))


# ---------------------------------------------------------------- inputs

def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _rows(V, dtype):
    """A row stride of V values or a few more, a multiple of 16 bytes."""
    per = 16 // torch.empty(0, dtype=dtype).element_size()
    return (V + per - 1) // per * per


def _logits(g, n, V, dtype):
    """Rows of a language model's logits: a broad bulk and a few likely tokens, in a padded row."""
    l = torch.randn((n, _rows(V, dtype)), device="cuda", generator=g, dtype=torch.float32).mul_(2.0)
    likely = torch.randint(0, V, (n, 12), device="cuda", generator=g)
    l.scatter_add_(1, likely, torch.rand((n, 12), device="cuda", generator=g) * 14.0)
    return l.to(dtype)[:, :V]


def _prepare_attn(c, g):
    B, kvh, hd, blk = c["B"], c["kv_heads"], c["head_dim"], c["block"]
    r = torch.rand(B, device="cuda", generator=g)
    lens = (c["min_len"] + (r * (c["max_len"] - c["min_len"] + 1)).floor()).clamp_(max=c["max_len"])
    if c["min_len"] == 0 and B > 2:
        lens[1] = 0  # an empty sequence of a padded batch
    lens[0] = c["max_len"]
    lens = lens.to(torch.int32)
    per = (c["max_len"] + blk - 1) // blk
    # the pages of the sequences, scattered over a pool of twice as many tokens as the batch may hold at
    # its longest, at most 1.5 M
    pages = max(per * B + 3, min(2 * per * B, 1500000 // blk))
    table = torch.randperm(pages, device="cuda", generator=g)[:per * B].view(B, per).to(torch.int32)
    slots = pages * blk

    def cache():
        codes = torch.empty((slots, kvh, hd), dtype=torch.float8_e4m3fn, device="cuda")
        step = max(1, (1 << 28) // (kvh * hd))
        for i in range(0, slots, step):  # (bounded temporaries)
            x = torch.randn((min(step, slots - i), kvh, hd), device="cuda", generator=g, dtype=torch.float32)
            x = x / x.abs().amax(-1, keepdim=True) * 448.0
            codes[i:i + step] = x.to(torch.float8_e4m3fn)
        scale = (2.5 + 1.5 * torch.rand((slots, kvh), device="cuda", generator=g)) / 448.0
        return codes, scale

    kc, ks = cache()
    vc, vs = cache()
    q_dim = c["q_heads"] * hd
    qkv = torch.randn((B, q_dim + 2 * kvh * hd), device="cuda", generator=g).mul_(1.5).to(torch.bfloat16)
    s = dict(c=c, qkv=qkv, q_dim=q_dim, kc=kc, ks=ks, vc=vc, vs=vs, table=table, lens=lens, scale=hd ** -0.5)
    if own:
        import w8a8_precision_gemm_gb300 as q
        s["ws"] = q.kv_attn_workspace(B, c["q_heads"], kvh, hd, per, blk)
    return s


def _prepare_sample(c, g):
    B, V, mode = c["B"], c["V"], c["mode"]
    s = dict(c=c, logits=_logits(g, B, V, _dtype(c)), u=torch.rand(B, device="cuda", generator=g),
             temperature=0.6 + 0.6 * torch.rand(B, device="cuda", generator=g), top_k=None, top_p=None, min_p=None)
    if mode == "top_p":
        s["top_p"] = 0.9 + 0.09 * torch.rand(B, device="cuda", generator=g)
    if mode == "mixed":
        r = torch.rand((4, B), device="cuda", generator=g)
        s["temperature"] = torch.where(r[0] < 0.1, torch.zeros_like(r[0]), s["temperature"])  # some greedy rows
        k = torch.randint(1, 101, (B,), device="cuda", generator=g)
        s["top_k"] = torch.where(r[1] < 0.5, torch.zeros_like(k), k).to(torch.int32)
        s["top_p"] = torch.where(r[2] < 0.3, torch.ones_like(r[2]), 0.8 + 0.19 * r[0])
        s["min_p"] = torch.where(r[3] < 0.6, torch.zeros_like(r[3]), 0.002 + 0.05 * r[1])
    return s


def _prepare_logprob(c, g):
    T, V = c["T"], c["V"]
    s = dict(c=c, logits=_logits(g, T, V, _dtype(c)))
    t = torch.randint(0, V, (T,), device="cuda", generator=g)
    best = s["logits"].argmax(-1)
    r = torch.rand((2, T), device="cuda", generator=g)
    t = torch.where(r[0] < 0.6, best, t)
    s["targets"] = torch.where(r[1] < 0.08, torch.full_like(t, -1), t)  # prompt and padding positions
    s["dterm"] = torch.randn(T, device="cuda", generator=g)  # d objective term / d logp
    s["n"] = (s["targets"] >= 0).sum().to(torch.float64).reshape(1).clamp_(min=1.0)
    if c["part"] == "backward":  # the forward call's result
        s["lse"] = torch.logsumexp(s["logits"].float() / c["temperature"], -1)
    return s


def _prepare_residual(c, g):
    M, K = c["M"], c["K"]
    h = torch.randn((M, K), device="cuda", generator=g).mul_(2.0)
    wild = torch.randint(0, K, (max(1, K // 100),), device="cuda", generator=g)
    h[:, wild] *= 20.0  # the outlier channels of a residual stream
    gain = lambda: 1.0 + 0.1 * torch.randn(K, device="cuda", generator=g)  # noqa: E731
    gate = None
    if c["gate"] != "none":
        gate = torch.randn((1 if c["gate"] == "vector" else M, K), device="cuda", generator=g).mul_(0.3).add_(1.0)
        gate = gate.to(torch.bfloat16)
    return dict(c=c, h=h.to(torch.bfloat16), y=torch.randn((M, K), device="cuda", generator=g).to(torch.bfloat16),
                gate=gate, post=gain() if c["post"] else None, gamma=gain() * 1.5, rs=0.5, eps=1e-6)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return dict(attn=_prepare_attn, sample=_prepare_sample, logprob=_prepare_logprob,
                residual=_prepare_residual)[case["op"]](case, g)


# ---------------------------------------------------------------- one pass

def _plain_attn(s):
    c, blk, hd = s["c"], s["c"]["block"], s["c"]["head_dim"]
    B, kvh = c["B"], c["kv_heads"]
    L = s["table"].shape[1] * blk
    j = torch.arange(L, device="cuda")
    slot = (s["table"].long()[:, j // blk] * blk + j % blk)                       # [B, L]
    lens = s["lens"].long()[:, None]
    seen = j < lens
    if c["window"]:
        seen = seen & (j >= lens - c["window"])
    q = s["qkv"][:, :s["q_dim"]].float().view(B, kvh, -1, hd)                     # [B, kvh, group, hd]
    k = s["kc"].view(torch.uint8)[slot].view(torch.float8_e4m3fn).float() * s["ks"][slot][..., None]
    x = torch.einsum("bhgd,blhd->bhgl", q, k) * s["scale"]
    del k
    x = torch.where(seen[:, None, None], x, NEG)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == NEG, 0.0, m)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    v = s["vc"].view(torch.uint8)[slot].view(torch.float8_e4m3fn).float() * s["vs"][slot][..., None]
    o = torch.einsum("bhgl,blhd->bhgd", p, v) / torch.where(total == 0, 1.0, total)
    return o.reshape(B, -1).to(torch.bfloat16), (m + torch.log(total)).reshape(B, -1)


def _plain_sample(s):
    # 64 bits: the choice of a token goes by values next to a border
    l = s["logits"].double()
    B, V = l.shape
    one = torch.ones(B, device="cuda", dtype=torch.float64)
    t = s["temperature"].double()
    greedy = t == 0
    t = torch.where(greedy, one, t)[:, None]
    z = (l - l.amax(-1, keepdim=True)) / t
    w = torch.exp(z)
    order = torch.sort(l, dim=-1, descending=True, stable=True).indices
    ws = torch.gather(w, 1, order)
    rank = torch.arange(V, device="cuda")[None]
    keep = torch.ones_like(ws, dtype=torch.bool)
    if s["top_k"] is not None:
        k = s["top_k"][:, None]
        keep = keep & ((k <= 0) | (rank < k))
    if s["min_p"] is not None:
        keep = keep & (ws >= s["min_p"].double()[:, None])
    kept = torch.where(keep, ws, 0.0)
    if s["top_p"] is not None:
        p = s["top_p"].double()[:, None]
        before = torch.cumsum(kept, -1) - kept
        keep = keep & ((p >= 1) | (before < p * kept.sum(-1, keepdim=True)))
    keep = keep & (~greedy[:, None] | (rank == 0))
    kept = torch.zeros_like(w).scatter_(1, order, torch.where(keep, ws, 0.0))
    cum = torch.cumsum(kept, -1)
    token = (cum <= s["u"].double()[:, None] * cum[:, -1:]).sum(-1).clamp_(max=V - 1)
    zt = torch.gather(z, 1, token[:, None])[:, 0]
    return token, (zt - torch.log(w.sum(-1))).float(), (zt - torch.log(cum[:, -1])).float()


def _plain_logprob(s):
    c = s["c"]
    t, targets = c["temperature"], s["targets"]
    seen = targets >= 0
    at = targets.clamp(min=0)[:, None]
    x = s["logits"].float() / t
    out = []
    if c["part"] == "backward":
        lse = s["lse"]
    else:
        m = x.amax(-1, keepdim=True)
        lse = (m + torch.log(torch.exp(x - m).sum(-1, keepdim=True)))[:, 0]
        out += [torch.where(seen, torch.gather(x, 1, at)[:, 0] - lse, 0.0), torch.where(seen, lse, 0.0)]
    if c["part"] != "forward":
        g = torch.where(seen, s["dterm"] * (-1.0 / (s["n"].float() * t)), 0.0)[:, None]
        d = torch.exp(x - lse[:, None]).mul_(-g)
        d.scatter_add_(1, at, g)
        out.append(d.to(s["logits"].dtype))
    return out


def _plain_residual(s):
    # every step in 32 bits as written (the mean of squares in 64), the residual stream rounded to bf16
    c = s["c"]
    y = s["y"].float()

    def rms(x, eps):
        return 1.0 / torch.sqrt(x.double().square().mean(-1, keepdim=True).float() + eps)

    if s["post"] is not None:
        y = (y * rms(y, s["eps"])) * s["post"]
    if s["gate"] is not None:
        y = y * s["gate"].float()
    h = (s["h"].float() + y * s["rs"]).to(torch.bfloat16)
    x = h.float()
    v = (x * rms(x, s["eps"])) * s["gamma"]
    top = v.abs().amax(-1, keepdim=True)
    most = 127.0 if c["qtype"] == "int8" else 448.0
    sx = torch.where(top == 0, 1.0, top / most)
    r = v / sx
    if c["qtype"] == "int8":
        return h, (torch.round(r).clamp(-127, 127) * sx).to(torch.bfloat16), sx[:, 0]
    return h, r.clamp(-448, 448).to(torch.float8_e4m3fn), sx[:, 0]


def _own(s):
    import w8a8_precision_gemm_gb300 as q

    c = s["c"]
    if c["op"] == "attn":
        return q.kv_attn_decode(s["qkv"], c["q_heads"], s["kc"], s["ks"], s["vc"], s["vs"], s["table"], c["block"],
                                s["lens"], s["scale"], window=c["window"], want_lse=True, ws=s["ws"])
    if c["op"] == "sample":
        return q.sample(s["logits"], s["u"], s["temperature"], s["top_k"], s["top_p"], s["min_p"], want_kept=True)
    if c["op"] == "logprob":
        out = []
        lse = s.get("lse")
        if c["part"] != "backward":
            logp, lse = q.token_logprob(s["logits"], s["targets"], c["temperature"])
            out += [logp, lse]
        if c["part"] != "forward":
            out.append(q.token_logprob_grad(s["logits"], s["targets"], lse, s["dterm"], c["temperature"], scale=-1.0,
                                            denom=s["n"]))
        return out
    qt = q.INT8 if c["qtype"] == "int8" else q.FP8_E4M3
    h, xq, sx = q.residual_rmsnorm_quant(s["h"], s["y"], s["gamma"], qt, gamma_post=s["post"], gate=s["gate"],
                                         residual_scale=s["rs"], eps=s["eps"], eps_post=s["eps"])
    if c["qtype"] == "int8":  # 8-bit integers come back as the values they stand for
        return h, (xq.float() * sx[:, None]).to(torch.bfloat16), sx
    return h, xq, sx


def run(state):
    if own:
        return _own(state)
    return dict(attn=_plain_attn, sample=_plain_sample, logprob=_plain_logprob,
                residual=_plain_residual)[state["c"]["op"]](state)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c = case
    if c["op"] == "attn":
        mean = (c["max_len"] + (c["B"] - 1) * 0.5 * (c["max_len"] + c["min_len"])) / c["B"]
        tokens = c["B"] * (min(mean, c["window"]) if c["window"] else mean)
        out = c["B"] * c["q_heads"]
        return {"bytes": tokens * c["kv_heads"] * 2 * (c["head_dim"] + 4) + out * (4 * c["head_dim"] + 4)
                + 4 * tokens / c["block"], "flops": 4 * tokens * c["q_heads"] * c["head_dim"]}
    size = {"bf16": 2, "fp32": 4}.get(c.get("dtype"))
    if c["op"] == "sample":
        n = c["B"] * c["V"]
        return {"bytes": n * size + 36 * c["B"], "flops": 4 * n}
    if c["op"] == "logprob":
        n = c["T"] * c["V"]
        passes = {"forward": 1, "backward": 2, "both": 2}[c["part"]]
        return {"bytes": n * size * passes + 20 * c["T"], "flops": 4 * n * passes}
    n = c["M"] * c["K"]
    gate = {"none": 0, "vector": 2 * c["K"], "rows": 2 * n}[c["gate"]]
    return {"bytes": 7 * n + gate + 4 * c["K"] * (2 if c["post"] else 1) + 4 * c["M"], "flops": 15 * n}


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_attn(s):
    c, blk, hd, kvh = s["c"], s["c"]["block"], s["c"]["head_dim"], s["c"]["kv_heads"]
    outs, lses = [], []
    for b in range(c["B"]):
        n = int(s["lens"][b])
        first = max(0, n - c["window"]) if c["window"] else 0
        at = torch.arange(first, n, device="cuda")
        slot = s["table"][b].long().index_select(0, torch.div(at, blk, rounding_mode="floor")) * blk + at.remainder(blk)
        q = s["qkv"][b, :s["q_dim"]].double().view(kvh, -1, hd)
        if n == 0:
            outs.append(torch.zeros(s["q_dim"], device="cuda", dtype=torch.float64))
            lses.append(torch.full((c["q_heads"],), NEG, device="cuda", dtype=torch.float64))
            continue
        o, lse = [], []
        for h in range(kvh):
            k = s["kc"][:, h].view(torch.uint8).index_select(0, slot).view(torch.float8_e4m3fn).double()
            k = k * s["ks"][:, h].index_select(0, slot).double()[:, None]
            v = s["vc"][:, h].view(torch.uint8).index_select(0, slot).view(torch.float8_e4m3fn).double()
            v = v * s["vs"][:, h].index_select(0, slot).double()[:, None]
            x = (q[h] @ k.T) * s["scale"]
            lse.append(torch.logsumexp(x, -1))
            o.append((torch.softmax(x, -1) @ v).reshape(-1))
        outs.append(torch.cat(o))
        lses.append(torch.cat(lse))
    return torch.stack(outs), torch.stack(lses)


def _exact_sample(s):
    tokens, logp, kept_logp = [], [], []
    for b in range(s["c"]["B"]):
        l = s["logits"][b].double()
        t = float(s["temperature"][b])
        x = l if t == 0 else l / t
        lse = torch.logsumexp(x, 0)
        if t == 0:
            i = int((l == l.max()).nonzero()[0, 0])
            kept = x[i]
        else:
            logw = x - x.max()
            value, index = torch.sort(l, descending=True, stable=True)
            n = l.numel()
            if s["top_k"] is not None and 0 < int(s["top_k"][b]) < n:
                n = int(s["top_k"][b])
            if s["min_p"] is not None:
                n = min(n, int((torch.exp(logw[index]) >= float(s["min_p"][b])).sum()))
            if s["top_p"] is not None and float(s["top_p"][b]) < 1:
                share = torch.softmax(x[index[:n]], 0)
                n = 1 + int((torch.cumsum(share, 0)[:-1] < float(s["top_p"][b])).sum())
            chosen = torch.sort(index[:n]).values
            share = torch.cumsum(torch.softmax(x[chosen], 0), 0)
            i = int(chosen[min(n - 1, int(torch.searchsorted(share, float(s["u"][b]), right=True)))])
            kept = torch.logsumexp(x[chosen], 0)
        tokens.append(i)
        logp.append(x[i] - lse)
        kept_logp.append(x[i] - kept)
    return torch.tensor(tokens, device="cuda"), torch.stack(logp), torch.stack(kept_logp)


def _exact_logprob(s):
    c = s["c"]
    logp, lses, grads = [], [], []
    step = max(1, (1 << 27) // c["V"])
    for i in range(0, c["T"], step):
        x = s["logits"][i:i + step].double() / c["temperature"]
        t = s["targets"][i:i + step]
        ok = (t >= 0).double()
        lse = s["lse"][i:i + step].double() if c["part"] == "backward" else torch.logsumexp(x, -1)
        rows = torch.arange(len(t), device="cuda")
        logp.append((x[rows, t.clamp(min=0)] - lse) * ok)
        lses.append(lse * ok)
        if c["part"] != "forward":
            d = -torch.exp(x - lse[:, None])
            d[rows, t.clamp(min=0)] += 1.0
            w = s["dterm"][i:i + step].double() * ok * (-1.0 / (float(s["n"]) * c["temperature"]))
            grads.append((d * w[:, None]).float())  # (fp32: half the memory, 2^-24 of the value)
    out = [] if c["part"] == "backward" else [torch.cat(logp), torch.cat(lses)]
    return out + ([torch.cat(grads)] if grads else [])


def _exact_residual(s):
    def norm(x, gain):
        return x / (x.square().mean(-1, keepdim=True) + s["eps"]).sqrt() * gain.double()

    y = s["y"].double()
    if s["post"] is not None:
        y = norm(y, s["post"])
    if s["gate"] is not None:
        y = y * s["gate"].double()
    h = s["h"].double() + s["rs"] * y
    # the codes and the scale belong to the bf16 residual stream that is stored, not to h itself: a value
    # of h next to a rounding border of bf16 decides them, so they have no value from 64 bits alone
    return h, None, None


def exact(case, seed):
    if case["op"] == "attn" and case["B"] * case["kv_heads"] > 600:
        return None
    s = prepare(case, seed)
    return dict(attn=_exact_attn, sample=_exact_sample, logprob=_exact_logprob,
                residual=_exact_residual)[case["op"]](s)
