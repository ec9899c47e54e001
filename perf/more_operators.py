"""The operators between the qkv linear and the output projection of a step that carries
prompts, chunks of prompts or several draft tokens per sequence, as they are measured.

Pages of the paged cache taken and given back on the GPU, rotary positions (alone in both
directions, and together with the FP8 quantization into the cache), and causal attention of
the new tokens over the cache.  `run` computes them either in their plain form (elementary
torch operations) or, where `own` is true, through the package's entry points.
"""
import math

import torch

own = False

NEG = float("-inf")


# ---------------------------------------------------------------- cases

def listed():
    return [
        # the latency of one request's prompt: 7B-class heads
        dict(name="chunk 7B one prompt", op="chunk", B=1, q_heads=28, kv_heads=4, head_dim=128, block=16, new=300,
             min_new=300, cached=0, min_cached=0, window=0),
        # a prefill batch of the 32B class: eight prompts of about a thousand tokens
        dict(name="chunk 32B prompts", op="chunk", B=8, q_heads=40, kv_heads=8, head_dim=128, block=16, new=1200,
             min_new=848, cached=0, min_cached=0, window=0),
        # one chunk of a long prompt, most of which is cached already
        dict(name="chunk 32B long prompt", op="chunk", B=1, q_heads=40, kv_heads=8, head_dim=128, block=64, new=2048,
             min_new=2048, cached=30720, min_cached=30720, window=0),
        # draft tokens of a rollout batch verified: four new tokens a sequence, responses of every length
        dict(name="chunk 32B four tokens each", op="chunk", B=64, q_heads=40, kv_heads=8, head_dim=128, block=16,
             new=4, min_new=4, cached=8192, min_cached=256, window=0),
        # a padded batch of a small model: chunks beside single tokens and empty sequences, odd heads, a sliding window
        dict(name="chunk odd heads window", op="chunk", B=21, q_heads=9, kv_heads=3, head_dim=80, block=24, new=500,
             min_new=0, cached=2500, min_cached=0, window=1000),
        # the bookkeeping of one decode step of a rollout batch
        dict(name="pages 64 requests", op="pages", B=64, new=1, min_new=1, cached=8192, block=16, finished=0.05),
        # a step of a large batch: finished responses give their pages back, prompts come in beside decoding requests
        dict(name="pages 1000 requests prompts", op="pages", B=1000, new=97, min_new=0, cached=4000, block=16,
             finished=0.2),
        # one request's next token, 7B-class heads
        dict(name="rope cache one token", op="cache", M=1, q_heads=28, kv_heads=4, head_dim=128, rot=128,
             layout="half", far=4096, scaling="none", pad=0.0),
        # a prefill batch of the 32B class, frequencies scaled for long contexts
        dict(name="rope cache 8192 tokens", op="cache", M=8192, q_heads=40, kv_heads=8, head_dim=128, rot=128,
             layout="half", far=131072, scaling="ramp", pad=0.02),
        # a small model that rotates part of its head, neighbouring values as pairs, odd counts
        dict(name="rope cache part interleaved", op="cache", M=997, q_heads=9, kv_heads=3, head_dim=80, rot=32,
             layout="interleaved", far=30000, scaling="linear", pad=0.1),
        # the gradient of the rotation in the trainer: queries and keys of one micro-batch, bf16
        dict(name="rope gradient 8192 tokens", op="rope", M=8192, heads=48, head_dim=128, rot=128, layout="half",
             far=8192, scaling="none", dtype="bf16", inverse=True),
        # fp32 rows, a head of which a quarter is rotated, positions of a very long context
        dict(name="rope fp32 part far", op="rope", M=1201, heads=12, head_dim=80, rot=20, layout="half", far=1000000,
             scaling="ramp", dtype="fp32", inverse=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "chunk", "pages", "cache", "rope"])
    if op == "chunk":
        group, kv = rng.choice([1, 2, 3, 5, 7, 8, 16]), rng.choice([1, 2, 4, 8])
        hd = rng.choice([64, 128, 128, 128, 80, 256, 16, 192])
        new = _log_int(rng, 1, 8192)
        cached = rng.choice([0, _log_int(rng, 1, 65536)])
        # pairs of a query head and a token, and tokens of the pool, as in the largest listed cases at most
        pairs = group * kv * hd * new * (cached + new / 2 + 1)
        B = max(1, min(_log_int(rng, 1, 128), int(2.5e11 / pairs), int(1.5e9 / ((cached + new) * kv * (hd + 4) * 6))))
        if pairs > 2.5e11:
            cached = 0
        if group * kv * hd * new * (cached + new / 2 + 1) > 2.5e11:
            new = 1024
        return dict(op="chunk", B=B, q_heads=group * kv, kv_heads=kv, head_dim=hd,
                    block=rng.choice([1, 7, 16, 16, 24, 32, 64, 128, 256]), new=new, min_new=rng.choice([0, new // 2, new]),
                    cached=cached, min_cached=rng.choice([0, cached // 2, cached]), window=rng.choice([0, 0, 0, 128, 1000, 4096]))
    if op == "pages":
        B = _log_int(rng, 1, 2000)
        new = rng.choice([1, 1, 4, _log_int(rng, 1, max(1, 65536 // B))])
        return dict(op="pages", B=B, new=new, min_new=rng.choice([0, 1]), cached=_log_int(rng, 1, 8192),
                    block=rng.choice([1, 7, 16, 16, 24, 32, 64, 128]), finished=rng.choice([0.0, 0.05, 0.3]))
    hd = rng.choice([64, 128, 128, 128, 80, 256, 96])
    layout = rng.choice(["half", "half", "interleaved"])
    rot = rng.choice([hd, hd, hd // 2, hd // 4])
    far, scaling = _log_int(rng, 100, 1000000), rng.choice(["none", "linear", "ramp"])
    M = _log_int(rng, 1, 8192)
    if op == "cache":
        group, kv = rng.choice([1, 3, 5, 7]), rng.choice([1, 2, 4, 8])
        if M * (group + 2) * kv * hd > 6e7:
            M = 1000
        return dict(op="cache", M=M, q_heads=group * kv, kv_heads=kv, head_dim=hd, rot=rot, layout=layout, far=far,
                    scaling=scaling, pad=rng.choice([0.0, 0.1]))
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    heads = rng.choice([1, 5, 12, 32, 48])
    if M * heads * hd * (2 if dtype == "fp32" else 1) > 5e7:
        M = 1000
    return dict(op="rope", M=M, heads=heads, head_dim=hd, rot=rot, layout=layout, far=far, scaling=scaling, dtype=dtype,
                inverse=rng.choice([False, True]))


# ---------------------------------------------------------------- inputs

def _chunk_lengths(c, seed):
    """(cached, new) tokens of each sequence, on the host.  A case adds the same numbers of new
    tokens whatever the seed, to sequences in another order."""
    g, fixed = torch.Generator(), torch.Generator()
    g.manual_seed(seed + 77)
    fixed.manual_seed(1)

    def spread(g, lo, hi):
        u = torch.rand(c["B"], generator=g, dtype=torch.float64)
        return (lo + (u * (hi - lo + 1)).floor()).clamp(max=hi).long()

    cached, new = spread(g, c["min_cached"], c["cached"]), spread(fixed, c["min_new"], c["new"])
    new[0] = c["new"]
    if c["min_new"] == 0 and c["B"] > 2:
        new[1], new[2] = 0, 1     # a sequence that adds nothing, and one that decodes
    order = torch.randperm(c["B"], generator=g)
    new, cached[order.argmin()] = new[order], c["cached"]
    if c["min_cached"] == 0 and c["B"] > 3:
        cached[order.argmax()] = 0     # a prompt from its first token
    return cached.tolist(), new.tolist()


def _prepare_chunk(c, g, seed):
    B, kvh, hd, blk = c["B"], c["kv_heads"], c["head_dim"], c["block"]
    cached, new = _chunk_lengths(c, seed)
    lens = [a + b for a, b in zip(cached, new)]
    per = max(1, (max(lens) + blk - 1) // blk)
    # the sequences' pages, scattered over a pool with some to spare
    pages = per * B + 3
    table = torch.randperm(pages, device="cuda", generator=g)[:per * B].view(B, per).to(torch.int32)
    slots = pages * blk

    def cache():
        codes = torch.empty((slots, kvh, hd), dtype=torch.float8_e4m3fn, device="cuda")
        step = max(1, (1 << 28) // (kvh * hd))
        for i in range(0, slots, step):  # (bounded temporaries)
            x = torch.randn((min(step, slots - i), kvh, hd), device="cuda", generator=g, dtype=torch.float32)
            codes[i:i + step] = (x / x.abs().amax(-1, keepdim=True) * 448.0).to(torch.float8_e4m3fn)
        return codes, (2.5 + 1.5 * torch.rand((slots, kvh), device="cuda", generator=g)) / 448.0

    kc, ks = cache()
    vc, vs = cache()
    M, q_dim = sum(new), c["q_heads"] * hd
    q = torch.randn((max(M, 1), q_dim), device="cuda", generator=g).mul_(1.5).to(torch.bfloat16)[:M]
    cu = torch.tensor([0] + new, dtype=torch.int64).cumsum(0).to(torch.int32).cuda()
    s = dict(c=c, q=q, kc=kc, ks=ks, vc=vc, vs=vs, table=table, cached=cached, new=new, cu=cu, scale=hd ** -0.5,
             lens=torch.tensor(lens, dtype=torch.int32).cuda())
    if own:
        import w8a8_precision_gemm_gb300 as pkg
        s["ws"] = pkg.kv_attn_chunk_workspace(c["q_heads"], kvh, hd)
    return s


def _prepare_pages(c, g, seed):
    B, blk = c["B"], c["block"]
    r = torch.rand((3, B), device="cuda", generator=g)
    held = 1 + (r[0] * c["cached"]).floor().clamp_(max=c["cached"] - 1)   # tokens that each request holds
    new = c["min_new"] + (r[1] * (c["new"] - c["min_new"] + 1)).floor().clamp_(max=c["new"] - c["min_new"])
    done = r[2] < c["finished"]
    held, new = held.to(torch.int32), torch.where(done, 0.0, new).to(torch.int32)
    per = (c["cached"] + c["new"] + blk - 1) // blk
    blocks = (held.long() + blk - 1) // blk
    pages = per * B + 5
    order = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)
    # the requests hold the last pages of a random order, the list of free ones is the rest
    table = torch.full((B, per), -1, dtype=torch.int32, device="cuda")
    has = torch.arange(per, device="cuda")[None] < blocks[:, None]
    used = has.sum()
    table[has] = order[pages - int(used):]
    free = order.clone()
    cached = torch.where(done, 0, held).to(torch.int32)
    M = B * c["new"]                                                       # rows of a step of fixed size
    return dict(c=c, held=held, cached=cached, new=new, table=table, free=free, M=M, per=per, pages=pages,
                n_free=(pages - used).to(torch.int32).reshape(1), given=torch.empty(1, dtype=torch.int32, device="cuda"),
                left=torch.empty(1, dtype=torch.int32, device="cuda"))


def _frequencies(c):
    """Radians a position of each pair, and the factor on the rotated values."""
    rot = c["rot"]
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if c["scaling"] == "none":
        return f, 1.0
    if c["scaling"] == "linear":
        return f / 4.0, 1.0
    # slow pairs stretched by 8, fast ones kept, a ramp between (by turns over the length trained on)
    turns = 4096 * f / (2 * math.pi)
    keep = ((turns - 1.0) / 31.0).clamp(0.0, 1.0)
    return f * keep + f / 8.0 * (1 - keep), 1.0 + 0.1 * math.log(8.0)


def _positions(c, g):
    return (torch.rand(c["M"], device="cuda", generator=g, dtype=torch.float64) * c["far"]).to(torch.int32)


def _prepare_cache(c, g, seed):
    M, hd, kvh = c["M"], c["head_dim"], c["kv_heads"]
    cols = (c["q_heads"] + 2 * kvh) * hd
    qkv = torch.randn((M, cols), device="cuda", generator=g)
    qkv[:, torch.randint(0, cols, (max(1, cols // 100),), device="cuda", generator=g)] *= 8.0  # outlier channels
    freq, factor = _frequencies(c)
    slots = 2 * M + 7
    slot = torch.randperm(slots, device="cuda", generator=g)[:M]
    slot = torch.where(torch.rand(M, device="cuda", generator=g) < c["pad"], -1, slot)
    z = lambda *s, dtype=torch.float32: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
    return dict(c=c, qkv=qkv.to(torch.bfloat16), freq=freq.cuda(), factor=factor, pos=_positions(c, g), slot=slot,
                caches=(z(slots, kvh, hd, dtype=torch.float8_e4m3fn), z(slots, kvh),
                        z(slots, kvh, hd, dtype=torch.float8_e4m3fn), z(slots, kvh)))


def _prepare_rope(c, g, seed):
    freq, factor = _frequencies(c)
    x = torch.randn((c["M"], c["heads"] * c["head_dim"]), device="cuda", generator=g)
    return dict(c=c, x=x.to(torch.bfloat16 if c["dtype"] == "bf16" else torch.float32), freq=freq.cuda(), factor=factor,
                pos=_positions(c, g))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return dict(chunk=_prepare_chunk, pages=_prepare_pages, cache=_prepare_cache,
                rope=_prepare_rope)[case["op"]](case, g, seed)


# ---------------------------------------------------------------- one pass

def _plain_chunk(s):
    c, blk, hd = s["c"], s["c"]["block"], s["c"]["head_dim"]
    kvh, hq = c["kv_heads"], c["q_heads"]
    M = s["q"].shape[0]
    out = torch.empty((M, hq * hd), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((M, hq), dtype=torch.float32, device="cuda")
    row = 0
    for b, (cached, new) in enumerate(zip(s["cached"], s["new"])):
        if new == 0:
            continue
        n = cached + new
        j0 = max(0, cached + 1 - c["window"]) if c["window"] else 0
        j = torch.arange(j0, n, device="cuda")
        slot = s["table"][b].long()[j // blk] * blk + j % blk
        k = s["kc"].view(torch.uint8)[slot].view(torch.float8_e4m3fn).float() * s["ks"][slot][..., None]
        v = s["vc"].view(torch.uint8)[slot].view(torch.float8_e4m3fn).float() * s["vs"][slot][..., None]
        k, v = k.permute(1, 2, 0).contiguous(), v.transpose(0, 1).contiguous()   # [kvh, hd, n], [kvh, n, hd]
        step = max(1, min(new, (1 << 29) // (hq * len(j))))
        for i in range(0, new, step):
            m = min(step, new - i)
            q = s["q"][row + i:row + i + m].float().view(m, kvh, -1, hd).permute(1, 2, 0, 3)  # [kvh, group, m, hd]
            x = torch.matmul(q.reshape(kvh, -1, hd), k).view(kvh, hq // kvh, m, -1) * s["scale"]
            at = torch.arange(cached + i, cached + i + m, device="cuda")[:, None]
            seen = j[None] <= at
            if c["window"]:
                seen = seen & (j[None] > at - c["window"])
            x = torch.where(seen, x, NEG)
            top = x.amax(-1, keepdim=True)
            p = torch.exp(x - top)
            del x
            total = p.sum(-1, keepdim=True)
            o = torch.matmul(p.view(kvh, -1, len(j)), v).view(kvh, hq // kvh, m, hd) / total
            out[row + i:row + i + m] = o.permute(2, 0, 1, 3).reshape(m, -1).to(torch.bfloat16)
            lse[row + i:row + i + m] = (top + torch.log(total))[..., 0].permute(2, 0, 1).reshape(m, -1)
        row += new
    return out, lse


def _plain_pages(s):
    c, blk, per, pages, M = s["c"], s["c"]["block"], s["per"], s["pages"], s["M"]
    k = torch.arange(per, device="cuda")[None]
    # the finished requests' pages go onto the list, in the order of requests and blocks
    done = (s["cached"] == 0) & (s["held"] > 0)
    back = (k < ((s["held"].long() + blk - 1) // blk)[:, None]) & done[:, None]
    place = torch.cumsum(back.flatten().long(), 0).view(back.shape) - 1 + s["n_free"].long()
    free = torch.cat([s["free"], s["free"][:1]])                       # (the last place takes what is not put back)
    free = free.scatter(0, torch.where(back, place, pages).flatten(), s["table"].flatten())[:pages]
    n = s["n_free"].long() + back.sum()
    # pages for the new tokens, from the end of the list
    first = (s["cached"].long() + blk - 1) // blk
    last = (s["cached"].long() + s["new"].long() + blk - 1) // blk
    need = last - first
    before = torch.cumsum(need, 0) - need
    take = (k >= first[:, None]) & (k < last[:, None])
    index = n - 1 - (before[:, None] + k - first[:, None])
    table = torch.where(take, free[index.clamp(0, pages - 1)], s["table"])
    cu = torch.zeros(c["B"] + 1, dtype=torch.int64, device="cuda")
    cu[1:] = torch.cumsum(s["new"].long(), 0)
    i = torch.arange(M, device="cuda")
    b = torch.searchsorted(cu[1:], i, right=True).clamp(max=c["B"] - 1)
    inside = i < cu[-1]
    pos = torch.where(inside, s["cached"].long()[b] + i - cu[b], 0)
    slot = torch.where(inside, table[b, (pos // blk).clamp(max=per - 1)].long() * blk + pos % blk, -1)
    return (slot, pos.to(torch.int32), cu.to(torch.int32), s["cached"] + s["new"], table, free,
            (n - need.sum()).to(torch.int32).reshape(1))


def _rotate(x, s, inverse=False):
    """Heads x [M, heads, head_dim] in fp32, their first `rot` values rotated."""
    c = s["c"]
    rot, half = c["rot"], c["rot"] // 2
    angle = s["pos"].double()[:, None] * s["freq"]                   # far positions: 64 bits
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    if inverse:
        sin = -sin
    y = x.clone()
    if c["layout"] == "half":
        a, b = x[..., :half], x[..., half:rot]
        y[..., :half], y[..., half:rot] = (a * cos - b * sin) * s["factor"], (a * sin + b * cos) * s["factor"]
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = (a * cos - b * sin) * s["factor"], (a * sin + b * cos) * s["factor"]
    return y


def _plain_cache(s):
    c = s["c"]
    M, hd, kvh, hq = c["M"], c["head_dim"], c["kv_heads"], c["q_heads"]
    x = s["qkv"].float().view(M, hq + 2 * kvh, hd)
    y = _rotate(x[:, :hq + kvh], s)
    kept = s["slot"] >= 0
    # (a padding token's row goes to a place behind the cache)
    out = []
    for vec, code, scale in ((y[:, hq:], s["caches"][0], s["caches"][1]), (x[:, hq + kvh:], s["caches"][2], s["caches"][3])):
        top = vec.abs().amax(-1)
        sc = torch.where(top == 0, 1.0, top / 448.0)
        q8 = (vec / sc[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
        at = torch.where(kept, s["slot"], len(scale))
        codes = torch.cat([code.view(torch.uint8), code.view(torch.uint8)[:1]]).index_copy(0, at, q8.view(torch.uint8))
        out += [codes[:-1].view(torch.float8_e4m3fn), torch.cat([scale, scale[:1]]).index_copy(0, at, sc)[:-1]]
    return [y[:, :hq].reshape(M, -1).to(torch.bfloat16)] + out


def _plain_rope(s):
    c = s["c"]
    y = _rotate(s["x"].float().view(c["M"], c["heads"], c["head_dim"]), s, c["inverse"])
    return y.view(c["M"], -1).to(s["x"].dtype)


def _own(s):
    import w8a8_precision_gemm_gb300 as q

    c = s["c"]
    if c["op"] == "chunk":
        return q.kv_attn_chunk(s["q"], c["q_heads"], s["kc"], s["ks"], s["vc"], s["vs"], s["table"], c["block"], s["cu"],
                               s["lens"], s["scale"], window=c["window"], want_lse=True, ws=s["ws"])
    if c["op"] == "pages":
        q.kv_release(s["held"], s["table"], c["block"], s["free"], s["n_free"], keep_lens=s["cached"], n_free_out=s["given"])
        slot, pos, cu, lens = q.kv_append(s["cached"], s["new"], s["table"], c["block"], s["free"], s["given"], s["M"],
                                          n_free_out=s["left"])
        return slot, pos, cu, lens, s["table"], s["free"], s["left"]
    layout = q.ROPE_HALF if c["layout"] == "half" else q.ROPE_INTERLEAVED
    if c["op"] == "cache":
        y = q.rope_kv_cache_quant(s["qkv"], c["q_heads"], s["pos"], s["freq"], s["slot"], *s["caches"], layout=layout,
                                  factor=s["factor"])
        return [y, *s["caches"]]
    return q.rope(s["x"], c["heads"], s["pos"], s["freq"], layout=layout, factor=s["factor"], inverse=c["inverse"])


def run(state):
    if own:
        return _own(state)
    return dict(chunk=_plain_chunk, pages=_plain_pages, cache=_plain_cache, rope=_plain_rope)[state["c"]["op"]](state)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c = case
    if c["op"] == "chunk":
        B = c["B"]
        new = (c["new"] + (B - 1) * 0.5 * (c["new"] + c["min_new"])) / B
        cached = (c["cached"] + (B - 1) * 0.5 * (c["cached"] + c["min_cached"])) / B
        seen = cached + 0.5 * (new + 1)                        # tokens a query sees
        read = cached + new                                    # tokens a sequence's queries see between them
        if c["window"]:
            seen, read = min(seen, c["window"]), min(read, c["window"] + new)
        rows = B * new * c["q_heads"]
        return {"bytes": B * read * c["kv_heads"] * 2 * (c["head_dim"] + 4) + rows * (4 * c["head_dim"] + 4)
                + 4 * B * read / c["block"], "flops": 4 * rows * seen * c["head_dim"]}
    if c["op"] == "pages":
        B = c["B"]
        tokens = B * (1 - c["finished"]) * 0.5 * (c["new"] + c["min_new"])
        pages = tokens / c["block"] + B * c["finished"] * 0.5 * c["cached"] / c["block"]
        return {"bytes": 12 * B * c["new"] + 8 * pages + 24 * B, "flops": 8 * tokens}
    if c["op"] == "cache":
        q, kv = c["q_heads"] * c["head_dim"], c["kv_heads"] * c["head_dim"]
        return {"bytes": c["M"] * (2 * (q + 2 * kv) + 2 * q + (1 - c["pad"]) * (2 * kv + 8 * c["kv_heads"]) + 12),
                "flops": c["M"] * (4 * (q + kv) * c["rot"] / c["head_dim"] + 6 * kv)}
    n = c["M"] * c["heads"] * c["head_dim"]
    return {"bytes": 2 * n * (2 if c["dtype"] == "bf16" else 4) + 4 * c["M"],
            "flops": 4 * n * c["rot"] / c["head_dim"]}


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_chunk(s):
    c, blk, hd, kvh = s["c"], s["c"]["block"], s["c"]["head_dim"], s["c"]["kv_heads"]
    group = c["q_heads"] // kvh
    M = s["q"].shape[0]
    out = torch.zeros((M, kvh, group, hd), dtype=torch.float64, device="cuda")
    lse = torch.full((M, kvh, group), NEG, dtype=torch.float64, device="cuda")
    q = s["q"].double().view(M, kvh, group, hd)
    for b in range(c["B"]):
        r0, n = int(s["cu"][b]), int(s["lens"][b])
        new = int(s["cu"][b + 1]) - r0
        if new == 0:
            continue
        at = torch.arange(n, device="cuda")
        slot = s["table"][b].long().index_select(0, torch.div(at, blk, rounding_mode="floor")) * blk + at.remainder(blk)
        for h in range(kvh):
            def values(codes, scale):
                v = codes[:, h].view(torch.uint8).index_select(0, slot).view(torch.float8_e4m3fn).double()
                return v * scale[:, h].index_select(0, slot).double()[:, None]
            k, v = values(s["kc"], s["ks"]), values(s["vc"], s["vs"])
            step = max(1, min(new, (1 << 28) // (group * n)))
            for i in range(0, new, step):
                here = torch.arange(i, min(i + step, new), device="cuda")
                pos = n - new + here
                first = max(0, n - new + i + 1 - c["window"]) if c["window"] else 0
                stop = int(n - new + min(i + step, new))            # no query of the piece sees what lies behind
                w = at[first:stop]
                hide = w[None] > pos[:, None]
                if c["window"]:
                    hide = hide | (w[None] <= pos[:, None] - c["window"])
                x = torch.einsum("mgd,ld->gml", q[r0 + here, h], k[first:stop]) * s["scale"]
                x = x.masked_fill(hide, NEG)
                lse[r0 + here, h] = torch.logsumexp(x, -1).T
                out[r0 + here, h] = torch.einsum("gml,ld->mgd", torch.softmax(x, -1), v[first:stop])
    return out.view(M, -1), lse.view(M, -1)


def _exact_pages(s):
    c, blk = s["c"], s["c"]["block"]
    held, cached, new = s["held"].tolist(), s["cached"].tolist(), s["new"].tolist()
    table, free, n = s["table"].tolist(), s["free"].tolist(), int(s["n_free"])
    for b in range(c["B"]):
        for k in range(-(-cached[b] // blk), -(-held[b] // blk)):
            free[n] = table[b][k]
            n += 1
    slot, pos, cu = [], [], [0]
    for b in range(c["B"]):
        for p in range(cached[b], cached[b] + new[b]):
            if p % blk == 0:
                n -= 1
                table[b][p // blk] = free[n]
            slot.append(table[b][p // blk] * blk + p % blk)
            pos.append(p)
        cu.append(len(slot))
    rest = s["M"] - len(slot)
    whole = lambda v: torch.tensor(v, dtype=torch.int64)  # noqa: E731
    return (whole(slot + [-1] * rest), whole(pos + [0] * rest), whole(cu), whole([a + b for a, b in zip(cached, new)]),
            whole(table), whole(free), whole([n]))


def _exact_turn(x, s, sign):
    """Complex numbers turned by position times frequency."""
    c, rot = s["c"], s["c"]["rot"]
    turn = torch.polar(torch.full_like(s["freq"], s["factor"])[None].expand(c["M"], -1).contiguous(),
                       sign * torch.outer(s["pos"].double(), s["freq"]))[:, None]
    part = x[..., :rot].unflatten(-1, (2, rot // 2) if c["layout"] == "half" else (rot // 2, 2))
    dim = -2 if c["layout"] == "half" else -1
    z = torch.complex(part.select(dim, 0), part.select(dim, 1)) * turn
    return torch.cat([torch.stack([z.real, z.imag], dim).flatten(-2), x[..., rot:]], -1)


def _exact_cache(s):
    c = s["c"]
    hq, kvh = c["q_heads"], c["kv_heads"]
    x = s["qkv"].double().view(c["M"], -1, c["head_dim"])
    turned = _exact_turn(x[:, :hq + kvh], s, 1.0)
    rows = (s["slot"] >= 0).nonzero()[:, 0]
    out = [turned[:, :hq].flatten(1)]
    for vec, code, scale in ((turned[:, hq:], *s["caches"][:2]), (x[:, hq + kvh:], *s["caches"][2:])):
        step = vec.abs().amax(-1) / 448.0
        step = torch.where(step == 0, 1.0, step)
        values, steps = code.double(), scale.double()      # (before the rounding to 8 bits)
        values[s["slot"][rows]], steps[s["slot"][rows]] = (vec / step[..., None])[rows], step[rows]
        out += [values, steps]
    return out


def _exact_rope(s):
    c = s["c"]
    x = s["x"].double().view(c["M"], c["heads"], c["head_dim"])
    return _exact_turn(x, s, -1.0 if c["inverse"] else 1.0).flatten(1)


def exact(case, seed):
    if case["op"] == "chunk":
        w = work(case)
        if w["flops"] > 6e12 or case["B"] * case["kv_heads"] > 600:
            return None
    if case["op"] == "pages" and case["B"] * (case["cached"] + case["new"]) / case["block"] > 8e6:
        return None
    s = prepare(case, seed)
    return dict(chunk=_exact_chunk, pages=_exact_pages, cache=_exact_cache, rope=_exact_rope)[case["op"]](s)
