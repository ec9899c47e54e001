"""The operators between the qkv linear and the output projection as a rollout runs them: pages taken for the new tokens
(qurl_kv_append), rotation and quantization into them (qurl_rope_kv_cache_quant), attention over them
(qurl_kv_attn_chunk, qurl_kv_attn_decode for single tokens), pages given back (qurl_kv_release).

Bounds.  Queries: the rotation in fp32 is off by less than 2^-20 of the pair's size, then half a step of bf16.
Cached keys: the same, then half a step of e4m3 (2^-4 of the value; 2^-10 of the head's step where that is more), the step
itself rounded to fp32.  Values: the latter alone.  Attention: the bounds beside its own tests, on the cache's codes.
Whole numbers and repeated runs: equal."""
import pytest
import torch

import w8a8_precision_gemm_gb300 as q
from test_gpu_attn_chunk import check, reference
from test_gpu_pages import append, i4, release

pytestmark = pytest.mark.gpu

HQ, HK, HD, BLOCK = 10, 2, 128, 16


@pytest.fixture(autouse=True)
def _status():
    yield
    q.qurl_check_device_status()


class Engine:
    """State of a batch of B requests: pages of a shared pool, what is cached."""

    def __init__(self, B=6, most=400, pages=90, seed=0):
        self.per = -(-most // BLOCK)
        slots = pages * BLOCK
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        byte = lambda: torch.randint(0, 120, (slots, HK, HD), device="cuda", generator=g, dtype=torch.uint8)  # noqa: E731
        self.caches = [byte(), torch.full((slots, HK), 0.01, device="cuda"), byte(), torch.full((slots, HK), 0.01, device="cuda")]
        self.free, self.n = q.kv_pages(pages)
        self.table = torch.zeros((B, self.per), dtype=torch.int32, device="cuda")
        self.cached = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.freq, self.factor = q.rope_frequencies(HD, scaling="yarn", factor=4.0, original_len=1024)
        self.ws = q.kv_attn_chunk_workspace(HQ, HK, HD)
        self.state = [self.free, self.n, self.table, self.cached, *self.caches]

    def step(self, new, qkv, keep=None, stream=None):
        """One step; keep: tokens that each request keeps at its end (all of them otherwise)."""
        slots, pos, cu, lens = q.kv_append(self.cached, new, self.table, BLOCK, self.free, self.n, qkv.shape[0], stream=stream)
        x = q.rope_kv_cache_quant(qkv, HQ, pos, self.freq, slots, *self.caches, factor=self.factor, stream=stream)
        out, lse = q.kv_attn_chunk(x, HQ, *self.caches, self.table, BLOCK, cu, lens, want_lse=True, ws=self.ws, stream=stream)
        left = lens if keep is None else torch.minimum(lens, keep)
        q.kv_release(lens, self.table, BLOCK, self.free, self.n, keep_lens=left, stream=stream)
        self.cached.copy_(left)
        return slots, pos, cu, lens, x, out, lse


def rows(M, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn((M, (HQ + 2 * HK) * HD), device="cuda", generator=g).to(torch.bfloat16)


def turned(x, pos, freq, factor):
    """Rows of heads in 64 bits, halves as pairs."""
    t = pos.double()[:, None, None] * freq
    a, b = x.double().chunk(2, -1)
    return torch.cat([a * t.cos() - b * t.sin(), a * t.sin() + b * t.cos()], -1) * factor


STEPS = [  # (new tokens, tokens kept at the end, rows behind the last)
    ([70, 1, 0, 33, 128, 300], None, 0),                       # prompts, one request idle
    ([1, 1, 17, 5, 4, 1], [71, 0, 17, 35, 132, 301], 3),       # single tokens, drafts of which some are dropped, one finished
    ([1, 200, 0, 1, 1, 90], [72, 200, 0, 36, 0, 0], 13),       # a prompt in the place of the finished one, three more end
    ([1, 1, 1, 1, 1, 1], None, 0),                             # single tokens
]


def test_steps_of_a_batch():
    e, host = Engine(), None
    for i, (new, keep, pad) in enumerate(STEPS):
        M, before = sum(new) + pad, [t.clone() for t in e.state]
        cached, table = before[3].tolist(), before[2].tolist()
        qkv = rows(M, i)
        slots, pos, cu, lens, x, out, lse = e.step(i4(new), qkv, None if keep is None else i4(keep))
        # pages, against the rules on the host
        want = append(cached, new, table, BLOCK, before[0].tolist(), int(before[1]), M)
        left = keep or want[3]
        free, n = release(want[3], left, want[4], BLOCK, before[0].tolist(), want[5])
        assert slots.tolist() == want[0] and pos.tolist() == want[1] and cu.tolist() == want[2] and lens.tolist() == want[3]
        assert int(e.n) == n and e.free.tolist()[:n] == free[:n] and e.cached.tolist() == left
        # queries, keys and values
        there = slots >= 0
        h = qkv.view(M, -1, HD)
        want_q = turned(h[:, :HQ], pos, e.freq, e.factor)
        size = (h[:, :HQ].double().abs() + h[:, :HQ].double().abs().roll(HD // 2, -1)) * e.factor
        d = (x.view(M, HQ, HD).double() - want_q).abs()
        assert bool(d.le(want_q.abs() * 2.0 ** -8 + size * 2.0 ** -19).all())
        keys, values = turned(h[:, HQ:HQ + HK], pos, e.freq, e.factor)[there], h[:, HQ + HK:].double()[there]
        for exact, codes, steps in ((keys, e.caches[0], e.caches[1]), (values, e.caches[2], e.caches[3])):
            step = steps[slots[there]].double()
            got = codes[slots[there]].view(torch.float8_e4m3fn).double() * step[..., None]
            err = exact.abs() * (2.0 ** -4 + 2.0 ** -18) + step[..., None] * (2.0 ** -10 + 448 * 2.0 ** -18)
            assert bool((got - exact).abs().le(err).all())
        other = torch.ones(len(e.caches[1]), dtype=torch.bool, device="cuda")
        other[slots[there]] = False
        for now, then in zip(e.caches, before[4:]):
            assert torch.equal(now[other], then[other])
        # attention
        a = dict(q=x, q_heads=HQ, k=e.caches[0].view(torch.float8_e4m3fn), ks=e.caches[1], v=e.caches[2].view(torch.float8_e4m3fn),
                 vs=e.caches[3], table=torch.tensor(want[4], dtype=torch.int32, device="cuda"), block=BLOCK, cu=cu, lens=lens,
                 scale=HD ** -0.5, window=0)
        check(a, (out, lse))
    # the last step's tokens are single: the attention of one token, to both kernels' bounds
    one, l1 = q.kv_attn_decode(x, HQ, *e.caches, e.table, BLOCK, lens, want_lse=True)
    _, _, to, tl = reference(a)
    assert bool((one.double() - out.double()).abs().le(2 * to).all()) and bool((l1 - lse).abs().le(2 * tl).all())


def test_a_captured_step_and_one_on_another_stream():
    """The same steps eager, replayed and on a stream of their own: the same bits, state included."""
    B = 6
    plan = [([40, 3, 0, 17, 25, 1], [400] * 6), ([1, 1, 30, 4, 1, 1], [41, 0, 30, 19, 400, 400]), ([1, 38, 1, 1, 1, 1], [400] * 6)]
    M = 128  # (rows behind the last sequence's in every step)
    eager, graph, side = Engine(), Engine(), Engine()
    new, keep, qkv = i4([0] * B), i4([0] * B), rows(M, 9)
    graph.step(new, qkv, keep)  # (workspaces and the library, before the capture)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            res = graph.step(new, qkv, keep)
    torch.cuda.current_stream().wait_stream(s)
    for i, (n, k) in enumerate(plan):
        x = rows(M, 20 + i)
        want = eager.step(i4(n), x, i4(k))
        t = torch.cuda.Stream()
        t.wait_stream(torch.cuda.current_stream())
        n_t, k_t = i4(n), i4(k)
        torch.cuda.synchronize()
        with torch.cuda.stream(t):
            got = side.step(n_t, x, k_t)
        new.copy_(i4(n)), keep.copy_(i4(k)), qkv.copy_(x)
        g.replay()
        torch.cuda.synchronize()
        rows_used = int(want[2][-1])
        for a, b, c in zip(want, got, res):
            part = slice(0, rows_used) if a.shape[0] == M else slice(None)
            assert torch.equal(a[part], b[part]) and torch.equal(a[part], c[part])
        for a, b, c in zip(eager.state, side.state, graph.state):
            assert torch.equal(a, b) and torch.equal(a, c)


def test_two_batches_at_once():
    """Two engines on two streams, each with its workspace, in flight together: as one behind the other."""
    plan = [([250, 1, 100, 33, 7, 300], None), ([1, 1, 1, 1, 1, 1], None), ([4, 4, 4, 4, 4, 4], None)]
    xs = [[rows(sum(n), 50 + 10 * b + i) for i, (n, _) in enumerate(plan)] for b in range(2)]
    news = [i4(n) for n, _ in plan]
    alone = [Engine(pages=100, seed=b) for b in range(2)]
    want = [[alone[b].step(news[i], xs[b][i])[5] for i in range(len(plan))] for b in range(2)]
    both = [Engine(pages=100, seed=b) for b in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for i in range(len(plan)):
        for b in range(2):
            with torch.cuda.stream(streams[b]):
                got[b].append(both[b].step(news[i], xs[b][i])[5])
    torch.cuda.synchronize()
    for b in range(2):
        for x, y in zip(want[b], got[b]):
            assert torch.equal(x, y)
        for x, y in zip(alone[b].state, both[b].state):
            assert torch.equal(x, y)


def test_stream_argument():
    """What a call with stream= allocates and launches belongs to that stream: the caller's stream is not waited for, and
    its results are there once the stream is through."""
    e, s = Engine(), torch.cuda.Stream()
    x, new = rows(60, 3), i4([10, 20, 0, 30, 0, 0])
    want = Engine().step(new, x)
    torch.cuda.synchronize()
    slots, pos, cu, lens = q.kv_append(e.cached, new, e.table, BLOCK, e.free, e.n, 60, stream=s)
    y = q.rope_kv_cache_quant(x, HQ, pos, e.freq, slots, *e.caches, factor=e.factor, stream=s)
    out, lse = q.kv_attn_chunk(y, HQ, *e.caches, e.table, BLOCK, cu, lens, want_lse=True, stream=s)  # (its own workspace)
    back = q.rope(y, HQ, pos, e.freq, factor=1 / e.factor, inverse=True, stream=s)
    s.synchronize()
    for a, b in zip((slots, pos, cu, lens, y, out, lse), want):
        assert torch.equal(a, b)
    # (there and back: half a step of both turned values, together 2^-8 of the pair's length, and half a step of the result)
    d = (back.double() - x[:, :HQ * HD].double()).abs()
    h = x[:, :HQ * HD].double().view(60, HQ, HD).abs()
    size = (h + h.roll(HD // 2, -1)).view(60, -1)
    assert bool(d.le(size * 2.0 ** -7 * (1 + 2.0 ** -6)).all())
