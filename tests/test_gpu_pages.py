"""Pages handed out and taken back on the GPU (qurl_kv_append, qurl_kv_release)
against the rules written as a loop on the host; whole numbers, so all are equal."""
import random

import pytest
import torch

import w8a8_precision_gemm_gb300 as q

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _status():
    yield
    q.qurl_check_device_status()


def i4(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def append(cached, new, table, block, free, n, M):
    """What qurl_kv_append gives: (slots, positions, cu, lens, table, n left)."""
    n, rows, room = max(n, 0), 0, len(table[0]) * block if table else 0
    table = [list(r) for r in table]
    slots, pos, cu, lens, taken = [], [], [0], [], 0
    for b, (c, k) in enumerate(zip(cached, new)):
        c = min(max(c, 0), room)
        k = min(max(k, 0), room - c, M - rows)
        for p in range(c, c + k):
            if p % block == 0:
                table[b][p // block] = free[n - 1 - taken] if taken < n else -1
                taken += 1
            page = table[b][p // block]
            slots.append(page * block + p % block if page >= 0 else -1)
            pos.append(p)
        rows += k
        cu.append(rows)
        lens.append(c + k)
    rest = M - rows
    return slots + [-1] * rest, pos + [0] * rest, cu, lens, table, n - taken


def release(lens, keep, table, block, free, n):
    n, free, room = max(n, 0), list(free), len(table[0]) * block if table else 0
    for b, t in enumerate(lens):
        t, k = min(max(t, 0), room), max(keep[b], 0) if keep else 0
        for page in table[b][-(-k // block):-(-t // block)]:
            if page >= 0:
                if n < len(free):
                    free[n] = page
                n += 1
    return free, min(n, len(free))


def random_case(seed, B, block, most, new):
    r = random.Random(seed)
    per = -(-(most + new) // block)
    cached, fresh = [r.randint(0, most) for _ in range(B)], [r.randint(0, new) for _ in range(B)]
    pages = per * B + 2
    order = list(range(pages))
    r.shuffle(order)
    table = [[order.pop() if k < -(-c // block) else -5 for k in range(per)] for c in cached]
    return cached, fresh, table, order + [0] * (pages - len(order)), len(order)


def run_append(cached, new, table, block, free, n, M):
    t, nf = i4(table).view(len(cached), -1), i4([n])
    out = q.kv_append(i4(cached), i4(new), t, block, i4(free), nf, M)
    return [v.tolist() for v in out] + [t.tolist(), int(nf)]


@pytest.mark.parametrize("B,block,most,new", [
    (1, 16, 0, 1), (1, 16, 40, 300), (3, 1, 10, 5), (7, 7, 100, 33), (64, 16, 2000, 1), (64, 24, 500, 64), (5, 128, 4000, 900),
    (300, 16, 90, 4), (1023, 3, 20, 2), (1024, 16, 100, 1), (1025, 16, 30, 3), (2500, 5, 12, 2), (16384, 16, 20, 1),
    (1, 1000, 5000, 5000), (2, 16, 100, 40000),
])
def test_append(B, block, most, new):
    c = random_case(B * block, B, block, most, new)
    cached, fresh, table, free, n = c
    total = sum(fresh)
    for M in {total, total + 77}:
        got = run_append(cached, fresh, table, block, free, n, M)
        assert got == list(append(cached, fresh, table, block, free, n, M))


@pytest.mark.parametrize("B,block,most", [(1, 16, 300), (3, 1, 10), (7, 7, 100), (64, 16, 2000), (5, 128, 40000), (300, 16, 90),
                                          (1025, 16, 300), (16384, 16, 20)])
def test_release(B, block, most):
    r = random.Random(B)
    cached, _, table, free, n = random_case(B + block, B, block, most, 1)
    free = free[:n] + [-9] * (len(free) - n)
    for keep in (None, cached, [r.choice([0, c, r.randint(0, c + 5), -3]) for c in cached]):
        t, f, nf = i4(table).view(B, -1), i4(free), i4([n])
        q.kv_release(i4(cached), t, block, f, nf, keep_lens=None if keep is None else i4(keep))
        want = release(cached, keep, table, block, free, n)
        assert (f.tolist(), int(nf)) == want
        assert t.tolist() == table


def test_pages_without_an_entry_are_not_given_back():
    table = [[4, -1, 6, -1], [-1, -1, -1, -1], [0, 1, 2, 3]]
    f, n = i4([9, 8, 0, 0, 0, 0, 0, 0, 0]), i4([2])
    q.kv_release(i4([64, 64, 50]), i4(table), 16, f, n)
    assert f.tolist() == [9, 8, 4, 6, 0, 1, 2, 3, 0] and int(n) == 8


def test_a_list_that_runs_out():
    """The last pages are missing: -1 in the table, slots of -1, minus their number left; a list that was short
    before counts as empty."""
    for n in (3, 0, -2):
        cached, new, table, free = [15, 0, 30], [20, 40, 3], [[7, -5, -5], [-5] * 3, [8, 9, -5]], [1, 2, 3, 0, 0, 0]
        want = append(cached, new, table, 16, free, n, 70)
        assert run_append(cached, new, table, 16, free, n, 70) == list(want)
        assert want[-1] == max(n, 0) - 6
    f, n = i4([5, 5, 5]), i4([-4])
    q.kv_release(i4([10]), i4([[2]]), 16, f, n)
    assert f.tolist() == [2, 5, 5] and int(n) == 1


def test_lengths_out_of_range_are_cut_and_reported():
    free = list(range(20))
    for cached, new, M in (([100, 3], [1, 1], 4), ([40, 3], [20, 1], 30), ([3, 3], [5, 9], 10), ([3, -7], [2 ** 31 - 1, 2 ** 31 - 1], 60)):
        table = [[30, 31, 32], [33, 34, 35]]
        got = run_append(cached, new, table, 16, free, 20, M)
        with pytest.raises(q.QurlError) as e:
            q.qurl_check_device_status()
        assert e.value.status == 1
        assert got == list(append(cached, new, table, 16, free, 20, M))
    # more free pages than the list has places
    got = run_append([0], [20], [[-5, -5]], 16, free, 99, 20)
    with pytest.raises(q.QurlError):
        q.qurl_check_device_status()
    assert got == list(append([0], [20], [[-5, -5]], 16, free, 20, 20))
    # more pages given back than there are places; a length past the table
    for lens, places in (([32, 32], 5), ([33, 10], 8)):
        f, n = i4([1] * places), i4([2])
        q.kv_release(i4(lens), i4([[6, 7], [8, 9]]), 16, f, n)
        with pytest.raises(q.QurlError):
            q.qurl_check_device_status()
        assert (f.tolist(), int(n)) == release(lens, None, [[6, 7], [8, 9]], 16, [1] * places, 2)


def test_nothing_to_do():
    e = torch.empty((0, 4), dtype=torch.int32, device="cuda")
    n = i4([3])
    slots, pos, cu, lens = q.kv_append(i4([]), i4([]), e, 16, i4([1, 2, 3]), n, 5)
    assert slots.tolist() == [-1] * 5 and pos.tolist() == [0] * 5 and cu.tolist() == [0] and lens.numel() == 0 and int(n) == 3
    q.kv_release(i4([]), e, 16, i4([1, 2, 3]), n)
    assert int(n) == 3
    slots, _, cu, lens = q.kv_append(i4([5, 0]), i4([0, 0]), i4([[1], [-1]]), 16, i4([2]), i4([1]), 0)
    assert slots.numel() == 0 and cu.tolist() == [0, 0, 0] and lens.tolist() == [5, 0]


def test_table_rows_side_by_side():
    """A table that is a slice of a wider one: what lies beside it stays."""
    wide = torch.full((3, 9), -5, dtype=torch.int32, device="cuda")
    n = i4([8])
    q.kv_append(i4([0, 0, 0]), i4([40, 48, 1]), wide[:, 2:5], 16, i4(list(range(8))), n, 89)
    assert wide[:, 2:5].tolist() == [[7, 6, 5], [4, 3, 2], [1, -5, -5]]
    assert bool((wide[:, :2] == -5).all()) and bool((wide[:, 5:] == -5).all()) and int(n) == 1


def test_steps_of_a_batch_in_a_graph():
    """A batch grows, finishes and starts again for many steps, its lengths and its list updated in place, from one
    captured step and eagerly; no page is ever in two places, and a released list is whole."""
    B, block, per, M, pages = 37, 16, 12, 260, 300
    for captured in (False, True):
        r = random.Random(5)
        free, n = q.kv_pages(pages)
        assert free.tolist()[::-1] == list(range(pages)) and int(n) == pages
        table = torch.full((B, per), -1, dtype=torch.int32, device="cuda")
        lens, new, held = i4([0] * B), i4([0] * B), i4([0] * B)
        slots = torch.empty(M, dtype=torch.int64, device="cuda")
        pos, cu = torch.empty(M, dtype=torch.int32, device="cuda"), torch.empty(B + 1, dtype=torch.int32, device="cuda")
        host = dict(lens=[0] * B, table=table.tolist(), free=free.tolist(), n=pages)

        def step():
            q.qurl_kv_release(held, table, block, free, n, n, keep_lens=lens)
            q.qurl_kv_append(lens, new, table, block, free, n, n, slots, pos, cu, lens)

        graph = None
        for t in range(30):
            done = [r.random() < 0.1 for _ in range(B)]
            now = [0 if d else c for d, c in zip(done, host["lens"])]
            add = [min(r.choice([1, 1, 1, 0, 9, 31]), per * block - c) for c in now]
            while sum(add) > M:
                add[add.index(max(add))] = 1
            held.copy_(i4(host["lens"]))
            lens.copy_(i4(now))
            new.copy_(i4(add))
            if captured and t == 1:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    step()
            step() if graph is None else graph.replay()
            host["free"], host["n"] = release(host["lens"], now, host["table"], block, host["free"], host["n"])
            s, p, c, l, tb, left = append(now, add, host["table"], block, host["free"], host["n"], M)
            assert (slots.tolist(), pos.tolist(), cu.tolist(), lens.tolist(), table.tolist(), int(n)) == (s, p, c, l, tb, left)
            host.update(lens=l, table=tb, n=left)
            used = [tb[b][k] for b in range(B) for k in range(-(-l[b] // block))]
            assert sorted(used + free.tolist()[:left]) == list(range(pages))


def test_another_stream():
    cached, fresh, table, free, n = random_case(3, 50, 16, 300, 9)
    want = append(cached, fresh, table, 16, free, n, 500)
    t, nf, s = i4(table), i4([n]), torch.cuda.Stream()
    args = i4(cached), i4(fresh), t, 16, i4(free), nf, 500
    s.wait_stream(torch.cuda.current_stream())
    out = q.kv_append(*args, stream=s)
    q.kv_release(out[3], t, 16, args[4], nf, stream=s)
    s.synchronize()
    assert [v.tolist() for v in out] + [t.tolist()] == list(want[:5])
    assert int(nf) == n + sum(-(-c // 16) for c in cached)


@pytest.mark.parametrize("M", [3000, 7000, 15000, 30000])
def test_counts_and_lengths_in_place_by_several_ctas(M):
    """The number of free pages and the lengths are read and written by all CTAs of a call at the same place: every step of a
    growing batch, as many times over, takes the pages and the places that the rules say."""
    r, B, block, per, pages = random.Random(M), 400, 8, 24, 400 * 24
    lens, new = [r.randint(0, 30) for _ in range(B)], None
    order = list(range(pages))
    r.shuffle(order)
    table = [[order.pop() if k < -(-c // block) else -5 for k in range(per)] for c in lens]
    free, n = order + [0] * (pages - len(order)), len(order)
    for _ in range(4):
        new = [r.randint(0, 30) for _ in range(B)]
        new = [min(v, M // B) for v in new]
        want = append(lens, new, table, block, free, n, M)
        for _ in range(5):
            t, nf, l, f = i4(table), i4([n]), i4(lens), i4(free)
            slots = torch.full((M,), 7, dtype=torch.int64, device="cuda")
            pos, cu = i4([7] * M), i4([7] * (B + 1))
            q.qurl_kv_append(l, i4(new), t, block, f, nf, nf, slots, pos, cu, l)
            assert [v.tolist() for v in (slots, pos, cu, l, t)] + [int(nf)] == list(want)
        lens, table, n = want[3], want[4], want[5]


def test_as_many_rows_as_an_int_counts():
    """A step padded to 2^31 - 1 rows: the tokens in front, padding up to the last row."""
    M, t, n = 2 ** 31 - 1, i4([[5, -5], [-5, -5]]), i4([3])
    slots, pos, cu, lens = q.kv_append(i4([10, 0]), i4([9, 2]), t, 16, i4([2, 8, 4]), n, M)
    assert slots[:12].tolist() == [90, 91, 92, 93, 94, 95, 64, 65, 66, 128, 129, -1]
    assert pos[:12].tolist() == [10, 11, 12, 13, 14, 15, 16, 17, 18, 0, 1, 0]
    assert bool((slots[11:] == -1).all()) and bool((pos[11:] == 0).all())
    assert cu.tolist() == [0, 9, 11] and lens.tolist() == [19, 2] and t.tolist() == [[5, 4], [8, -5]] and int(n) == 1
