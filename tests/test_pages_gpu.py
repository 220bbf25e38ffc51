"""Pages shared, given out, taken back and brought together, against a plain model of the pool: everything is whole numbers
and has to be equal."""
import random

import pytest
import torch

import lossless_float_compression_amd as zx
from pages_util import Device, Model, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", (16, 64, 4096))
@pytest.mark.parametrize("groups,K", [(1, 1), (1, 4), (3, 5), (40, 8), (2, 64), (1, 100)])
def test_a_search(T, groups, K):
    """Steps of a beam search from a prompt on: every state after every call."""
    r = random.Random(T * K + groups)
    n, steps = groups * K, 12
    W = 8 + -(-(steps * T) // T)
    m = Model(n * (W + 3) + 50, T, n, W, seed=K)
    d = Device(m.fill([r.randint(1, 4 * T) if i % K == 0 else 0 for i in range(n)]))
    d.same()
    d.fork([0] * n, K)                           # all beams go on from the prompt
    for i in range(steps):
        d.extend([r.choice((1, 1, 1, 2, T // 2, 0))] * n)
        parents = [r.randrange(K) for _ in range(n)] if i % 4 else [r.choice((-1, 0, K - 1, r.randrange(K))) for _ in range(n)]
        d.fork(parents, K)
        if i % 5 == 4:
            d.trim([max(0, h - r.randint(0, T + 2)) for h in m.held])
        if i % 6 == 5:
            d.compact()
        assert sum(x for x in m.refs if x > 0) == sum(m.pages(s) for s in range(n))
    d.trim(None)
    assert not any(m.refs) and not any(m.held)


@pytest.mark.parametrize("seed", range(12))
def test_any_calls(seed):
    """Calls in any order on rows of any lengths, in pools that are nearly full."""
    r = random.Random(seed)
    T, K, groups = r.choice((16, 32, 128)), r.choice((1, 2, 3, 7, 16)), r.randint(1, 20)
    n, W = groups * K, r.randint(2, 40)
    m = Model(r.randint(n, 4 * n + 40), T, n, W, seed=seed)
    total = []
    for _ in range(n):
        t = r.choice((0, 1, T, r.randint(0, W * T)))
        total.append(t if sum(-(-x // T) for x in total) + -(-t // T) <= m.n else 0)
    d = Device(m.fill(total))
    for _ in range(25):
        what = r.choice(("fork", "fork", "extend", "extend", "extend", "trim", "compact"))
        if what == "fork":
            d.fork([r.choice((r.randrange(K), r.randrange(K), -1)) for _ in range(n)], K)
        elif what == "extend":
            new = [r.choice((0, 1, 1, 2, T, r.randint(0, 3 * T))) for _ in range(n)]
            d.extend(new, err=4 if any(h + q > W * T for h, q in zip(m.held, new)) else 0)
        elif what == "trim":
            d.trim([r.choice((0, h, 1 << 30, r.randint(0, max(h, 1)), max(0, h - 1))) for h in m.held])
        else:
            d.compact()


def test_who_keeps_a_page():
    """A shared page with tokens: all that hold it go on (the first keeps it), some do, one does, and it is pinned besides."""
    def state():
        m = Model(40, 16, 4, 5).fill([20, 0, 0, 0])
        d = Device(m)
        d.fork([0, 0, 0, -1], 4)
        return m, d
    m, d = state()
    assert len(d.extend([1, 1, 1, 0])) == 2 and m.table[0][1] not in (m.table[1][1], m.table[2][1])
    m, d = state()
    assert len(d.extend([0, 1, 1, 0])) == 2
    m, d = state()
    assert len(d.extend([0, 0, 1, 0])) == 1
    assert len(d.extend([1, 1, 0, 0])) == 1      # two are left, and both go on
    assert len(d.extend([1, 1, 1, 0])) == 0
    m, d = state()
    m.refs[m.table[0][1]] += 1
    d.pool.refs[m.table[0][1]] += 1
    assert len(d.extend([1, 1, 1, 0])) == 3
    # rows of unequal lengths in one page
    m, d = state()
    d.trim([20, 18, 17, 0])
    c = d.extend([3, 0, 9, 0])
    assert [x[2] for x in c] == [4, 1]
    # rows that end at a page's end share it for good
    m = Model(40, 16, 2, 5).fill([32, 0])
    d = Device(m)
    d.fork([0, 0], 2)
    assert d.extend([1, 1]) == []


def test_too_few_pages():
    """Nothing changes but kv_len, and the call can be made again when pages are free."""
    m = Model(10, 16, 4, 8).fill([33, 48, 0, 15])
    d = Device(m)                                # 7 pages taken, 3 free
    assert d.extend([16, 16, 16, 16]) == []      # 4 wanted
    assert d.extend([16, 0, 16, 16]) == []       # 3
    d.extend([0, 0, 0, 1])                       # none are left, one is wanted
    d.extend([0, 0, 0, 0])
    d.extend([3, 0, 0, 0])                       # room in its page
    d.trim([33, 20, 0, 0])
    d.extend([0, 30, 1, 0])


def test_rows_out_of_range():
    """They are left out and reported, the others are served."""
    def state():
        m = Model(60, 16, 6, 4, seed=2).fill([20, 5, 64, 1, 0, 17])
        return m, Device(m)
    m, d = state()
    d.extend([1, 1, 1, 1, 1, 1], err=4)          # row 2 is full
    d.extend([0, 70, 0, 2, 65, 0], err=4)
    d.extend([0, 2, 0, 9, 1, 0], err=4, max_q=8)
    d.extend([9, 2, 0, 0, 1, 9], err=4, max_kv=22)
    for bad in (-1, -2 ** 31, 65, 2 ** 31 - 1):
        m, d = state()
        m.held[3] = bad
        d.held[3] = bad
        d.extend([1, 1, 0, 1, 1, 1], err=4)
        keep = m.held[3]
        d.trim([9, 1 << 30, 1 << 30, 0, 0, 0], err=4)
        d.fork([1, 0, 2, 1, 0, 2], 3, err=4)     # its group stays
        assert m.held[3] == keep
    m, d = state()
    d.trim([9, -1, 3, -2 ** 31, 0, 0], err=4)
    for bad in (-2, 3, 2 ** 31 - 1, -2 ** 31):
        d.fork([1, 0, 2, 1, bad, 2], 3, err=4)
    # a batch whose q_start falls, or begins below zero
    m, d = state()
    b = zx.PagedBatch(i32([0, 1, 3, 2, 2, 2, 2]), d.kv, d.table)
    d.pool.extend(b, d.held, copies=d.copies, err=d.err)
    assert d.kv.tolist() == [21, 7, 0, 1, 0, 17] and int(d.err) == 4
    m, d = state()
    b = zx.PagedBatch(i32([-2 ** 31, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1, -5, 0, 0]), d.kv, d.table)
    d.pool.extend(b, d.held, copies=d.copies, err=d.err)
    assert d.kv.tolist() == [0, 5, 64, 0, 0, 17] and d.held.tolist() == m.held and int(d.err) == 4


def test_entries_that_are_no_pages():
    m = Model(30, 16, 3, 4, seed=1).fill([40, 20, 33])
    d = Device(m)
    for bad in (-1, 30, 2 ** 31 - 1, -2 ** 31):
        good = m.table[1][1]
        m.table[1][1] = bad
        d.table[1, 1] = bad
        d.extend([0, 1, 1], err=4)               # row 1 cannot go on in it
        before = d.pool.refs.tolist()
        d.pool.fork(d.table, d.held, i32([[2, 1, 2]]), err=d.err)
        d.pool.fork(d.table, d.held, i32([[0, 1, 1]]), err=d.err)
        assert int(d.err) == 4
        d.table.copy_(i32(m.table))
        d.held.copy_(i32(m.held))
        d.pool.refs.copy_(i32(before))
        d.err.zero_()
        d.pool.trim(d.table, d.held, i32([99, 0, 99]), err=d.err)
        assert int(d.err) == 4
        want = list(m.refs)
        want[m.table[1][0]] -= 1
        assert d.pool.refs.tolist() == want and d.held.tolist() == [m.held[0], 0, m.held[2]]
        d.held.copy_(i32(m.held))
        d.pool.refs.copy_(i32(before))
        d.err.zero_()
        d.pool.compact(d.table, d.held, copies=d.copies, err=d.err)
        assert int(d.err) == 4 and int(d.table[1, 1]) == bad
        d.table.copy_(i32(m.table))
        d.pool.refs.copy_(i32(before))
        d.err.zero_()
        d.copies.pairs.fill_(-1)
        m.table[1][1] = good
        d.table[1, 1] = good


def test_counts_that_do_not_add_up():
    """A page given back more often than it is held is reported and free; one that nobody is said to hold is not written to."""
    m = Model(20, 16, 2, 4).fill([40, 20])
    d = Device(m)
    d.pool.refs[m.table[0][2]] = 0
    d.pool.refs[m.table[1][1]] = -3
    d.pool.extend(d.batch([1, 1]), d.held, copies=d.copies, err=d.err)
    assert int(d.err) == 4 and d.kv.tolist() == [0, 0] and d.held.tolist() == [40, 20]
    d.err.zero_()
    d.pool.trim(d.table, d.held, err=d.err)
    assert int(d.err) == 4 and int(d.pool.refs.max()) == 0
    d.err.zero_()
    d.pool.extend(d.batch([16 * 4, 16 * 4]), d.held, copies=d.copies, err=d.err)
    assert int(d.err) == 0 and d.table.tolist() == [[0, 1, 2, 3], [4, 5, 6, 7]]


@pytest.mark.parametrize("n_pages", (1, 2, 4095, 4096, 4097, 70001, 1 << 23))
def test_pools_of_any_size(n_pages):
    """Free pages at both ends and in the middle of the segments that workgroups count."""
    T, n, W = 16, 5, min(n_pages, 3000)
    g = torch.Generator(device="cuda").manual_seed(n_pages)
    refs = (torch.rand(n_pages, generator=g, device="cuda") < 0.7).to(torch.int32)
    refs[-1] = 0
    free = torch.nonzero(refs == 0).view(-1)
    pool = zx.PagePool(n_pages, T, refs=refs.clone())
    total = min(free.numel(), n * W)
    new = [min(W, max(0, total - i * W)) * T for i in range(n)]
    start = i32([sum(new[:i]) for i in range(n + 1)])
    table, held, kv, err = torch.full((n, W), -1, dtype=torch.int32, device="cuda"), i32([0] * n), i32([0] * n), i32([0])
    b = zx.PagedBatch(start, kv, table)
    pool.extend(b, held, err=err)
    assert held.tolist() == new and int(err) == 0
    got = torch.cat([table[i, :x // T] for i, x in enumerate(new)]).long()
    assert torch.equal(got, free[:total])
    assert torch.equal(pool.refs.long(), refs.long().index_fill(0, got, 1))
    if total == free.numel():
        more = zx.PagedBatch(i32([0] * n + [1]), kv, table)
        pool.extend(more, held, err=err)
        assert int(err) in (4, 6) and not kv[-1:].any() and held.tolist() == new
        err.zero_()
    pool.trim(table, held, i32([T] * n), err=err)
    live = (pool.refs > 0)
    L = int(live.sum())
    was = pool.refs.clone()
    copies, remap = pool.compact(table, held, err=err)
    count = int(copies.count)
    pairs = copies.pairs[:count].long()
    src, dst = torch.nonzero(live[L:]).view(-1) + L, torch.nonzero(~live[:L]).view(-1)
    assert count == src.numel() and torch.equal(pairs[:, 0], src) and torch.equal(pairs[:, 1], dst) and bool((pairs[:, 2] == T).all())
    want = torch.where(live, torch.arange(n_pages, device="cuda"), -1)
    want[src] = dst
    assert torch.equal(remap.long(), want)
    assert bool((pool.refs[:L] > 0).all()) and not bool(pool.refs[L:].any()) and torch.equal(pool.refs[want[live]], was[live]) and int(err) == 0


def test_many_rows():
    """2048 rows, as one group and as many; wide tables that several workgroups share."""
    r = random.Random(5)
    m = Model(9000, 16, 2048, 6).fill([r.randint(0, 40) for _ in range(2048)])
    d = Device(m)
    d.fork([r.choice((-1, r.randrange(2048), r.randrange(9))) for _ in range(2048)], 2048)
    d.extend([r.choice((0, 1, 5)) for _ in range(2048)])
    d.fork([r.randrange(64) for _ in range(2048)], 64)
    d.extend([1] * 2048)
    d.compact()


@pytest.mark.parametrize("groups,K,W", [(1, 4, 9000), (2, 33, 5000), (1, 300, 700), (70, 2, 9001), (1, 1, 5000)])
def test_wide_tables(groups, K, W):
    r = random.Random(W)
    T, n = 16, groups * K
    lengths = [r.choice((W * T - 3, W * T // 2, 5, 0)) if n < 10 else r.choice((W * T // 9, 5, W * T - 3 if i < 3 else 1)) for i in range(n)]
    m = Model(sum(-(-x // T) for x in lengths) + 4 * n + 50, T, n, W).fill(lengths)
    d = Device(m)
    for _ in range(2):
        d.fork([r.choice((r.randrange(K), 0)) for _ in range(n)], K)
        d.extend([r.randint(0, 3) for _ in range(n)])
    d.compact()
    d.trim([h // 3 for h in m.held])


@pytest.mark.parametrize("K", (1, 2))
def test_the_most_rows(K):
    """65536 rows, as groups of their own and of two."""
    n, T = 65536, 16
    g = torch.Generator(device="cuda").manual_seed(K)
    pool, err = zx.PagePool(2 * n, T), i32([0])
    perm = torch.randperm(2 * n, generator=g, device="cuda").to(torch.int32).view(n, 2)
    table, held = perm.clone(), torch.randint(0, 33, (n,), generator=g, device="cuda", dtype=torch.int32)
    per = (held + T - 1) // T
    used = torch.arange(2, device="cuda") < per[:, None]
    pool.refs[table[used].long()] = 1
    was = held.clone()
    parents = torch.randint(-1, K, (n // K, K), generator=g, device="cuda", dtype=torch.int32)
    pool.fork(table, held, parents, err=err)
    goes = parents.view(-1) >= 0
    of = (torch.arange(n, device="cuda") // K * K + parents.view(-1).clamp(min=0)).long()
    assert torch.equal(held, torch.where(goes, was[of], 0))
    mine = torch.arange(2, device="cuda") < ((held + T - 1) // T)[:, None]
    assert torch.equal(table, torch.where(mine, perm[of], perm))
    assert torch.equal(pool.refs.long(), torch.bincount(table[mine].long(), minlength=2 * n))
    pool.trim(table, held, err=err)
    assert not bool(pool.refs.any()) and not bool(held.any()) and int(err) == 0


def test_rows_beyond_the_limit():
    d = Device(Model(100, 16, 3, 2))
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")   # noqa: E731
    with pytest.raises(ValueError):
        d.pool.extend(zx.PagedBatch(i(2050), i(2049), i(2049, 1)), i(2049))
    with pytest.raises(ValueError):
        d.pool.fork(i(2049, 1), i(2049), i(1, 2049))
    d.pool.trim(i(2049, 1), i(2049))
    with pytest.raises(zx.ZxError):
        d.pool.trim(i(65537, 1), i(65537))


def test_no_rows():
    pool = zx.PagePool(50, 16, refs=i32([0, 1] * 25))
    e = torch.zeros((0, 4), dtype=torch.int32, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda")
    pool.fork(*e, torch.zeros((0, 3), dtype=torch.int32, device="cuda"))
    pool.trim(*e)
    c = pool.extend(zx.PagedBatch(i32([0]), e[1], e[0]), e[1].clone())
    assert int(c.count) == 0
    copies, remap = pool.compact()
    assert int(copies.count) == 13 and pool.refs.tolist() == [1] * 25 + [0] * 25 and remap.tolist()[49] == 24
    copies, remap = pool.compact(*e)
    assert int(copies.count) == 0
    w0 = torch.zeros((2, 0), dtype=torch.int32, device="cuda")       # a table without columns
    pool.fork(w0, i32([0, 0]), i32([[1, 0]]))
    err = i32([0])
    pool.extend(zx.PagedBatch(i32([0, 0, 1]), i32([9, 9]), w0), i32([0, 0]), err=err)
    assert int(err) == 4


def test_streams_and_graphs():
    """Behind other work, on a side stream, and captured: a step replayed on states that change between."""
    m = Model(300, 16, 8, 12).fill([30, 0, 0, 0, 77, 0, 0, 0])
    d = Device(m)
    side = torch.cuda.Stream()
    w = torch.randn(4096, 4096, device="cuda")
    for _ in range(3):
        w = (w @ w).mul_(0.01)
    late = torch.zeros(8, dtype=torch.int32, device="cuda") + w[0, 0].clamp(0, 0).to(torch.int32)
    d.pool.fork(d.table, d.held, late.view(2, 4), err=d.err, stream=side)
    m.fork([0] * 8, 4)
    torch.cuda.current_stream().wait_stream(side)
    d.same()
    d.extend([1] * 8, stream=side)
    start, parents = i32(list(range(9))), i32([[0, 0, 1, 2], [3, 3, 3, 0]])
    batch = zx.PagedBatch(start, d.kv, d.table)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        d.pool.fork(d.table, d.held, parents, err=d.err)
        d.pool.extend(batch, d.held, copies=d.copies, err=d.err)
    d.same()
    r = random.Random(3)
    for i in range(6):
        p = [r.randrange(4) for _ in range(8)]
        parents.copy_(i32(p).view(2, 4))
        g.replay()
        m.fork(p, 4)
        kv, copies, enough = m.extend([1] * 8)
        assert enough and d.kv.tolist() == kv and d.listed() == copies
        d.same()
        if i == 3:
            d.compact()


def test_refusals():
    m = Model(40, 16, 4, 5).fill([20, 0, 0, 0])
    d = Device(m)
    t, h, p = d.table, d.held, i32([[0, 0, 0, 0]])
    b = d.batch([1] * 4)
    pool = d.pool
    bad = [lambda: zx.PagePool(0, 16), lambda: zx.PagePool((1 << 23) + 1, 16), lambda: zx.PagePool(4, 8), lambda: zx.PagePool(4, 48),
           lambda: zx.PagePool(4, 16, refs=i32([0] * 5)), lambda: zx.PagePool(4, 16, refs=torch.zeros(4, device="cuda")),
           lambda: zx.PagePool(4, 16, refs=torch.zeros(4, dtype=torch.int32)), lambda: pool.fork(t, h, p[0]), lambda: pool.fork(t, h, i32([[0, 0]])),
           lambda: pool.fork(t, h.long(), p), lambda: pool.fork(t[:, :3], h, p), lambda: pool.fork(t, h[:3], p), lambda: pool.fork(t, h, p.cpu()),
           lambda: pool.fork(t, h, h.view(1, 4)), lambda: pool.fork(t, t.view(-1)[:4], p), lambda: pool.fork(t, pool.refs[:4], p),
           lambda: pool.trim(t, h, i32([0] * 3)), lambda: pool.trim(t, h, h), lambda: pool.trim(t, h, torch.zeros(4, device="cuda")),
           lambda: pool.extend(b, d.kv), lambda: pool.extend(b, b.q_start[:4]), lambda: pool.extend(b, h, copies=zx.PageCopies(3)),
           lambda: pool.extend(b, h, err=torch.zeros(1, device="cuda")), lambda: pool.compact(t), lambda: pool.compact(None, h),
           lambda: pool.compact(t, h, copies=zx.PageCopies(19)), lambda: pool.compact(t, h, remap=i32([0] * 39)), lambda: pool.compact(t, h, remap=pool.refs),
           lambda: zx.PageCopies(-1), lambda: zx.PageCopies(2, pairs=i32([[0] * 3])), lambda: zx.PageCopies(1, pairs=i32([[0] * 3]), count=i32([0, 1])),
           lambda: pool.fork(t, h, p, stream=7), lambda: pool.trim(t, h, stream=7), lambda: pool.extend(b, h, stream=7), lambda: pool.compact(t, h, stream=7)]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was taken")
    d.same()
