"""Pages of the cache: qdr_kv_assign, qdr_kv_compact, qdr_kv_copy, and
qdr_slot_copy, compared whole with row-by-row computations on the host: tables,
reference counts, contexts, error bits and every byte of the memory."""
import random

import numpy as np
import pytest

from quantized_delta_rule_decode_amd import qdr
from test_gpu_kv import BF16, D, INT8, counts, held, i32, vectors

pytestmark = pytest.mark.gpu
BLOCK = {INT8: 2 * 32 * (D + 4), BF16: 2 * 32 * 2 * D}


@pytest.fixture(scope="module")
def torch_dev():
    import torch
    assert torch.cuda.is_available(), "device tests need a HIP GPU"
    qdr.load()
    return torch


def a_cache(torch, pages, page, heads, kind, seed=1):
    """A cache of random bytes and its memory [pages][heads][blocks][bytes]."""
    mem = torch.empty(qdr.qdr_kv_bytes(pages, page, heads, kind), dtype=torch.uint8, device="cuda")
    cache = qdr.KVCache(pages, page, heads, kind, dev_mem=mem)
    mem.copy_(torch.randint(0, 256, mem.shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda", dtype=torch.uint8))
    return cache, mem.view(pages, heads, page // 32, BLOCK[kind])


def assigned(rows, context, parent, add, refs, page, width):
    """What an assignment gives, and the copies it makes: (from, to, blocks)."""
    total, err = len(refs), 0
    room = min(width * page, 2 ** 30)
    valid = lambda p: 0 <= p < total
    hold = list(refs)
    old = []
    for r, c in zip(rows, context):
        ok = 0 <= c <= room
        err |= 0 if ok else qdr.DEVERR_LENGTH
        held_ = r[:-(-c // page)] if ok else []
        old.append((held_, ok))
        for p in held_:
            if valid(p):
                hold[p] -= 1
            else:
                err |= qdr.DEVERR_PAGE
    plan = []
    for a, x in zip(parent, add):
        ok = -1 <= a < len(rows) and (a < 0 or old[a][1])
        have = context[a] if ok and a >= 0 else 0
        ok = ok and 0 <= have + x <= room
        err |= 0 if ok else qdr.DEVERR_LENGTH
        after = have + x if ok else 0
        kept = min(have, after) if ok else 0
        plan.append([old[a][0] if kept else [], after, kept])
    for r, after, kept in plan:
        for p in r[:kept // page]:
            if valid(p):
                hold[p] += 1
            else:
                err |= qdr.DEVERR_PAGE
    first = {}
    for j, (r, after, kept) in enumerate(plan):
        if kept % page and valid(r[kept // page]):
            first.setdefault(r[kept // page], j)
    free = [p for p, x in enumerate(refs) if x == 0]
    new_refs, pages, contexts, copies, at = list(hold), [], [], [], 0
    for j, (r, after, kept) in enumerate(plan):
        full = kept // page
        row = [p if valid(p) else -1 for p in r[:full]]
        last = r[full] if kept % page and valid(r[full]) else -1
        stays = last >= 0 and hold[last] == 0 and first[last] == j
        need = -(-after // page) - full - stays
        take = free[at:at + need]
        at += need
        if len(take) < need:
            err |= qdr.DEVERR_FULL
            for p in row:
                if p >= 0:
                    new_refs[p] -= 1
            pages.append([-1] * width)
            contexts.append(0)
            continue
        if last >= 0 and not stays:
            copies.append((last, take[0], -(-(kept % page) // 32)))
        fresh = ([last] if stays else []) + take
        for p in fresh:
            new_refs[p] = 1
        pages.append((row + fresh + [-1] * width)[:width])
        contexts.append(after)
    return pages, contexts, new_refs, copies, err


def check_assign(torch, kind, rows, context, parent, add, refs, page, heads, width, seed=0, junk=-1):
    cache, mem = a_cache(torch, len(refs), page, heads, kind, seed + 1)
    before = mem.clone()
    want = assigned(rows, context, parent, add, refs, page, width)
    n, m = len(rows), len(parent)
    table = i32(torch, [(r + [junk] * width)[:width] for r in rows]).view(n, width)
    inputs = [table, i32(torch, context), i32(torch, parent), i32(torch, add), i32(torch, refs)]
    kept = [x.clone() for x in inputs]
    new = [torch.full((m, width), 77, dtype=torch.int32, device="cuda"), torch.full((m,), 77, dtype=torch.int32, device="cuda"),
           torch.full((len(refs),), 77, dtype=torch.int32, device="cuda")]
    cache.qdr_kv_assign(*inputs, *new)
    assert cache.qdr_kv_poll_device_error() == want[4]
    assert all(torch.equal(a, b) for a, b in zip(inputs, kept))
    assert new[0].tolist() == want[0]
    assert new[1].tolist() == want[1]
    assert new[2].tolist() == want[2]
    for a, b, blocks in want[3]:
        before[b, :, :blocks] = before[a, :, :blocks]
    assert torch.equal(mem, before)
    return want


def in_use(r, n, page, most, extra, common=0, held_by_program=0):
    """Random tables in use: rows, contexts, refs."""
    context = [r.randrange(common * page + 1, most + 1) for _ in range(n)]
    need = [-(-c // page) for c in context]
    total = sum(need) + extra
    order = list(range(total))
    r.shuffle(order)
    refs, rows = [0] * total, []
    for b in range(n):
        rows.append((rows[0][:common] if b else []) + [order.pop() for _ in range(need[b] - (common if b else 0))])
        for p in rows[-1]:
            refs[p] += 1
    for _ in range(held_by_program):
        refs[r.randrange(total)] += 1
    return rows, context, refs


@pytest.mark.parametrize("kind", [INT8, BF16])
@pytest.mark.parametrize("page", [32, 128, 1024])
@pytest.mark.parametrize("n,m", [(1, 1), (4, 9), (9, 4), (40, 40), (7, 0), (0, 5)])
def test_assign_random(torch_dev, kind, page, n, m):
    """Rows go on, fork, are taken back, end and begin, in one call."""
    r = random.Random(n * 100 + m + page)
    most = 5 * page
    rows, context, refs = in_use(r, n, page, most, 3 * m + 2, common=1 if n > 2 else 0, held_by_program=2)
    parent = [r.randrange(-1, n) for _ in range(m)]
    if n == m:
        parent = [j if r.random() < 0.7 else a for j, a in enumerate(parent)]
    add = [r.choice((0, 1, 1, page, -1, -7, 3, -page, 2 * page)) for _ in range(m)]
    add = [max(x, -(context[a] if a >= 0 else 0)) for a, x in zip(parent, add)]
    check_assign(torch_dev, kind, rows, context, parent, add, refs, page, 2, 9, seed=n)


def test_assign_steps_of_a_decode_loop(torch_dev):
    """Twenty steps, each from the tables of the one before: contexts, counts and pages stay consistent."""
    r = random.Random(5)
    page, total, width = 32, 90, 12
    rows, context, refs = [], [], [0] * total
    for step in range(20):
        n = len(rows)
        parent = [j for j in range(n) if r.random() < 0.85]
        parent += [r.randrange(n) for _ in range(r.randrange(0, 3)) if n] + [-1] * r.randrange(0, 3)
        add = [r.randrange(1, 120) if a < 0 else r.choice((1, 1, 1, 40)) for a in parent]
        pages, context, refs, _, err = check_assign(torch_dev, BF16, rows, context, parent, add, refs, page, 1, width, seed=step)
        rows = [p[:-(-c // page)] for p, c in zip(pages, context)]
        held_ = [0] * total
        for p in (p for row in rows for p in row):
            held_[p] += 1
        assert held_ == refs and err in (0, qdr.DEVERR_FULL, qdr.DEVERR_LENGTH, qdr.DEVERR_FULL | qdr.DEVERR_LENGTH)


def test_assign_last_page(torch_dev):
    """Who keeps a page in part: the first row, where nobody holds it otherwise."""
    page, width = 32, 4
    one = lambda **kw: check_assign(torch_dev, INT8, page=page, heads=3, width=width, **kw)
    # one row goes on: in place.  Held by the program too: a copy
    assert one(rows=[[3, 1]], context=[40], parent=[0], add=[1], refs=[0, 1, 0, 1])[3] == []
    assert one(rows=[[3, 1]], context=[40], parent=[0], add=[1], refs=[0, 2, 0, 1])[3] == [(1, 0, 1)]
    # three forks: the first keeps it
    assert one(rows=[[3, 1]], context=[40], parent=[0, 0, 0], add=[0, 1, 5], refs=[0, 1, 0, 1])[3] == [(1, 0, 1), (1, 2, 1)]
    # one row keeps the page whole, the other in part: a copy
    assert one(rows=[[3, 1]], context=[64], parent=[0, 0], add=[0, -10], refs=[0, 1, 0, 1])[3] == [(1, 0, 1)]
    # taken back by itself: in place; a full last page is not copied
    assert one(rows=[[3, 1]], context=[64], parent=[0], add=[-10], refs=[0, 1, 0, 1])[3] == []
    assert one(rows=[[3, 1]], context=[64], parent=[0, 0], add=[1, 1], refs=[0, 1, 0, 1])[3] == []
    # two old rows that share a page in part
    assert one(rows=[[3, 1], [3, 1]], context=[40, 50], parent=[1, 0], add=[1, 1], refs=[0, 2, 0, 2])[3] == [(1, 0, 1)]


def test_assign_runs_out_of_pages(torch_dev):
    page, width = 32, 8
    rows, context = [[0], [1], [2, 3]], [32, 32, 60]
    refs = [1, 1, 1, 1, 0, 0, 0]
    for add in ([1, 1, 100], [97, 1, 1], [200, 1, 1], [1, 1, 40], [96, 0, 0], [97, 0, 0]):
        want = check_assign(torch_dev, BF16, rows, context, [0, 1, 2], add, refs, page, 1, width)
        assert bool(want[4]) == (sum(-(-(c + x) // page) for c, x in zip(context, add)) - 4 > 3)
    # the row that found none gives up what it shared
    check_assign(torch_dev, BF16, [[0, 1]], [64], [0, 0, 0], [1, 1, 1], [1, 1, 0, 0], page, 1, width)
    check_assign(torch_dev, BF16, [], [], [-1, -1], [256, 1], [0] * 8, page, 1, width)


def test_assign_bad_values(torch_dev):
    torch, page, width = torch_dev, 32, 4
    refs = [1, 1, 1, 1, 0, 0, 0, 0]
    rows, context = [[0, 1], [2, 3]], [50, 64]
    for parent, add in (([2, 1], [1, 1]), ([-2, 1], [1, 1]), ([2 ** 31 - 1, 0], [1, 1]), ([0, 1], [-51, 1]), ([0, 1], [79, 0]), ([0, 1], [2 ** 31 - 1, 1]),
                        ([0, 1], [-2 ** 31, 1]), ([-1, 1], [-1, 1]), ([-1, 1], [129, 1])):
        assert check_assign(torch, INT8, rows, context, parent, add, refs, page, 1, width)[4] == qdr.DEVERR_LENGTH
    for bad in ([129, 64], [-1, 64], [2 ** 31 - 1, 64]):
        assert check_assign(torch, INT8, [[0, 1, 4, 5], [2, 3]], bad, [0, 1], [1, 1], refs, page, 1, width)[4] == qdr.DEVERR_LENGTH
    for page_ in (-1, 8, 2 ** 31 - 1, -2 ** 31):
        for at in (0, 1):
            r = [[0, 1], [2, 3]]
            r[0][at] = page_
            assert check_assign(torch, INT8, r, context, [0, 1, 0], [1, 1, 1], refs, page, 1, width)[4] == qdr.DEVERR_PAGE
    # tables without room
    cache, _ = a_cache(torch, 4, page, 1, INT8)
    none, out = torch.empty((2, 0), dtype=torch.int32, device="cuda"), i32(torch, [9, 9])
    refs4, new = i32(torch, [0, 0, 0, 5]), torch.empty(4, dtype=torch.int32, device="cuda")
    cache.qdr_kv_assign(none, i32(torch, [0, 0]), i32(torch, [0, 1]), i32(torch, [0, 1]), refs4, none.clone(), out, new)
    assert out.tolist() == [0, 0] and new.tolist() == [0, 0, 0, 5] and cache.qdr_kv_poll_device_error() == qdr.DEVERR_LENGTH


@pytest.mark.parametrize("m", [1023, 2500])
def test_assign_many_rows_and_pages(torch_dev, m):
    """More rows than the offsets are made at once, more pages than a workgroup lists, long tables."""
    r = random.Random(m)
    page, width = 32, 300
    n = 600
    rows, context, refs = in_use(r, n, page, 200, 6000, held_by_program=50)
    parent = [r.randrange(-1, n) for _ in range(m)]
    add = [r.choice((0, 1, 30)) for _ in range(m)]
    add[5], parent[5] = 9000, -1
    check_assign(torch_dev, INT8, rows, context, parent, add, refs, page, 1, width)


def compacted(refs, rows):
    live = [p for p, x in enumerate(refs) if x]
    free = iter([p for p, x in enumerate(refs) if not x])
    moved, new = [-1] * len(refs), [0] * len(refs)
    for p in live:
        moved[p] = p if p < len(live) else next(free)
        new[moved[p]] = refs[p]
    return moved, new, [[moved[p] if 0 <= p < len(refs) else -1 for p in row] for row in rows]


@pytest.mark.parametrize("kind", [INT8, BF16])
@pytest.mark.parametrize("total,live", [(1, 0), (1, 1), (7, 3), (64, 64), (64, 0), (500, 100), (2048, 2047), (2049, 1), (5000, 2600)])
def test_compact(torch_dev, kind, total, live):
    torch, r = torch_dev, random.Random(total + live)
    page, heads = (32, 1) if total > 600 else (64, 3)
    cache, mem = a_cache(torch, total, page, heads, kind)
    refs = [0] * total
    for p in r.sample(range(total), live):
        refs[p] = r.choice((1, 1, 2, -3, 40))
    rows = [[r.choice((-1, total, -2 ** 31, 2 ** 31 - 1, r.randrange(total), r.randrange(total))) for _ in range(33)] for _ in range(11)]
    moved, new_refs, tables = compacted(refs, rows)
    before = mem.clone()
    for p, to in enumerate(moved):
        if to >= 0 and to != p:
            before[to] = mem[p]
    ins = [i32(torch, refs), i32(torch, rows)]
    kept = [x.clone() for x in ins]
    outs = [torch.full_like(ins[0], 77), torch.full_like(ins[0], 77), torch.full_like(ins[1], 77)]
    cache.qdr_kv_compact(*ins, *outs)
    assert [x.tolist() for x in outs] == [moved, new_refs, tables]
    assert all(torch.equal(a, b) for a, b in zip(ins, kept)) and torch.equal(mem, before)
    assert cache.qdr_kv_poll_device_error() == 0
    # once more, from the new numbers: nothing moves; and without tables
    again = [torch.full_like(ins[0], 77) for _ in range(2)]
    cache.qdr_kv_compact(outs[1], ins[1][:0], *again, ins[1][:0].clone())
    assert again[1].tolist() == new_refs and again[0].tolist() == [p if p < live else -1 for p in range(total)] and torch.equal(mem, before)


@pytest.mark.parametrize("kind", [INT8, BF16])
@pytest.mark.parametrize("page,heads", [(32, 1), (256, 3), (1024, 5)])
def test_copy(torch_dev, kind, page, heads):
    """Within a cache and into another; -1 and bad numbers on either side."""
    torch = torch_dev
    (a, x), (b, y) = a_cache(torch, 9, page, heads, kind, 1), a_cache(torch, 5, page, heads, kind, 2)
    a.qdr_kv_copy(i32(torch, [0, 3, -1, 7, 7, 5]), i32(torch, [1, 4, 2, -1, 8, 5]))
    want = x.clone()
    assert a.qdr_kv_poll_device_error() == 0 and torch.equal(x[1], x[0]) and torch.equal(x[4], x[3]) and torch.equal(x[8], x[7])
    want_b = y.clone()
    a.qdr_kv_copy(i32(torch, [8, 9, 1, 2]), i32(torch, [0, 1, 5, 4]), to=b)
    want_b[0], want_b[4] = x[8], x[2]
    assert torch.equal(y, want_b) and torch.equal(x, want)
    assert a.qdr_kv_poll_device_error() == qdr.DEVERR_PAGE and b.qdr_kv_poll_device_error() == qdr.DEVERR_PAGE
    a.qdr_kv_copy(i32(torch, [-2, 2 ** 31 - 1]), i32(torch, [0, 1]))
    assert torch.equal(x, want) and a.qdr_kv_poll_device_error() == qdr.DEVERR_PAGE
    a.qdr_kv_copy(i32(torch, []), i32(torch, []), to=b)


@pytest.mark.parametrize("kinds", [[6, 8, 4, 16], [32, 32], [2]])
def test_slot_copy(torch_dev, kinds):
    torch, n = torch_dev, 6
    pool = qdr.Pool(n, len(kinds), kinds, np.ones((len(kinds), D), np.float32))
    S = torch.randn((n, len(kinds), D, D), generator=torch.Generator("cuda").manual_seed(4), device="cuda")
    pool.qdr_pack(i32(torch, list(range(n))), S)
    raw = [pool.qdr_read_raw(i) for i in range(n)]
    pool.qdr_slot_copy(i32(torch, [0, 0, -1, 5, 4]), i32(torch, [1, 2, 3, -1, 4]))
    assert pool.qdr_poll_device_error() == 0
    want = [raw[0], raw[0], raw[0], raw[3], raw[4], raw[5]]
    for i in range(n):
        assert np.array_equal(pool.qdr_read_raw(i), want[i])
    for s, d in ((n, 0), (0, n), (-2, 0), (0, 2 ** 31 - 1)):
        pool.qdr_slot_copy(i32(torch, [s, 5]), i32(torch, [d, 3]))
        assert pool.qdr_poll_device_error() == qdr.DEVERR_SLOT
    want[3] = raw[5]
    for i in range(n):
        assert np.array_equal(pool.qdr_read_raw(i), want[i])


def test_pages_beyond_32_bits(torch_dev):
    """Pages that lie above 2^32 bytes of the cache: copied, forked and moved."""
    torch, page, heads = torch_dev, 1024, 4
    size = qdr.qdr_kv_bytes(1, page, heads, BF16)
    total = (2 ** 32 + 2 ** 29) // size
    mem = torch.empty(total * size, dtype=torch.uint8, device="cuda")
    cache = qdr.KVCache(total, page, heads, BF16, dev_mem=mem)
    x = mem.view(total, size)
    for p in (total - 1, total - 2, 1):
        x[p] = torch.randint(0, 256, (size,), dtype=torch.uint8, device="cuda")
    cache.qdr_kv_copy(i32(torch, [1, total - 1]), i32(torch, [total - 3, 0]))
    assert torch.equal(x[total - 3], x[1]) and torch.equal(x[0], x[total - 1])
    refs = [2] * (total - 4) + [0, 1, 1, 1]
    new = [torch.empty((2, 1), dtype=torch.int32, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda"), torch.empty(total, dtype=torch.int32, device="cuda")]
    cache.qdr_kv_assign(i32(torch, [[total - 1]]), i32(torch, [1000]), i32(torch, [0, 0]), i32(torch, [1, 1]), i32(torch, refs), *new)
    assert new[0].tolist() == [[total - 1], [total - 4]] and torch.equal(x[total - 4], x[total - 1])
    refs = [0, 0, 5] + [0] * (total - 5) + [1, 1]
    outs = [torch.empty(total, dtype=torch.int32, device="cuda") for _ in range(2)]
    last = x[total - 2:].clone()
    cache.qdr_kv_compact(i32(torch, refs), i32(torch, [[total - 1]]), *outs, table := i32(torch, [[9]]))
    assert torch.equal(x[:2], last) and table.tolist() == [[1]] and outs[1][:3].tolist() == [1, 1, 5]


def test_pages_captured(torch_dev):
    """A compaction, copies of pages and of slots in one graph: every replay takes
    the numbers that its inputs hold by then, with eager calls between replays."""
    torch, total, heads, n = torch_dev, 40, 2, 6
    r = random.Random(9)
    (a, x), (b, y) = a_cache(torch, total, 32, heads, BF16, 1), a_cache(torch, 7, 32, heads, BF16, 2)
    pool = qdr.Pool(n, 1, [32], np.ones((1, D), np.float32))
    S = torch.randn((n, 1, D, D), generator=torch.Generator("cuda").manual_seed(4), device="cuda")
    slots = i32(torch, list(range(n)))
    refs, table = i32(torch, [0] * total), i32(torch, [[-1] * 5] * 3)
    outs = [torch.empty_like(refs), torch.empty_like(refs), torch.empty_like(table)]
    pairs = [i32(torch, [-1, -1, -1]) for _ in range(4)]
    ws = torch.empty(a.qdr_kv_compact_workspace(), dtype=torch.uint8, device="cuda")

    def calls():
        a.qdr_kv_compact(refs, table, *outs, workspace=ws)
        a.qdr_kv_copy(pairs[0], pairs[1], to=b)
        pool.qdr_slot_copy(pairs[2], pairs[3])

    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        calls()
    for i in range(4):
        held_now = [r.choice((0, 1, 2)) for _ in range(total)]
        rows = [[r.randrange(-1, total) for _ in range(5)] for _ in range(3)]
        src, dst, s, d = r.sample(range(total), 3), r.sample(range(7), 3), r.sample(range(3), 3), r.sample(range(3, 6), 3)
        for to, values in zip([refs, table, *pairs], [held_now, rows, src, dst, s, d]):
            to.copy_(i32(torch, values))
        pool.qdr_pack(slots, S * (i + 1))
        raw = [pool.qdr_read_raw(k) for k in range(n)]
        moved, new_refs, tables = compacted(held_now, rows)
        want, other = x.clone(), y.clone()
        for p, to in enumerate(moved):
            if to >= 0 and to != p:
                want[to] = x[p]
        for p, q in zip(src, dst):
            other[q] = want[p]
        torch.cuda.synchronize()
        if i == 2:
            calls()
        else:
            g.replay()
        torch.cuda.synchronize()
        assert [z.tolist() for z in outs] == [moved, new_refs, tables], f"turn {i}"
        assert torch.equal(x, want) and torch.equal(y, other), f"turn {i}"
        for p, q in zip(s, d):
            assert np.array_equal(pool.qdr_read_raw(q), raw[p])
        assert a.qdr_kv_poll_device_error() == 0 and b.qdr_kv_poll_device_error() == 0 and pool.qdr_poll_device_error() == 0


def test_pages_refusals(torch_dev):
    torch = torch_dev
    cache, _ = a_cache(torch, 4, 32, 1, INT8)
    pages, refs, one = i32(torch, [[0, 1]]), i32(torch, [1, 1, 0, 0]), i32(torch, [40])
    new = lambda: [torch.empty_like(pages), torch.empty_like(one), torch.empty_like(refs)]
    ok = [pages, one, i32(torch, [0]), i32(torch, [1]), refs]
    cache.qdr_kv_assign(*ok, *new())
    for i, bad, kind in ((0, pages[0], ValueError), (0, pages.long(), TypeError), (1, i32(torch, [1, 2]), ValueError), (3, i32(torch, [1, 2]), ValueError),
                         (4, refs[:3], ValueError), (2, i32(torch, [[0]]), ValueError)):
        args = list(ok)
        args[i] = bad
        with pytest.raises(kind):
            cache.qdr_kv_assign(*args, *new())
    a, b, c = new()
    for out in ((pages, b, c), (a, one, c), (a, b, refs), (a, c[:1], c)):
        with pytest.raises(qdr.QdrError):
            cache.qdr_kv_assign(*ok, *out)
    with pytest.raises(qdr.QdrError):
        cache.qdr_kv_assign(*ok, *new(), workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    for out in ((refs, c, a), (c, refs, a), (c, c, a), (c, torch.empty_like(c), pages)):
        with pytest.raises(qdr.QdrError):
            cache.qdr_kv_compact(refs, pages, *out)
    with pytest.raises(ValueError):
        cache.qdr_kv_compact(refs, pages, c, c[:3], a)
    for other in (qdr.KVCache(4, 64, 1, INT8), qdr.KVCache(4, 32, 2, INT8), qdr.KVCache(4, 32, 1, BF16)):
        with pytest.raises(qdr.QdrError):
            cache.qdr_kv_copy(i32(torch, [0]), i32(torch, [1]), to=other)
    with pytest.raises(ValueError):
        cache.qdr_kv_copy(i32(torch, [0]), i32(torch, [1, 2]))
    assert cache.qdr_kv_poll_device_error() == 0
