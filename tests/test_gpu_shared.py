"""Attention of sequences that share their first tokens (qdr_kv_attend_shared)
against fp64 softmax over the values that the cache holds, with the bound of
test_gpu_kv.py: the passes over shared and own keys are joined in fp32 (a few
u more, inside the bound's (N + 8) u for N >= 2 keys), and their weights have one
rounding of 2^-8 at most, as there."""
import numpy as np
import pytest

from quantized_delta_rule_decode_amd import qdr
from test_gpu_kv import BF16, D, INT8, counts, held, i32, reference, vectors

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch_dev():
    import torch
    assert torch.cuda.is_available(), "device tests need a HIP GPU"
    qdr.load()
    return torch


class Scene:
    """Groups (prefix, [(new, tail), ...]) over a cache whose unused rows are not finite."""

    def __init__(self, torch, groups, page, heads, q_heads, kind, seed=3, alone=(), wide=True):
        self.lens, self.contexts, self.shared, self.group_cu, ks, vs, spans = [], [], [], [0], [], [], []
        every = list(groups) + [(0, [x]) for x in alone]
        for p, rows in every:
            k, v = vectors(torch, seed, p, heads), vectors(torch, seed + 1, p, heads)
            seed += 2
            for new, tail in rows:
                ks.append(torch.cat([k, vectors(torch, seed, tail, heads)]))
                vs.append(torch.cat([v, vectors(torch, seed + 1, tail, heads)]))
                seed += 2
                self.lens.append(new)
                self.contexts.append(p + tail)
            spans.append((p // page, len(rows)))
        for p, rows in groups:
            self.shared.append(p)
            self.group_cu.append(self.group_cu[-1] + len(rows))
        n = len(self.lens)
        width = max([-(-c // page) for c in self.contexts] + [1])
        if wide and n > len(groups):   # tables that show enough keys for the groups' rows to go together
            width = max(width, -(-12288 * 32 // ((n - len(groups)) * heads * page)))
        need = sum(-(-c // page) for c in self.contexts)
        order = np.random.default_rng(seed).permutation(need + 3).tolist()
        table, b = [[-1] * width for _ in range(n)], 0
        for common, members in spans:
            first = [order.pop() for _ in range(common)]
            for _ in range(members):
                table[b][:common] = first
                for i in range(common, -(-self.contexts[b] // page)):
                    table[b][i] = order.pop()
                b += 1
        self.pages = i32(torch, table)
        mem = torch.empty(qdr.qdr_kv_bytes(need + 3, page, heads, kind), dtype=torch.uint8, device="cuda")
        self.cache = qdr.KVCache(need + 3, page, heads, kind, dev_mem=mem)
        mem.fill_(255)
        for b in range(n):         # (shared pages again and again, with the same values)
            self.cache.qdr_kv_write(self.pages[b:b + 1], i32(torch, [0, self.contexts[b]]), i32(torch, [self.contexts[b]]), ks[b], vs[b])
        self.k, self.v = (held(torch, torch.cat(x), kind).double() for x in (ks, vs))
        self.ks, self.vs = ks, vs
        self.lead, self.T = 2, 2 + sum(self.lens) + 3
        self.q = vectors(torch, seed + 5, self.T, q_heads)
        self.rows = slice(self.lead, self.lead + sum(self.lens))
        self.args = [self.pages, counts(torch, self.lens, self.lead), i32(torch, self.contexts), i32(torch, self.group_cu), i32(torch, self.shared)]

    def run(self, torch, scale=0.11, **kw):
        o = torch.full_like(self.q, 7)
        self.cache.qdr_kv_attend_shared(*self.args, self.q, o, scale=scale, **kw)
        return o

    def check(self, torch, o, scale=0.11):
        assert (o[:self.lead] == 7).all() and (o[self.rows.stop:] == 7).all()
        ref, room = reference(torch, self.q[self.rows], self.k, self.v, self.lens, self.contexts, scale)
        off = (o[self.rows].double() - ref).abs()
        assert (off <= room).all(), f"off by {(off - room).max().item():.3g} over the bound"


SCENES = [
    # groups, page, q_heads, heads, sequences in no group
    ([(300, [(1, 40), (1, 40)])], 32, 8, 2, []),
    ([(64, [(1, 1), (1, 1), (1, 1)])], 32, 1, 1, []),
    ([(31, [(1, 2), (1, 5)])], 32, 4, 4, []),                       # less than a block
    ([(33, [(1, 3)] * 5)], 64, 12, 4, [(1, 70), (3, 9)]),
    ([(1000, [(1, 30 + i) for i in range(20)])], 64, 8, 2, []),     # 80 rows a head
    ([(500, [(1, 7)] * 40), (0, [(1, 9)] * 2), (77, [(1, 1)]), (2049, [(1, 300), (2, 2), (1, 64)])], 128, 16, 4, [(1, 500)]),
    ([(512, [(3, 40), (0, 5), (17, 17), (1, 33), (40, 90)])], 32, 6, 2, [(0, 4), (50, 60)]),
    ([(200, [(150, 200), (130, 130), (5, 9)])], 256, 4, 1, []),     # rows that fill tiles by themselves
    ([(700, [(100, 100), (120, 300)]), (320, [(2, 2), (1, 1)])], 64, 32, 8, []),
    ([(96, [(0, 3), (0, 0), (1, 1), (1, 2)])], 32, 2, 1, []),       # the first has no rows
    ([(4000, [(1, 1), (1, 1000)])], 1024, 200, 1, []),              # 200 query heads of one key head
    ([(640, [(1, 2), (2, 40), (1, 3)])], 32, 40, 1, [(1, 3), (1, 700)]),
    ([], 32, 4, 2, [(1, 100), (20, 50)]),
]


@pytest.mark.parametrize("kind", [INT8, BF16])
@pytest.mark.parametrize("wide", [True, False])
@pytest.mark.parametrize("groups,page,q_heads,heads,alone", SCENES, ids=str)
def test_attend_shared(torch_dev, kind, groups, page, q_heads, heads, alone, wide):
    torch = torch_dev
    s = Scene(torch, groups, page, heads, q_heads, kind, alone=alone, wide=wide)
    o = s.run(torch)
    s.check(torch, o)
    assert s.cache.qdr_kv_poll_device_error() == 0
    # smaller shared counts are as good, and none at all
    for part in ([x // 2 for x in s.shared], [0] * len(s.shared)):
        s.args[4] = i32(torch, part)
        s.check(torch, s.run(torch))
    s.args[3:] = [i32(torch, [0]), i32(torch, [])]
    s.check(torch, s.run(torch))
    assert s.cache.qdr_kv_poll_device_error() == 0


@pytest.mark.parametrize("kind", [INT8, BF16])
@pytest.mark.parametrize("members", [64, 100])
def test_attend_shared_long(torch_dev, kind, members):
    """A batch behind a long prefix, cut into many pieces."""
    torch = torch_dev
    s = Scene(torch, [(9000, [(1, 1 + 13 * i % 90) for i in range(members)])], 64, 2, 8, kind)
    s.check(torch, s.run(torch))
    assert s.cache.qdr_kv_poll_device_error() == 0


@pytest.mark.parametrize("kind", [INT8, BF16])
@pytest.mark.parametrize("groups", [255, 256, 257, 600])
def test_attend_shared_many_groups(torch_dev, kind, groups):
    """More groups than a workgroup has at hand, some of them of one sequence, empty, or without whole blocks."""
    torch = torch_dev
    s = Scene(torch, [(64 + 32 * (i % 5) - 60 * (i % 7 == 3), [(1 + (i % 50 == 7) * 8, 9 + i % 40)] * (i % 4)) for i in range(groups)], 32, 1, 2, kind)
    s.check(torch, s.run(torch))
    assert s.cache.qdr_kv_poll_device_error() == 0


@pytest.mark.parametrize("kind", [INT8, BF16])
@pytest.mark.parametrize("scale", [-0.3, 0.0, 8.0])
def test_attend_shared_scales(torch_dev, kind, scale):
    torch = torch_dev
    s = Scene(torch, [(200, [(1, 30), (2, 5)]), (130, [(30, 40), (9, 9), (1, 3)])], 64, 2, 8, kind)
    s.check(torch, s.run(torch, scale), scale)
    d, e = torch.empty_like(s.q), torch.empty_like(s.q)
    s.cache.qdr_kv_attend_shared(*s.args, s.q, d)
    s.cache.qdr_kv_attend_shared(*s.args, s.q, e, scale=D ** -0.5)
    assert torch.equal(d[s.rows], e[s.rows])


@pytest.mark.parametrize("kind", [INT8, BF16])
@pytest.mark.parametrize("members", [3, 30])
def test_attend_shared_bad_pages(torch_dev, kind, members):
    """A bad page among the shared ones takes no part; where all are bad and a row has no other key, it is 0."""
    torch = torch_dev
    s = Scene(torch, [(96, [(1, 1)] * members)], 32, 1, 4, kind)
    s.pages[:, 1] = -1
    o = s.run(torch)
    assert s.cache.qdr_kv_poll_device_error() == qdr.DEVERR_PAGE
    some = torch.tensor([i for i in range(97) if not 32 <= i < 64], device="cuda")
    for b in range(members):
        row = slice(s.lead + b, s.lead + b + 1)
        ref, room = reference(torch, s.q[row], s.k[97 * b:97 * b + 97][some], s.v[97 * b:97 * b + 97][some], [1], [len(some)], 0.11)
        assert ((o[row].double() - ref).abs() <= room).all()
    s.pages.fill_(2 ** 31 - 1)
    o = s.run(torch)
    assert (o[s.rows] == 0).all() and s.cache.qdr_kv_poll_device_error() == qdr.DEVERR_PAGE


def test_attend_shared_bad_counts(torch_dev):
    """Groups and sequences that are skipped, and the others as they are."""
    torch = torch_dev
    s = Scene(torch, [(64, [(1, 3), (2, 2), (1, 1)]), (100, [(1, 1), (20, 30)])], 32, 2, 4, INT8)
    good = s.run(torch)
    s.check(torch, good)
    first, second = slice(s.lead, s.lead + 4), slice(s.lead + 4, s.lead + 25)
    # (where keys are cut follows from every length, so the others may round differently)
    ref, room = reference(torch, s.q[s.rows], s.k, s.v, s.lens, s.contexts, 0.11)
    fits = lambda o, rows: ((o[rows].double() - ref[rows.start - s.lead:rows.stop - s.lead]).abs() <= room[rows.start - s.lead:rows.stop - s.lead]).all()
    for shared in ([-1, 100], [67, 100], [2 ** 31 - 1, 100], [32 * 100, 100]):
        s.args[4] = i32(torch, shared)
        o = s.run(torch)
        assert s.cache.qdr_kv_poll_device_error() == qdr.DEVERR_LENGTH
        assert (o[first] == 0).all() and fits(o, second)
    # only the first has that many older tokens
    s.args[4] = i32(torch, [66, 100])
    o = s.run(torch)
    assert s.cache.qdr_kv_poll_device_error() == qdr.DEVERR_LENGTH
    assert (o[s.lead + 1:s.lead + 4] == 0).all() and fits(o, second) and (o[s.lead] != 0).any()
    s.args[4] = i32(torch, [64, 100])
    for at, ctx in ((0, -1), (0, 10 ** 6), (4, 19), (4, 2 ** 31 - 1)):
        context = list(s.contexts)
        context[at] = ctx
        s.args[2] = i32(torch, context)
        o = s.run(torch)
        assert s.cache.qdr_kv_poll_device_error() == qdr.DEVERR_LENGTH
        if at == 0:
            assert (o[first] == 0).all() and fits(o, second)
        else:
            assert (o[s.lead + 5:s.lead + 25] == 0).all() and fits(o, first)
    s.args[2] = i32(torch, s.contexts)
    # pairs out of order or range: nothing outside the rows is touched
    for bad in ([0, 5, 3], [-1, 3, 5], [0, 3, 6], [3, 0, 5], [0, -2 ** 31, 5], [2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1]):
        s.args[3] = i32(torch, bad)
        o = s.run(torch)
        assert s.cache.qdr_kv_poll_device_error() == qdr.DEVERR_LENGTH, bad
        assert (o[:s.lead] == 7).all() and (o[s.rows.stop:] == 7).all()
    s.args[3] = i32(torch, [0, 3, 5])
    for bad in ([2, 3, 5, 1, 7, 27], [-1, 3, 5, 6, 7, 27], [2, 3, 5, 6, 7, 31], [2 ** 31 - 1] * 6):
        s.args[1] = i32(torch, bad)
        o = s.run(torch)
        assert s.cache.qdr_kv_poll_device_error() == qdr.DEVERR_LENGTH, bad


@pytest.mark.parametrize("kind", [INT8, BF16])
@pytest.mark.parametrize("members", [3, 40])
def test_attend_shared_non_finite(torch_dev, kind, members):
    """A NaN among the shared keys or values reaches the group's rows in its own head, and nobody else's."""
    torch = torch_dev
    for part in (0, 1):
        s = Scene(torch, [(100, [(1, 4)] * members), (64, [(1, 2)] * 3)], 32, 2, 8, kind)
        clean = s.run(torch, 0.02)
        s.check(torch, clean, 0.02)
        x = [s.ks[0][40:41].clone(), s.vs[0][40:41].clone()]
        x[part][0, 1, 9] = float("nan")
        s.cache.qdr_kv_write(s.pages[:1], i32(torch, [0, 1]), i32(torch, [41]), *x)
        o = s.run(torch, 0.02)
        hit = o[s.lead:s.lead + members]
        assert torch.equal(hit[:, :4], clean[s.lead:s.lead + members, :4]) and torch.equal(o[s.lead + members:], clean[s.lead + members:])
        assert hit[:, 4:, 9].isnan().all()
        if part == 0 or kind == INT8:
            assert hit[:, 4:].isnan().all()
        else:
            assert hit[:, 4:].isnan().sum() == members * 4


@pytest.mark.parametrize("width", [12, 1600])      # entries of a table: each sequence by itself, or all together
@pytest.mark.parametrize("kind", [INT8, BF16])
def test_fork_write_attend(torch_dev, kind, width):
    """A run as a server makes it: a prompt is written, forks into samples, and
    for some steps each sample's tokens are turned, written and attended to, the
    shared pages once; captured as graphs (two tables in turn) and eagerly."""
    torch, page, heads, q_heads, prompt, m, steps = torch_dev, 32, 2, 8, 150, 5, 6
    total = 40
    freq, amplitude = qdr.qdr_rotary_frequencies(qdr.ROTARY_TURNS, 128, 10000.0, 4.0, 64.0, 1.0, 4.0)
    rot = qdr.Rotary(freq, qdr.ROTARY_HALF, amplitude)
    g0 = torch.Generator("cuda").manual_seed(8)
    rand = lambda *shape: torch.randn(shape, generator=g0, device="cuda").bfloat16()
    start = [rand(prompt, h, D) for h in (heads, heads)]
    tokens = [[rand(m, h, D) for h in (q_heads, heads, heads)] for _ in range(steps)]
    every = torch.arange(m + 1, dtype=torch.int32, device="cuda")
    groups, shared = i32(torch, [0, m]), i32(torch, [prompt])
    ones, ident = i32(torch, [1] * m), i32(torch, list(range(m)))

    def begin():
        cache = qdr.KVCache(total, page, heads, kind)
        books = [[torch.zeros((m, width), dtype=torch.int32, device="cuda"), torch.zeros(m, dtype=torch.int32, device="cuda"),
                  torch.zeros(total, dtype=torch.int32, device="cuda")] for _ in range(2)]
        one = [torch.empty((1, width), dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda"), torch.empty(total, dtype=torch.int32, device="cuda")]
        cache.qdr_kv_assign(one[0][:0], one[1][:0], i32(torch, [-1]), i32(torch, [prompt]), torch.zeros(total, dtype=torch.int32, device="cuda"), *one)
        cache.qdr_kv_write_rotary(rot, one[0], i32(torch, [0, prompt]), one[1], *start)
        cache.qdr_kv_assign(one[0], one[1], i32(torch, [0] * m), i32(torch, [0] * m), one[2], *books[0])
        return cache, books

    def step(cache, old, new, q, k, v, q_out, o, ws):
        cache.qdr_kv_assign(old[0], old[1], ident, ones, old[2], *new, workspace=ws[0])
        cache.qdr_kv_write_rotary(rot, new[0], every, new[1], k, v, q=q, q_out=q_out)
        cache.qdr_kv_attend_shared(new[0], every, new[1], groups, shared, q_out, o, workspace=ws[1])

    def spaces(cache):
        return [torch.empty(b, dtype=torch.uint8, device="cuda")
                for b in (cache.qdr_kv_assign_workspace(m), cache.qdr_kv_attend_shared_workspace(m, m, 1, q_heads, width))]

    eager, books = begin()
    twin, twin_books = begin()
    static = [torch.empty_like(x) for x in tokens[0]]
    outs = [torch.empty_like(static[0]) for _ in range(4)]
    ws, ws2 = spaces(eager), spaces(twin)
    graphs = []
    for turn in range(2):
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            step(twin, twin_books[turn], twin_books[1 - turn], *static, outs[2], outs[3], ws2)
        graphs.append(g)
    for i in range(steps):
        for a, b in zip(static, tokens[i]):
            a.copy_(b)
        graphs[i % 2].replay()
        step(eager, books[i % 2], books[1 - i % 2], *tokens[i], outs[0], outs[1], ws)
        torch.cuda.synchronize()
        now, other = books[1 - i % 2], twin_books[1 - i % 2]
        assert all(torch.equal(a, b) for a, b in zip(now, other))
        assert torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[3]), f"step {i}"
        assert now[1].tolist() == [prompt + i + 1] * m
        # against the formula over what the cache holds
        context = prompt + i + 1
        k, v = (torch.empty((m * context, heads, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        eager.qdr_kv_read(now[0], counts(torch, [context] * m), now[1], k, v)
        plain = torch.empty_like(outs[0])
        eager.qdr_kv_attend(now[0], every, now[1], outs[0], plain)
        ref, room = reference(torch, outs[0], k.double(), v.double(), [1] * m, [context] * m, D ** -0.5)
        if kind == BF16:       # (what is read of 8-bit codes is rounded once more)
            assert ((outs[1].double() - ref).abs() <= room).all() and ((plain.double() - ref).abs() <= room).all()
        else:                  # two evaluations of the same: both bounds, from the values as they are read (2^-8 off)
            assert ((outs[1].double() - plain.double()).abs() <= 2 * (room * (1 + 2.0 ** -7))).all()
        for b in range(1, m):
            at = slice(b * context, b * context + prompt)
            assert torch.equal(k[at], k[:prompt]) and torch.equal(v[at], v[:prompt])
    assert eager.qdr_kv_poll_device_error() == 0 and twin.qdr_kv_poll_device_error() == 0
    # the samples end: every page is free
    last = books[steps % 2]
    freed = torch.empty(total, dtype=torch.int32, device="cuda")
    eager.qdr_kv_assign(last[0], last[1], i32(torch, []), i32(torch, []), last[2], last[0][:0].clone(), last[1][:0].clone(), freed)
    assert not freed.any()


def test_attend_shared_streams(torch_dev):
    """Two calls at once, on streams of their own, with workspaces of their own; and on a side stream without one."""
    torch = torch_dev
    s = Scene(torch, [(600, [(1, 9)] * 30), (64, [(2, 70)] * 2)], 64, 2, 8, INT8)
    want = s.run(torch)
    s.check(torch, want)
    n, groups = len(s.lens), len(s.shared)
    outs, streams, keep = [], [torch.cuda.Stream() for _ in range(2)], []
    torch.cuda.synchronize()
    for x in streams:
        with torch.cuda.stream(x):
            ws = torch.empty(s.cache.qdr_kv_attend_shared_workspace(n, s.T, groups, 8, s.pages.shape[1]), dtype=torch.uint8, device="cuda")
            keep.append(ws)
            outs.append(s.run(torch, workspace=ws))
    side = torch.cuda.Stream()
    o = torch.full_like(s.q, 7)
    side.wait_stream(torch.cuda.current_stream())
    s.cache.qdr_kv_attend_shared(*s.args, s.q, o, scale=0.11, stream=side)
    torch.cuda.synchronize()
    for x in outs + [o]:
        assert torch.equal(x, want)


def test_attend_shared_refusals(torch_dev):
    torch = torch_dev
    s = Scene(torch, [(64, [(1, 3), (2, 2)])], 32, 2, 4, BF16)
    pages, cu, ctx, gcu, shared = s.args
    o = torch.empty_like(s.q)
    for args, kw, kind in (((pages, cu, ctx, gcu[:1], shared, s.q, o), {}, ValueError), ((pages, cu, ctx, gcu, shared[None], s.q, o), {}, ValueError),
                           ((pages, cu, ctx, gcu.long(), shared, s.q, o), {}, TypeError), ((pages, cu, ctx, gcu, shared, s.q[:, :3].contiguous(), o[:, :3].contiguous()), {}, qdr.QdrError),
                           ((pages, cu, ctx, gcu, shared, s.q, o), dict(scale=float("inf")), qdr.QdrError), ((pages, cu, ctx, gcu, shared, s.q, o), dict(scale=3e38), qdr.QdrError),
                           ((pages, cu, ctx, gcu, shared, s.q, o), dict(workspace=torch.empty(64, dtype=torch.uint8, device="cuda")), qdr.QdrError),
                           ((pages, cu, ctx, gcu, shared, s.q, o.float()), {}, TypeError), ((pages, cu, ctx[:1], gcu, shared, s.q, o), {}, ValueError)):
        with pytest.raises(kind):
            s.cache.qdr_kv_attend_shared(*args, **kw)
    assert s.cache.qdr_kv_poll_device_error() == 0
