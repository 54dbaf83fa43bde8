"""Edges of qdr_kv_attend_shared.

Weights in two parts: the bound is that of test_mixer_weights.py.  The join of a
row's passes adds three fp32 roundings a pass; a pass takes a block of 32 keys or
more, whose weights are summed in 32 roundings at most by themselves, so that
3 (N / 32 + 2) more stay within (N + 8) u for N keys with what those sums leave of
it (a block's 32 products are one matrix instruction's, 8 deep)."""
import numpy as np
import pytest

from quantized_delta_rule_decode_amd import qdr
import test_mixer_weights as weights
from test_gpu_kv import BF16, INT8, i32, vectors
from test_gpu_shared import Scene


@pytest.fixture(scope="module")
def torch_dev():
    import torch
    assert torch.cuda.is_available(), "device tests need a HIP GPU"
    qdr.load()
    return torch


@pytest.mark.gpu
@pytest.mark.parametrize("kind", [INT8, BF16])
@pytest.mark.parametrize("wide", [True, False])
@pytest.mark.parametrize("prefix", [64, 900])
def test_rows_that_no_count_covers(torch_dev, kind, wide, prefix):
    """Counts out of order or range: rows of no sequence are left as they are, also where an earlier call left its results of them in the workspace."""
    torch = torch_dev
    s = Scene(torch, [(prefix, [(1, 3), (2, 2), (1, 1)]), (100, [(1, 1), (20, 30)])], 32, 2, 4, kind, wide=wide)
    assert s.T == 30 and s.args[1].tolist() == [2, 3, 5, 6, 7, 27]
    ws = torch.full((s.cache.qdr_kv_attend_shared_workspace(5, s.T, 2, 4, s.pages.shape[1]),), 1, dtype=torch.uint8, device="cuda")
    good = s.args[1]
    for bad in ([2, 3, 5, 7, 7, 31], [-1, 3, 5, 6, 7, 27], [2, 3, 5, 1, 1, 1], [2, 3, 5, 6, 100, 27], [2, 3, 5, 6, -5, 27], [31, 3, 2, 1, 0, -1], [2 ** 31 - 1] * 6):
        s.args[1] = good
        s.check(torch, s.run(torch, workspace=ws))
        s.args[1] = i32(torch, bad)
        o = s.run(torch, workspace=ws)
        assert s.cache.qdr_kv_poll_device_error() == qdr.DEVERR_LENGTH, bad
        own = np.zeros(s.T, bool)
        for a, b in zip(bad, bad[1:]):
            if 0 <= a <= b <= s.T:
                own[a:b] = True
        assert (o[torch.from_numpy(~own).cuda()] == 7).all(), bad


# prefixes and their sequences' (new tokens, own tokens): groups of up to four tokens,
# that is 16 rows of four query heads, in one part and in several of the line
FEW = [[(64, [(1, 3), (1, 40), (1, 1)])], [(33, [(1, 3), (3, 4)]), (700, [(2, 2), (1, 90), (1, 5)])], [(2500, [(1, 1), (1, 9), (2, 300)])]]


def few_calls(groups, seed=7):
    """Keys and values of every sequence (fp64, bfloat16 values), queries, and where each is."""
    lens = [m for _, rows in groups for m, _ in rows]
    contexts = [p + tail for p, rows in groups for _, tail in rows]
    k, v, q = weights.inputs(seed, contexts, sum(lens))
    at = 0
    for p, rows in groups:           # the first tokens of a group are the same
        first = at
        for _, tail in rows:
            k[at:at + p], v[at:at + p] = k[first:first + p], v[first:first + p]
            at += p + tail
    return lens, contexts, k, v, q


@pytest.mark.parametrize("kind", [INT8, BF16])
def test_the_bound_tells_one_part_from_two(kind):
    """In the scenes of up to some hundred keys; over 2500 the roundings of one part average out below it."""
    over = {1: [], 2: []}
    for groups in FEW:
        lens, contexts, k, v, q = few_calls(groups)
        k, v, off = weights.held(k, kind), weights.held(v, kind), {1: 0, 2: 0}
        for m, c, rows, keys in weights.sequences(lens, contexts):
            ref, room = weights.attend(q[rows], k[keys], v[keys], c)
            for parts in off:
                off[parts] += int((np.abs(weights.attend(q[rows], k[keys], v[keys], c, parts)[0] - ref) > room).sum())
        for parts in off:
            over[parts].append(off[parts])
    assert over[2] == [0, 0, 0] and over[1][0] > 0 and over[1][1] > 0, over


@pytest.mark.gpu
@pytest.mark.parametrize("kind", [INT8, BF16])
@pytest.mark.parametrize("wide,groups", [(True, x) for x in FEW] + [(False, x) for x in FEW + [[(150, [(1, 3 + i) for i in range(9)])], [(90, [(4, 4 + i) for i in range(3)])]]], ids=str)
def test_few_rows_have_their_weights_in_two_parts(torch_dev, kind, wide, groups):
    """Groups of up to 16 rows a key head; and, where tables are narrow and every
    sequence goes by itself, sequences of up to 16 of any group."""
    torch, page = torch_dev, weights.PAGE
    lens, contexts, k, v, q = few_calls(groups)
    n, width = len(lens), max(-(-c // page) for c in contexts)
    if wide:
        width = max(width, -(-12288 * 32 // ((n - len(groups)) * weights.H * page)))
    table, num, b, dev = np.full((n, width), -1), 0, 0, lambda x: torch.from_numpy(x).cuda().bfloat16()
    for p, rows in groups:
        common = np.arange(num, num + p // page)
        num += p // page
        for _, tail in rows:
            own = -(-(p + tail) // page) - p // page
            table[b, :p // page] = common
            table[b, p // page:p // page + own] = np.arange(num, num + own)
            num, b = num + own, b + 1
    count = lambda x: i32(torch, np.concatenate([[0], np.cumsum(x)]).tolist())     # noqa: E731
    with qdr.KVCache(num, page, weights.H, kind) as cache:
        pages = i32(torch, table.tolist())
        cache.qdr_kv_write(pages, count(contexts), i32(torch, contexts), dev(k), dev(v))
        o = torch.empty((sum(lens), weights.Q, weights.D), dtype=torch.bfloat16, device="cuda")
        cache.qdr_kv_attend_shared(pages, count(lens), i32(torch, contexts), count([len(rows) for _, rows in groups]),
                                   i32(torch, [p for p, _ in groups]), dev(q), o, scale=weights.SCALE)
        assert cache.qdr_kv_poll_device_error() == 0
        got = o.double().cpu().numpy()
    k, v = weights.held(k, kind), weights.held(v, kind)
    for b, (m, c, rows, keys) in enumerate(weights.sequences(lens, contexts)):
        ref, room = weights.attend(q[rows], k[keys], v[keys], c)
        off = np.abs(got[rows] - ref)
        assert (off <= room).all(), f"sequence {b}: {(off > room).sum()} results off, by up to {(off - room).max():.3g} over the bound"


@pytest.mark.gpu
@pytest.mark.parametrize("kind", [INT8, BF16])
@pytest.mark.parametrize("wide", [True, False])
@pytest.mark.parametrize("members,new", [(3, 1), (30, 1), (3, 20), (3, 50)])
def test_values_of_no_weight_that_are_nan(torch_dev, kind, wide, members, new):
    """Shared values that are NaN behind keys whose weights underflow: NaN for the
    group's rows, in their head (bfloat16: and channel), and nothing for others."""
    torch = torch_dev
    s = Scene(torch, [(200, [(new, new + 9)] * members), (64, [(1, 2)] * 3)], 32, 2, 8, kind, wide=wide)
    s.q.fill_(1)
    # (scores of some hundreds: one key has all the weight)
    clean = s.run(torch, 1.0)
    s.check(torch, clean, 1.0)
    for at in (40, 41, 70, 191):
        k, v = torch.full((1, 2, 128), -60.0, dtype=torch.bfloat16, device="cuda"), s.vs[0][at:at + 1].clone()     # a score of -7680
        v[0, 1, 9] = float("nan")
        s.cache.qdr_kv_write(s.pages[:1], i32(torch, [0, 1]), i32(torch, [at + 1]), k, v)
    o = s.run(torch, 1.0)
    assert s.cache.qdr_kv_poll_device_error() == 0
    end = s.lead + members * new
    hit = o[s.lead:end]
    assert torch.isfinite(hit[:, :4]).all() and torch.isfinite(o[end:]).all() and torch.equal(o[end:], clean[end:])
    assert hit[:, 4:, 9].isnan().all()
    if kind == INT8:
        assert hit[:, 4:].isnan().all()
    else:
        assert hit[:, 4:].isnan().sum() == members * new * 4


@pytest.mark.gpu
@pytest.mark.parametrize("kind", [INT8, BF16])
def test_group_arrays_of_a_fixed_shape(torch_dev, kind):
    """One group and empty ones behind it, as many as sequences; and a group among many sequences of none."""
    torch = torch_dev
    s = Scene(torch, [(900, [(1, 5 + i) for i in range(12)])], 64, 2, 8, kind)
    want = s.run(torch)
    s.check(torch, want)
    s.args[3:] = [i32(torch, [0] + [12] * 12), i32(torch, [900] + [0] * 11)]
    s.check(torch, s.run(torch))
    s.args[3:] = [i32(torch, [0] * 11 + [0, 12]), i32(torch, [900] * 12)]
    s.check(torch, s.run(torch))
    assert s.cache.qdr_kv_poll_device_error() == 0
    s = Scene(torch, [(300, [(1, 5), (2, 2)])], 64, 2, 8, kind, alone=[(1, 40 + i) for i in range(60)], wide=True)
    s.check(torch, s.run(torch))
    assert s.cache.qdr_kv_poll_device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("kind", [INT8, BF16])
@pytest.mark.parametrize("wide", [True, False])
def test_a_call_repeats_itself(torch_dev, kind, wide):
    """The same bits again, whatever the workspace held before."""
    torch = torch_dev
    s = Scene(torch, [(3000, [(1, 1 + 13 * i % 90) for i in range(30)]), (500, [(20, 30)] * 4)], 64, 2, 8, kind, wide=wide)
    want = s.run(torch)
    s.check(torch, want)
    ws = torch.empty(s.cache.qdr_kv_attend_shared_workspace(34, s.T, 2, 8, s.pages.shape[1]), dtype=torch.uint8, device="cuda")
    for fill in (0, 255, 127, 60):
        ws.fill_(fill)
        assert torch.equal(s.run(torch, workspace=ws), want)
