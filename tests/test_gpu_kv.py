"""The paged key/value cache (qdr_kv_write, qdr_kv_read) and the attention over
it (qdr_kv_attend).

Quantising is compared bit for bit with the definition: r = max |x| (1 below
2^-126), z = nearest-even(127 x / r) from the exact quotient (rational
arithmetic in fp64: 127 x is exact there and ties are exact), value z (r / 127)
in fp32, rounded to bfloat16.

Attention is compared with fp64 softmax over the values that the cache holds.
With u = 2^-24: a score's 128 products and two scalings err by at most
130 u |scale| sum |q||k| = e, which moves a weight by a factor 2^(+-2 e log2 e)
at most (the score's and the maximum's); 2^x errs by 2 u; the weights' sum over
N keys by N u; the weight enters its product rounded to bfloat16 (2^-8), and
the result is rounded to bfloat16 (2^-8):
|o - ref| <= 2^-8 |ref| + (2^-8 + 4 e + (N + 8) u) sum p |v| + f.
f is what underflow takes away, which no relative bound covers: a weight p, or
with 8-bit values p times the value's scale, below the smallest normal number
2^-126 may become 0.  The first loses at most 2^-126 |v| a key, the second
2^-126 times a code, and the sum of the weights is at least the largest, 1:
f = 2^-126 N (max |v| + 127).  (It matters where a channel's large values all
have weights that small: the fp64 result then is 10^-40 and less.)
"""
import numpy as np
import pytest

from quantized_delta_rule_decode_amd import qdr

pytestmark = pytest.mark.gpu
D = 128
U = 2.0 ** -24
INT8, BF16 = qdr.KV_INT8, qdr.KV_BF16


@pytest.fixture(scope="module")
def torch_dev():
    import torch
    assert torch.cuda.is_available(), "device tests need a HIP GPU"
    qdr.load()
    return torch


def i32(torch, x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def counts(torch, lens, lead=0):
    return i32(torch, np.concatenate([[lead], lead + np.cumsum(lens)]).astype(int).tolist())


def held(torch, x, kind):
    """What the cache holds of bfloat16 vectors: fp32 values (exact fp64 quotient, ties to even)."""
    if kind == BF16:
        return x.float()
    y = x.double()
    r = y.abs().amax(-1, keepdim=True)
    r = torch.where(r < 2.0 ** -126, torch.ones_like(r), r)
    z = torch.round(127 * y / r)
    scale = (r.float() / 127).float()
    bad = ~torch.isfinite(r)
    return torch.where(bad, torch.full_like(scale, float("nan")), z.float() * scale)


def table(torch, contexts, page, extra=2, seed=0, width=None):
    """Pages of every sequence in random order, -1 behind them."""
    need = [-(-c // page) for c in contexts]
    order = np.random.default_rng(seed).permutation(sum(need) + extra)
    width = max(need + [1]) if width is None else width
    t, at = np.full((len(contexts), width), -1), 0
    for b, m in enumerate(need):
        t[b, :m] = order[at:at + m]
        at += m
    return i32(torch, t.tolist()), sum(need) + extra


def vectors(torch, seed, T, H):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((T, H, D), generator=g, device="cuda") * torch.exp2(2 * torch.rand((T, H, 1), generator=g, device="cuda"))
    x[..., 5] *= 4
    return x.bfloat16()


def same(torch, a, b):
    """Equal, NaN for NaN."""
    return torch.equal(a.isnan(), b.isnan()) and torch.equal(torch.nan_to_num(a.float()), torch.nan_to_num(b.float()))


CASES = [([1], [1], 32), ([31, 1, 0, 64], [31, 40, 9, 64], 32), ([33, 100], [90, 300], 64), ([1] * 9, [1, 32, 33, 64, 65, 127, 128, 129, 255], 128),
         ([700], [1500], 1024), ([2, 37], [2, 57], 256)]


@pytest.mark.parametrize("kind", [INT8, BF16])
@pytest.mark.parametrize("lens,contexts,page", CASES, ids=str)
@pytest.mark.parametrize("H", [1, 3])
def test_write_and_read(torch_dev, kind, lens, contexts, page, H):
    """Rows go to the ends of their contexts and come back as held; tokens
    written before in the same blocks stay."""
    torch = torch_dev
    pages, num = table(torch, contexts, page)
    cache = qdr.KVCache(num, page, H, kind)
    old = [c - m if m else 0 for c, m in zip(contexts, lens)]
    k0, v0 = vectors(torch, 1, sum(old), H), vectors(torch, 2, sum(old), H)
    cache.qdr_kv_write(pages, counts(torch, old), i32(torch, old), k0, v0)
    lead, tail = 3, 2
    T = lead + sum(lens) + tail
    k1, v1 = vectors(torch, 3, T, H), vectors(torch, 4, T, H)
    cu, ctx = counts(torch, lens, lead), i32(torch, contexts)
    cache.qdr_kv_write(pages, cu, ctx, k1, v1)
    k, v = (torch.full((T, H, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cache.qdr_kv_read(pages, cu, ctx, k, v)
    rows = slice(lead, lead + sum(lens))
    for got, x in ((k, k1), (v, v1)):
        assert (got[:lead] == 7).all() and (got[rows.stop:] == 7).all()
        assert torch.equal(got[rows], held(torch, x[rows], kind).bfloat16())
    ko, vo = torch.empty_like(k0), torch.empty_like(v0)
    cache.qdr_kv_read(pages, counts(torch, old), i32(torch, old), ko, vo)
    assert torch.equal(ko, held(torch, k0, kind).bfloat16()) and torch.equal(vo, held(torch, v0, kind).bfloat16())
    assert cache.qdr_kv_poll_device_error() == 0


def test_quantising_at_the_edges(torch_dev):
    """Ties, zero, the smallest and largest values, infinity and NaN."""
    torch = torch_dev
    x = torch.zeros((9, 1, D), device="cuda")
    x[0, 0, :7] = torch.tensor([127, 0.5, 1.5, -2.5, 63.5, -126.5, 126.5])       # exact ties
    x[1, 0, :3] = torch.tensor([3.3895e38, -3.3895e38, 1e37])                    # the largest
    x[2, 0, :3] = torch.tensor([2.0 ** -126, -2.0 ** -127, 2.0 ** -133])         # the smallest normal
    x[3, 0, :2] = torch.tensor([2.0 ** -127, 2.0 ** -133])                       # below it: r = 1, codes 0
    x[5, 0, 9] = float("inf")
    x[6, 0, 9], x[6, 0, 10] = float("nan"), 2.0
    x[7, 0, 64] = -float("inf")
    x[8] = torch.linspace(-1, 1, D, device="cuda")
    x = x.bfloat16()
    cache = qdr.KVCache(2, 32, 1, INT8)
    pages, cu, ctx = i32(torch, [[1]]), i32(torch, [0, 9]), i32(torch, [9])
    cache.qdr_kv_write(pages, cu, ctx, x, x.flip(0).contiguous())
    k, v = torch.empty_like(x), torch.empty_like(x)
    cache.qdr_kv_read(pages, cu, ctx, k, v)
    ref = held(torch, x, INT8).bfloat16()
    assert same(torch, k, ref) and same(torch, v, ref.flip(0))
    assert k[5:8].isnan().all() and (k[3:5] == 0).all()


@pytest.mark.parametrize("kind", [INT8, BF16])
def test_bad_pages_and_counts(torch_dev, kind):
    torch = torch_dev
    H, page = 2, 32
    cache = qdr.KVCache(3, page, H, kind)
    x = vectors(torch, 1, 70, H)
    good = i32(torch, [[0, 1, 2]])
    cache.qdr_kv_write(good, i32(torch, [0, 70]), i32(torch, [70]), x, x)
    y = vectors(torch, 2, 70, H)
    k, v = torch.full_like(y, 7), torch.full_like(y, 7)
    for bad in ([[0, 3, 2]], [[0, -1, 2]], [[0, 2 ** 31 - 1, 2]]):
        cache.qdr_kv_write(i32(torch, bad), i32(torch, [0, 70]), i32(torch, [70]), x, x)
        assert cache.qdr_kv_poll_device_error() == qdr.DEVERR_PAGE
        cache.qdr_kv_read(i32(torch, bad), i32(torch, [0, 70]), i32(torch, [70]), k, v)
        assert cache.qdr_kv_poll_device_error() == qdr.DEVERR_PAGE
        ref = held(torch, x, kind).bfloat16()
        ref[32:64] = 0
        assert torch.equal(k, ref) and torch.equal(v, ref)
    # a context below the rows, above the table; counts out of range
    q = vectors(torch, 3, 70, 2 * H)
    for cu, ctx in (([0, 70], [69]), ([0, 70], [97]), ([0, 70], [-5]), ([0, 71], [71]), ([-1, 70], [71]), ([5, 3], [70]), ([0, 70], [2 ** 31 - 1])):
        k.fill_(7)
        o = torch.full_like(q, 7)
        cache.qdr_kv_write(good, i32(torch, cu), i32(torch, ctx), y, y)
        assert cache.qdr_kv_poll_device_error() == qdr.DEVERR_LENGTH, (cu, ctx)
        cache.qdr_kv_read(good, i32(torch, cu), i32(torch, ctx), k, v)
        assert cache.qdr_kv_poll_device_error() == qdr.DEVERR_LENGTH, (cu, ctx)
        cache.qdr_kv_attend(good, i32(torch, cu), i32(torch, ctx), q, o)
        assert cache.qdr_kv_poll_device_error() == qdr.DEVERR_LENGTH, (cu, ctx)
        if cu == [0, 70]:
            assert (k == 0).all() and (o == 0).all()
    cache.qdr_kv_read(good, i32(torch, [0, 70]), i32(torch, [70]), k, v)
    assert torch.equal(k, held(torch, x, kind).bfloat16())
    assert cache.qdr_kv_poll_device_error() == 0


def fill(torch, contexts, page, H, kind, seed=5, poison=True):
    """A cache that holds the contexts, its unused rows non-finite; the held values of each sequence."""
    pages, num = table(torch, contexts, page, seed=seed)
    mem = torch.empty(qdr.qdr_kv_bytes(num, page, H, kind), dtype=torch.uint8, device="cuda")
    cache = qdr.KVCache(num, page, H, kind, dev_mem=mem)
    if poison:
        mem.fill_(255)     # NaN as bfloat16 values and as scales
    k, v = vectors(torch, seed, sum(contexts), H), vectors(torch, seed + 1, sum(contexts), H)
    cache.qdr_kv_write(pages, counts(torch, contexts), i32(torch, contexts), k, v)
    return cache, pages, held(torch, k, kind).double(), held(torch, v, kind).double()


def reference(torch, q, k, v, lens, contexts, scale):
    """fp64 attention of every row, and the bound on its error (see above)."""
    out, room, first, at = [], [], 0, 0
    group = q.shape[1] // k.shape[1]
    for m, c in zip(lens, contexts):
        K, V = (x[at:at + c].repeat_interleave(group, 1).transpose(0, 1) for x in (k, v))     # [q_heads][c][D]
        Q = q[first:first + m].double().transpose(0, 1)
        s = scale * (Q @ K.transpose(1, 2).contiguous())
        e = 130 * U * abs(scale) * (Q.abs() @ K.abs().transpose(1, 2).contiguous()).amax(-1, keepdim=True)
        future = torch.arange(c, device="cuda") > torch.arange(c - m, c, device="cuda")[:, None]
        p = torch.softmax(s.masked_fill(future, -float("inf")), -1)
        ref, mag = p @ V, p @ V.abs()
        out.append(ref.transpose(0, 1))
        room.append((2.0 ** -8 * ref.abs() + (2.0 ** -8 + 4 * e + (c + 8) * U) * mag
                     + 2.0 ** -126 * c * (V.abs().max() + 127 if c else 0)).transpose(0, 1))
        first, at = first + m, at + c
    return torch.cat(out), torch.cat(room)


ATTEND = [
    # rows a sequence, contexts, page, q_heads, heads
    ([1], [1], 32, 1, 1),
    ([1], [777], 32, 8, 2),
    ([1, 1, 1, 1, 1], [33, 1, 500, 64, 2000], 64, 12, 4),
    ([1, 1], [300, 65], 32, 40, 1),
    ([2, 5, 16], [2, 100, 16], 32, 3, 1),
    ([17], [17], 32, 1, 1),
    ([64, 0, 1, 130], [64, 9, 200, 400], 64, 7, 7),
    ([100, 3], [1000, 3], 128, 16, 2),
    ([129], [129], 256, 34, 2),
    ([1, 300, 1, 40], [900, 700, 31, 40], 64, 8, 2),
    ([5], [90], 32, 200, 1),
    # single tokens among long chunks
    ([1, 700, 2, 600], [900, 700, 31, 900], 64, 8, 2),
    # no more rows than sequences, and yet one of several tiles
    ([0] * 9 + [7] + [0] * 5 + [1], [5] * 9 + [40] + [8] * 5 + [2100], 32, 16, 2),
    ([1, 0, 6, 0, 0, 3, 0, 0, 0, 0], [3000, 4, 2500, 1, 2, 3, 9, 70, 1, 33], 64, 16, 1),
]


@pytest.mark.parametrize("kind", [INT8, BF16])
@pytest.mark.parametrize("lens,contexts,page,q_heads,heads", ATTEND, ids=str)
def test_attend(torch_dev, kind, lens, contexts, page, q_heads, heads):
    torch = torch_dev
    cache, pages, k, v = fill(torch, contexts, page, heads, kind)
    lead, tail = 1, 4
    T = lead + sum(lens) + tail
    q = vectors(torch, 9, T, q_heads)
    o = torch.full((T, q_heads, D), 7.0, dtype=torch.bfloat16, device="cuda")
    scale = 0.11
    cache.qdr_kv_attend(pages, counts(torch, lens, lead), i32(torch, contexts), q, o, scale=scale)
    assert cache.qdr_kv_poll_device_error() == 0
    rows = slice(lead, lead + sum(lens))
    assert (o[:lead] == 7).all() and (o[rows.stop:] == 7).all()
    ref, room = reference(torch, q[rows], k, v, lens, contexts, scale)
    off = (o[rows].double() - ref).abs()
    assert (off <= room).all(), f"off by {(off - room).max().item():.3g} over the bound"


@pytest.mark.parametrize("kind", [INT8, BF16])
@pytest.mark.parametrize("scale", [-0.3, 0.0, 8.0])
def test_attend_scales(torch_dev, kind, scale):
    """Sharp, flat and negative weights; the default is 1 / sqrt(128)."""
    torch = torch_dev
    lens, contexts = [3, 50], [200, 90]
    cache, pages, k, v = fill(torch, contexts, 64, 2, kind)
    q = vectors(torch, 9, 53, 4)
    o, d, e = torch.empty_like(q), torch.empty_like(q), torch.empty_like(q)
    cache.qdr_kv_attend(pages, counts(torch, lens), i32(torch, contexts), q, o, scale=scale)
    ref, room = reference(torch, q, k, v, lens, contexts, scale)
    assert ((o.double() - ref).abs() <= room).all()
    cache.qdr_kv_attend(pages, counts(torch, lens), i32(torch, contexts), q, d)
    cache.qdr_kv_attend(pages, counts(torch, lens), i32(torch, contexts), q, e, scale=D ** -0.5)
    assert torch.equal(d, e)


@pytest.mark.parametrize("kind", [INT8, BF16])
def test_attend_bad_page_and_shared_pages(torch_dev, kind):
    """A bad page's keys take no part; two sequences may read the same pages."""
    torch = torch_dev
    cache, pages, k, v = fill(torch, [96], 32, 1, kind)
    ids = pages[0].tolist()
    both = i32(torch, [ids, [ids[0], -1, ids[2]]])
    q = vectors(torch, 9, 2, 2)
    o = torch.empty_like(q)
    cache.qdr_kv_attend(both, i32(torch, [0, 1, 2]), i32(torch, [96, 96]), q, o)
    assert cache.qdr_kv_poll_device_error() == qdr.DEVERR_PAGE
    some = torch.tensor([i for i in range(96) if not 32 <= i < 64], device="cuda")
    for row, keys in ((0, torch.arange(96, device="cuda")), (1, some)):
        ref, room = reference(torch, q[row:row + 1], k[keys], v[keys], [1], [len(keys)], D ** -0.5)
        assert ((o[row:row + 1].double() - ref).abs() <= room).all()
    bad = i32(torch, [[-1, 7, -1]])
    for rows in (1, 40):       # no page is good: rows are 0
        q = vectors(torch, 9, rows, 2)
        o = torch.full_like(q, 7)
        cache.qdr_kv_attend(bad, i32(torch, [0, rows]), i32(torch, [96]), q, o)
        assert (o == 0).all() and cache.qdr_kv_poll_device_error() == qdr.DEVERR_PAGE


@pytest.mark.parametrize("kind", [INT8, BF16])
@pytest.mark.parametrize("rows", [1, 40])
def test_attend_non_finite(torch_dev, kind, rows):
    """A NaN key makes the rows that see it NaN in its own head, and no others."""
    torch = torch_dev
    H, c = 2, 100
    cache, pages, k, v = fill(torch, [c], 32, H, kind)
    q = vectors(torch, 9, rows, 2 * H)
    cu, ctx = i32(torch, [0, rows]), i32(torch, [c])
    clean, o = torch.empty_like(q), torch.empty_like(q)
    cache.qdr_kv_attend(pages, cu, ctx, q, clean)
    at = c - 1 if rows == 1 else c - 10      # only the last ten rows of 40 see it
    kk, vv = k[at:at + 1].bfloat16(), v[at:at + 1].bfloat16()
    kk[0, 1, 3] = float("nan")
    cache.qdr_kv_write(pages, i32(torch, [0, 1]), i32(torch, [at + 1]), kk, vv)
    cache.qdr_kv_attend(pages, cu, ctx, q, o)
    seen = max(rows - 10, 0)
    assert torch.equal(o[:seen], clean[:seen])
    assert o[seen:, 2:].isnan().all() and not o[:, :2].isnan().any()


@pytest.mark.parametrize("kind", [INT8, BF16])
@pytest.mark.parametrize("rows", [3, 40, 150])
def test_attend_values_that_are_not_finite(torch_dev, kind, rows):
    """A value that is NaN or infinite reaches the rows that see its token, in
    its own head and (bfloat16) channel, and no row before it."""
    torch = torch_dev
    H, c, Q = 2, 200, 4
    cache, pages, k, v = fill(torch, [c], 32, H, kind)
    q = vectors(torch, 9, rows, Q)
    cu, ctx = i32(torch, [0, rows]), i32(torch, [c])
    clean, o = torch.empty_like(q), torch.empty_like(q)
    cache.qdr_kv_attend(pages, cu, ctx, q, clean, scale=0.02)
    ref, room = reference(torch, q, k, v, [rows], [c], 0.02)
    assert ((clean.double() - ref).abs() <= room).all()
    places = [(c - 1, 7, float("inf")), (c - 2, 7, float("-inf")), (c - 3 if rows == 3 else c - 20, 99, float("nan"))]
    for at, channel, bad in places:
        vv = v[at:at + 1].bfloat16()
        vv[0, 1, channel] = bad
        cache.qdr_kv_write(pages, i32(torch, [0, 1]), i32(torch, [at + 1]), k[at:at + 1].bfloat16(), vv)
    cache.qdr_kv_attend(pages, cu, ctx, q, o, scale=0.02)
    position = torch.arange(c - rows, c, device="cuda")
    same_as = o[:, :2]
    assert torch.isfinite(same_as).all() and ((same_as.double() - ref[:, :2]).abs() <= room[:, :2]).all()
    for row in range(rows):
        seen = [(ch, x) for at, ch, x in places if at <= position[row]]
        got = o[row, 2:]
        if kind == INT8:       # the scale of the vector is NaN: all its channels
            assert got.isnan().all() if seen else torch.isfinite(got).all()
        else:
            bad = torch.zeros(D, dtype=torch.bool, device="cuda")
            for ch, _ in seen:
                bad[ch] = True
            assert torch.isfinite(got[:, ~bad]).all(), f"row {row}"
            if any(ch == 99 for ch, _ in seen):
                assert got[:, 99].isnan().all()
            if bad[7]:         # the older token first: -inf alone, then both
                both = position[row] >= c - 1
                assert got[:, 7].isnan().all() if both else (got[:, 7] == float("-inf")).all()
        if not seen:
            assert ((got.double() - ref[row, 2:]).abs() <= room[row, 2:]).all()


@pytest.mark.parametrize("rows", [1, 40, 150])
def test_attend_values_of_no_weight_that_are_not_finite(torch_dev, rows):
    """Some 8-bit vectors of values that are NaN, several in a block and one in each
    of two neighbouring ones, behind keys whose weights underflow: still NaN for the
    rows that see any, in their head, and nothing for the others."""
    torch = torch_dev
    H, c, Q = 2, 300, 4
    cache, pages, k, v = fill(torch, [c], 32, H, INT8)
    q = torch.ones((rows, Q, D), dtype=torch.bfloat16, device="cuda")
    cu, ctx = i32(torch, [0, rows]), i32(torch, [c])
    clean, o = torch.empty_like(q), torch.empty_like(q)
    cache.qdr_kv_attend(pages, cu, ctx, q, clean, scale=1.0)
    assert torch.isfinite(clean).all()
    first = c - 1 if rows == 1 else c - 30
    for at in {first, c - 1, c - 2, c - 3} if rows > 1 else {first}:
        kk, vv = torch.full((1, H, D), -60.0, dtype=torch.bfloat16, device="cuda"), v[at:at + 1].bfloat16()   # a score of -7680
        vv[0, 1, 5] = float("nan")
        cache.qdr_kv_write(pages, i32(torch, [0, 1]), i32(torch, [at + 1]), kk, vv)
    cache.qdr_kv_attend(pages, cu, ctx, q, o, scale=1.0)
    seen = max(rows - 30, 0)
    assert torch.equal(o[:seen], clean[:seen])
    assert o[seen:, 2:].isnan().all() and torch.isfinite(o[:, :2]).all()


@pytest.mark.parametrize("kind", [INT8, BF16])
def test_attend_graphs_and_streams(torch_dev, kind):
    """The cache as a decode loop uses it, captured: write the token, attend.
    Two graphs with workspaces of their own replay beside each other and equal
    the eager calls, with eager work between the replays."""
    torch = torch_dev
    n, H, page = 3, 2, 32
    contexts = [200, 33, 64]
    eager, pages, k, v = fill(torch, contexts, page, H, kind)
    twins = [fill(torch, contexts, page, H, kind)[0] for _ in range(2)]
    cu, ctx = i32(torch, [0, 1, 2, 3]), i32(torch, contexts)
    static = [vectors(torch, 50, n, h) for h in (4, H, H)]
    graphs, outs, keep = [], [], []
    for c in twins:
        o, g = torch.zeros((n, 4, D), dtype=torch.bfloat16, device="cuda"), torch.cuda.CUDAGraph()
        ws = torch.empty(c.qdr_kv_attend_workspace(n, n, 4, pages.shape[1]), dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            c.qdr_kv_write(pages, cu, ctx, static[1], static[2])
            c.qdr_kv_attend(pages, cu, ctx, static[0], o, workspace=ws)
        graphs.append(g), outs.append(o), keep.append(ws)
    for turn in range(4):
        new = [vectors(torch, 60 + 3 * turn + i, n, h) for i, h in enumerate((4, H, H))]
        for a, b in zip(static, new):
            a.copy_(b)
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in twins]
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        ref = torch.empty_like(outs[0])
        eager.qdr_kv_write(pages, cu, ctx, new[1], new[2])
        eager.qdr_kv_attend(pages, cu, ctx, new[0], ref)
        torch.cuda.synchronize()
        for o in outs:
            assert torch.equal(o, ref), f"replay {turn}"
            o.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o = torch.empty_like(ref)
        eager.qdr_kv_attend(pages, cu, ctx, new[0], o)
        copy = o.clone()
    side.synchronize()
    assert torch.equal(copy, ref)


def test_a_prompt_in_chunks_and_tokens(torch_dev):
    """Chunks and single tokens, written and attended in turn, give the rows of
    the whole prompt in one call (the split of the keys may differ: one bf16
    step and the weights' rounding on either side)."""
    torch = torch_dev
    H, Q, page, total = 2, 6, 64, 333
    k, v, q = vectors(torch, 1, total, H), vectors(torch, 2, total, H), vectors(torch, 3, total, Q)
    pages, num = table(torch, [total], page)
    for kind in (INT8, BF16):
        one, two = qdr.KVCache(num, page, H, kind), qdr.KVCache(num, page, H, kind)
        whole = torch.empty_like(q)
        one.qdr_kv_write(pages, i32(torch, [0, total]), i32(torch, [total]), k, v)
        one.qdr_kv_attend(pages, i32(torch, [0, total]), i32(torch, [total]), q, whole)
        parts, at = torch.empty_like(q), 0
        for m in (1, 100, 31, 1, 1, 64, 130, 5):
            rows = slice(at, at + m)
            cu, ctx = i32(torch, [0, m]), i32(torch, [at + m])
            two.qdr_kv_write(pages, cu, ctx, k[rows], v[rows])
            two.qdr_kv_attend(pages, cu, ctx, q[rows], parts[rows])
            at += m
        ref, room = reference(torch, q, held(torch, k, kind).double(), held(torch, v, kind).double(), [total], [total], D ** -0.5)
        for o in (whole, parts):
            assert ((o.double() - ref).abs() <= room).all()


@pytest.mark.parametrize("kind", [INT8, BF16])
def test_cache_beyond_32_bits(torch_dev, kind):
    """Pages that lie above 2^32 bytes of the cache."""
    torch = torch_dev
    H, page = 2, 1024
    pages = (2 ** 32 + 2 ** 30) // qdr.qdr_kv_bytes(1, page, H, kind)
    cache, small = qdr.KVCache(pages, page, H, kind), qdr.KVCache(4, page, H, kind)
    lens, contexts = [1, 200], [1500, 2000]
    k, v = vectors(torch, 31, 3500, H), vectors(torch, 32, 3500, H)
    q = vectors(torch, 33, 201, 4 * H)
    got = []
    for c, where in ((small, [[2, 0], [1, 3]]), (cache, [[pages - 1, pages - 4], [0, pages - 2]])):
        t, all_of = i32(torch, where), counts(torch, contexts)
        c.qdr_kv_write(t, all_of, i32(torch, contexts), k, v)
        rk, rv, o = torch.empty_like(k), torch.empty_like(v), torch.empty_like(q)
        c.qdr_kv_read(t, all_of, i32(torch, contexts), rk, rv)
        c.qdr_kv_attend(t, counts(torch, lens), i32(torch, contexts), q, o)
        assert c.qdr_kv_poll_device_error() == 0
        got.append((rk, rv, o))
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert torch.equal(got[0][0], held(torch, k, kind).bfloat16())


@pytest.mark.parametrize("rows", [1, 40])
def test_largest_context(torch_dev, rows):
    """2^30 tokens, a cache's pages over and over; one token more is refused."""
    torch = torch_dev
    page, most = 1024, 2 ** 30
    cache = qdr.KVCache(1, page, 1, INT8)
    k, v = vectors(torch, 34, page, 1), vectors(torch, 35, page, 1)
    table_ = torch.zeros((1, most // page + 1), dtype=torch.int32, device="cuda")
    cache.qdr_kv_write(table_, i32(torch, [0, page]), i32(torch, [page]), k, v)
    q, cu = vectors(torch, 36, rows, 1), i32(torch, [0, rows])
    for context in (most + 1, most + page):
        o, x = torch.full_like(q, 7), torch.full_like(q, 7)
        cache.qdr_kv_attend(table_, cu, i32(torch, [context]), q, o)
        assert cache.qdr_kv_poll_device_error() == qdr.DEVERR_LENGTH and not o.any()
        cache.qdr_kv_read(table_, cu, i32(torch, [context]), x, x.clone())
        assert cache.qdr_kv_poll_device_error() == qdr.DEVERR_LENGTH and not x.any()
        cache.qdr_kv_write(table_, cu, i32(torch, [context]), q, q)
        assert cache.qdr_kv_poll_device_error() == qdr.DEVERR_LENGTH
    x, y = torch.empty_like(k), torch.empty_like(v)
    cache.qdr_kv_read(table_, i32(torch, [0, page]), i32(torch, [most]), x, y)      # its last page's tokens
    assert torch.equal(x, held(torch, k, INT8).bfloat16()) and torch.equal(y, held(torch, v, INT8).bfloat16())
    # The whole context: every key 2^20 times, so the result is the page's own
    # attention.  A row misses up to 40 of the 2^30 tokens (40 / 2^20 of the
    # weights' sum at most), and no running sum has more than 2^20 terms
    # (2^20 u = 2^-4 of the weighted values).
    o = torch.empty_like(q)
    cache.qdr_kv_attend(table_, cu, i32(torch, [most]), q, o)
    K, V = held(torch, k, INT8).double(), held(torch, v, INT8).double()
    for i in range(rows):
        ref, room = reference(torch, q[i:i + 1], K, V, [1], [page], D ** -0.5)
        room = room + (2.0 ** -4 + 80 / 2 ** 20) * V.abs().amax(0)
        assert ((o[i:i + 1].double() - ref).abs() <= room).all(), i
    assert cache.qdr_kv_poll_device_error() == 0


def test_attend_of_very_many_rows(torch_dev):
    """2^24 (token, head) rows in one call: 4096 sequences of 64 tokens and 64
    query heads; every fourth has the same queries and pages, and results."""
    torch = torch_dev
    n, m, H, Q = 4096, 64, 8, 64
    cache, pages, k, v = fill(torch, [m] * 4, 64, H, BF16)
    few = vectors(torch, 9, 4 * m, Q)
    q = few.repeat(n // 4, 1, 1)
    o = torch.full_like(q, 7)
    cache.qdr_kv_attend(pages.repeat(n // 4, 1), counts(torch, [m] * n), i32(torch, [m] * n), q, o)
    assert cache.qdr_kv_poll_device_error() == 0
    ref, room = reference(torch, few, k, v, [m] * 4, [m] * 4, D ** -0.5)
    assert ((o[:4 * m].double() - ref).abs() <= room).all()
    assert (o.view(n // 4, 4 * m, Q, D) == o[:4 * m]).all()


def test_refusals(torch_dev):
    torch = torch_dev
    cache = qdr.KVCache(2, 32, 2, INT8)
    x = vectors(torch, 1, 5, 2)
    pages, cu, ctx = i32(torch, [[0, 1]]), i32(torch, [0, 5]), i32(torch, [5])
    odd = torch.empty(5 * 2 * D + 1, dtype=torch.bfloat16, device="cuda")[1:].view(5, 2, D)
    for args, kind in (((pages, cu, ctx, x, odd), qdr.QdrError), ((pages, cu, ctx, x.float(), x), TypeError), ((pages, cu, ctx, x, x[:4]), ValueError),
                       ((pages, cu, i32(torch, [5, 5]), x, x), ValueError), ((pages[0], cu, ctx, x, x), ValueError),
                       ((pages.long(), cu, ctx, x, x), TypeError), ((pages, cu, ctx, x[:, :1], x[:, :1]), ValueError)):
        for call in (cache.qdr_kv_write, cache.qdr_kv_read):
            with pytest.raises(kind):
                call(*args)
    q = vectors(torch, 1, 5, 4)
    for args, kw, kind in (((pages, cu, ctx, q[:, :3].contiguous(), q[:, :3].contiguous()), {}, qdr.QdrError), ((pages, cu, ctx, q, q.float()), {}, TypeError),
                           ((pages, cu, ctx, q, q), dict(scale=float("nan")), qdr.QdrError),
                           ((pages, cu, ctx, q, x), {}, ValueError)):
        with pytest.raises(kind):
            cache.qdr_kv_attend(*args, **kw)
    with pytest.raises(qdr.QdrError):
        qdr.KVCache(2, 32, 2, INT8, dev_mem=torch.empty(100, dtype=torch.uint8, device="cuda"))
    assert cache.qdr_kv_poll_device_error() == 0
