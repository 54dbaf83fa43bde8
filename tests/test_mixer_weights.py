"""Weights of few rows enter the attention's product in two bfloat16 parts.

With u = 2^-24, a weight's parts leave 2^-8 2^-8 of it, a score's products and
scalings err by e = 130 u |scale| sum |q||k| (a weight by 4 e), the sums over N
keys by (N + 8) u, and the result is rounded to bfloat16:
    |o - ref| <= 2^-8 |ref| + (2^-16 + 4 e + (N + 8) u) sum p |v|.
One part would leave 2^-8 of each weight: far more than this allows wherever
the values nearly cancel, which the first test shows with an oracle that rounds
so.  The scores are small (|scale| sum |q||k| < 1/2), so that the weights, not
the scores, are what is tested.
"""
import numpy as np
import pytest

from quantized_delta_rule_decode_amd import qdr

D, U, SCALE = 128, 2.0 ** -24, 0.01
# rows a sequence, contexts: single tokens; few rows; both among long chunks
CALLS = [([1], [40]), ([1] * 5, [33, 2, 300, 64, 200]), ([4], [90]), ([1, 700, 2, 600], [60, 700, 31, 900]),
         ([1, 1, 1, 2048], [200, 65, 33, 2048])]
FEW, Q, H, PAGE = 4, 8, 2, 64        # four query heads a key head: up to four tokens are few rows


def bf16(x):
    import torch
    return torch.tensor(x).to(torch.bfloat16).double().numpy()


def inputs(seed, contexts, rows):
    g = np.random.default_rng(seed)
    return bf16(g.standard_normal((sum(contexts), H, D))), bf16(g.standard_normal((sum(contexts), H, D))), bf16(0.5 * g.standard_normal((rows, Q, D)))


def held(x, kind):
    """What the cache holds."""
    if kind == qdr.KV_BF16:
        return x
    r = np.abs(x).max(-1, keepdims=True)
    return np.rint(127 * x / r) * (r.astype(np.float32) / np.float32(127)).astype(np.float64)


def attend(q, k, v, context, parts=None):
    """fp64 attention of a sequence's last rows, and the bound; parts: weights as so many bfloat16 values."""
    m, out, room = q.shape[0], np.empty(q.shape), np.empty(q.shape)
    for j in range(Q):
        K, V = k[:, j * H // Q], v[:, j * H // Q]
        s = SCALE * (q[:, j] @ K.T)
        s[np.arange(context) > np.arange(context - m, context)[:, None]] = -np.inf
        e = 130 * U * SCALE * (np.abs(q[:, j]) @ np.abs(K).T).max(-1, keepdims=True)
        p = np.exp(s - s.max(-1, keepdims=True))
        total, w = p.sum(-1, keepdims=True), p
        if parts:
            w, left = np.zeros_like(p), p
            for _ in range(parts):
                w, left = w + bf16(left), left - bf16(left)
        o, mag = w @ V / total, p @ np.abs(V) / total
        out[:, j] = bf16(o) if parts else o
        room[:, j] = 2.0 ** -8 * np.abs(o) + (2.0 ** -16 + 4 * e + (context + 8) * U) * mag
    return out, room


def sequences(lens, contexts):
    first = at = 0
    for m, c in zip(lens, contexts):
        yield m, c, slice(first, first + m), slice(at, at + c)
        first, at = first + m, at + c


@pytest.mark.parametrize("kind", [qdr.KV_INT8, qdr.KV_BF16])
@pytest.mark.parametrize("lens,contexts", CALLS, ids=str)
def test_the_bound_tells_one_part_from_two(kind, lens, contexts):
    k, v, q = inputs(7, contexts, sum(lens))
    k, v = held(k, kind), held(v, kind)
    over = {1: 0, 2: 0}
    for m, c, rows, keys in sequences(lens, contexts):
        if m > FEW:
            continue
        ref, room = attend(q[rows], k[keys], v[keys], c)
        for parts in over:
            over[parts] += (np.abs(attend(q[rows], k[keys], v[keys], c, parts)[0] - ref) > room).sum()
    assert over[2] == 0 and over[1] > 0, over


@pytest.mark.gpu
@pytest.mark.parametrize("kind", [qdr.KV_INT8, qdr.KV_BF16])
@pytest.mark.parametrize("lens,contexts", CALLS, ids=str)
def test_few_rows_have_their_weights_in_two_parts(kind, lens, contexts):
    import torch
    qdr.load()
    i32 = lambda x: torch.tensor(np.asarray(x).tolist(), dtype=torch.int32, device="cuda")      # noqa: E731
    dev = lambda x: torch.from_numpy(x).cuda().bfloat16()                                       # noqa: E731
    k, v, q = inputs(7, contexts, sum(lens))
    need = [-(-c // PAGE) for c in contexts]
    pages = np.full((len(lens), max(need)), -1)
    for b, m in enumerate(need):
        pages[b, :m] = np.arange(sum(need[:b]), sum(need[:b + 1]))
    with qdr.KVCache(sum(need), PAGE, H, kind) as cache:
        counts = lambda x: i32(np.concatenate([[0], np.cumsum(x)]))     # noqa: E731
        cache.qdr_kv_write(i32(pages), counts(contexts), i32(contexts), dev(k), dev(v))
        o = torch.empty((sum(lens), Q, D), dtype=torch.bfloat16, device="cuda")
        cache.qdr_kv_attend(i32(pages), counts(lens), i32(contexts), dev(q), o, scale=SCALE)
        got = o.double().cpu().numpy()
    k, v = held(k, kind), held(v, kind)
    for b, (m, c, rows, keys) in enumerate(sequences(lens, contexts)):
        if m > FEW:
            continue
        ref, room = attend(q[rows], k[keys], v[keys], c)
        off = np.abs(got[rows] - ref)
        assert (off <= room).all(), f"sequence {b}: {(off > room).sum()} results off, by up to {(off - room).max():.3g} over the bound"
