"""Rotary positions: qdr_rotate, qdr_rotate_bf16 and qdr_kv_write_rotary against
the exact rotation: the angle p f modulo one turn in whole numbers of 2^-120
turns (Python integers), its sine and cosine and the products in fp64.

Bound, with u = 2^-24 and A the amplitude: the kernels' angle is off by 2^-31 of a
turn at most (2^-32 of it and the truncation before it), 3e-9 < u / 10; reduced
to an eighth of a turn it is at most 0.7854, twice rounded and times a constant
(2.5 u 0.79 = 2 u); the series and its roundings add 2 u, the amplitude's
rounding and product 1.5 u: sine and cosine are off by 6 u A.  A turned value is
two products and a sum: |y - ref| <= 8 u A (|a| + |b|) =: e; rounded to bfloat16
2^-8 (|ref| + e) more.  8-bit codes: the largest magnitude is within e of the
exact one, the code within half a step of the fp32 quotient, which is right to 4 u
of up to 127: (0.5 + 2^-14) scale + e, and the scale is (r + e) / 127 (1 + 2 u).
"""
import math

import numpy as np
import pytest

from quantized_delta_rule_decode_amd import qdr
from test_gpu_kv import BF16, D, INT8, counts, held, i32, table, vectors

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF, PAIRS = qdr.ROTARY_HALF, qdr.ROTARY_PAIRS
PI = 3141592653589793238462643383279502884197169399375105820974944592307816406286  # 10^75 pi


@pytest.fixture(scope="module")
def torch_dev():
    import torch
    assert torch.cuda.is_available(), "device tests need a HIP GPU"
    qdr.load()
    return torch


def turned(torch, x, positions, freq, layout, amplitude=1.0):
    """fp64 rotation of x [T][heads][128] and the bound e on a fp32 result."""
    angles = np.empty((len(positions), len(freq)))
    for j, f in enumerate(freq):
        num, den = float(f).as_integer_ratio()
        step = (num * 10 ** 75 << 120) // (den * 2 * PI)
        for i, p in enumerate(positions):
            angles[i, j] = (p * step % (1 << 120)) / (1 << 120) * 2 * math.pi
    angles = torch.tensor(angles, device="cuda")
    c = 2 * len(freq)
    z = x.double()
    y, e = z.clone(), torch.zeros_like(z)
    cos, sin = amplitude * angles.cos()[:, None], amplitude * angles.sin()[:, None]
    first, second = (slice(0, c // 2), slice(c // 2, c)) if layout == HALF else (slice(0, c, 2), slice(1, c, 2))
    a, b = z[..., first], z[..., second]
    y[..., first], y[..., second] = a * cos - b * sin, a * sin + b * cos
    e[..., first] = e[..., second] = 8 * U * abs(amplitude) * (a.abs() + b.abs()) + 2.0 ** -140
    return y, e


FAR = [0, 1, 7, 4095, 131071, 2 ** 30, 2 ** 31 - 1, -1, -70000, -2 ** 31, 12345, 2 ** 24 + 1]


@pytest.mark.parametrize("layout", [HALF, PAIRS])
@pytest.mark.parametrize("channels", [16, 48, 64, 128])
@pytest.mark.parametrize("T,heads", [(1, 1), (12, 3), (70, 8), (5, 130), (3, 300)])
def test_rotate(torch_dev, layout, channels, T, heads):
    torch = torch_dev
    freq, amplitude = qdr.qdr_rotary_frequencies(qdr.ROTARY_INDEX, channels, 10000.0, 4.0, 4096.0)
    rot = qdr.Rotary(freq, layout, amplitude)
    pos = (FAR * 6)[:T]
    x = torch.randn((T, heads, D), generator=torch.Generator("cuda").manual_seed(1), device="cuda")
    y = torch.full_like(x, 7)
    rot.qdr_rotate(i32(torch, pos), x, y)
    ref, e = turned(torch, x, pos, freq, layout, amplitude)
    assert ((y.double() - ref).abs() <= e).all()
    assert torch.equal(y[..., channels:], x[..., channels:])
    xb = x.bfloat16()
    yb = torch.full_like(xb, 7)
    rot.qdr_rotate_bf16(i32(torch, pos), xb, yb)
    ref, e = turned(torch, xb, pos, freq, layout, amplitude)
    assert ((yb.double() - ref).abs() <= 2.0 ** -8 * (ref.abs() + e) + e).all()
    assert torch.equal(yb[..., channels:], xb[..., channels:])
    # in place, and from and to rows that are parts of longer ones
    z = xb.clone()
    rot.qdr_rotate_bf16(i32(torch, pos), z, z)
    assert torch.equal(z, yb)
    for a, ref, call in ((x, y, rot.qdr_rotate), (xb, yb, rot.qdr_rotate_bf16)):
        wide, out = torch.full((T, heads + 3, D), 9, dtype=a.dtype, device="cuda"), torch.full((T, heads + 2, D), 5, dtype=a.dtype, device="cuda")
        wide[:, 1:heads + 1] = a
        call(i32(torch, pos), wide[:, 1:heads + 1], out[:, 2:])
        assert torch.equal(out[:, 2:], ref) and (out[:, :2] == 5).all()


def test_rotate_frequencies_of_any_size(torch_dev):
    """Zero, negative, below 2^-40 and above a turn a token."""
    torch = torch_dev
    freq = np.array([0.0, -0.7, 1e-13, 7.5, 2.0 ** 20, -1000.25, math.pi, 2 * math.pi])
    rot = qdr.Rotary(freq, PAIRS, -0.5)
    pos = FAR
    x = torch.randn((len(pos), 2, D), generator=torch.Generator("cuda").manual_seed(2), device="cuda")
    y = torch.empty_like(x)
    rot.qdr_rotate(i32(torch, pos), x, y)
    # (turns a token as they are kept are off by 2^-64 |turns| and 2^-65: at 2^31 positions and 2^18 turns 2^-15 of a turn)
    ref, e = turned(torch, x, pos, freq, PAIRS, -0.5)
    off = torch.tensor(2 * math.pi * 2.0 ** -63 * (np.abs(freq) / 6 + 1), device="cuda")
    e[..., :16] += 0.5 * (torch.tensor(pos, device="cuda").double().abs()[:, None] * off).repeat_interleave(2, 1)[:, None] * (
        x[..., 0:16:2].abs() + x[..., 1:16:2].abs()).double().repeat_interleave(2, -1)
    assert ((y.double() - ref).abs() <= e).all()


@pytest.mark.parametrize("layout", [HALF, PAIRS])
def test_rotate_gradient(torch_dev, layout):
    """The call at negated positions is the gradient: <g, R x> = <R' g, x> for
    the formula's R, and by differences along random directions."""
    torch = torch_dev
    freq, amplitude = qdr.qdr_rotary_frequencies(qdr.ROTARY_TURNS, 96, 500.0, 2.0, 300.0, 1.0, 4.0)
    amplitude = 1.25
    rot = qdr.Rotary(freq, layout, amplitude)
    pos = [0, 3, 500, 70000, -9]
    g0 = torch.Generator("cuda").manual_seed(3)
    x, g, d = (torch.randn((len(pos), 3, D), generator=g0, device="cuda") for _ in range(3))
    back = torch.empty_like(x)
    rot.qdr_rotate(i32(torch, [-p for p in pos]), g, back)
    xr = x.double().requires_grad_()
    y, _ = turned(torch, xr, pos, freq, layout, amplitude)
    y.backward(g.double())
    _, e = turned(torch, g, [-p for p in pos], freq, layout, amplitude)
    assert ((back.double() - xr.grad).abs() <= e).all()
    # the map is linear, so a difference over a step of 1 has no error but the evaluations'
    y0, y1 = torch.empty_like(x), torch.empty_like(x)
    rot.qdr_rotate(i32(torch, pos), x, y0)
    rot.qdr_rotate(i32(torch, pos), x + d, y1)
    left = ((y1.double() - y0.double()) * g.double()).sum()
    right = (back.double() * ((x + d).double() - x.double())).sum()
    _, e0 = turned(torch, x, pos, freq, layout, amplitude)
    _, e1 = turned(torch, x + d, pos, freq, layout, amplitude)
    assert (left - right).abs() <= ((e0 + e1) * g.abs()).sum() + (e * ((x + d).double() - x.double()).abs()).sum()


WRITE = [
    # rows a sequence, contexts, page, query heads, heads
    ([1], [1], 32, 1, 1),
    ([1] * 6, [1, 32, 33, 1000, 4097, 64], 64, 8, 2),
    ([31, 0, 64, 5], [31, 9, 200, 5], 32, 3, 3),
    ([100, 33], [300, 33], 128, 40, 5),
    ([700], [1500], 1024, 4, 9),
    ([4500], [4600], 64, 6, 3),
]


@pytest.mark.parametrize("kind", [INT8, BF16])
@pytest.mark.parametrize("layout,channels", [(HALF, 128), (HALF, 48), (PAIRS, 128), (PAIRS, 32)])
@pytest.mark.parametrize("lens,contexts,page,q_heads,heads", WRITE, ids=str)
def test_write_rotary(torch_dev, kind, layout, channels, lens, contexts, page, q_heads, heads):
    torch = torch_dev
    freq, amplitude = qdr.qdr_rotary_frequencies(qdr.ROTARY_LINEAR, channels, 10000.0, 2.0)
    rot = qdr.Rotary(freq, layout, 1.1)
    pages, num = table(torch, contexts, page)
    cache = qdr.KVCache(num, page, heads, kind)
    old = [c - m if m else 0 for c, m in zip(contexts, lens)]
    k0, v0 = vectors(torch, 1, sum(old), heads), vectors(torch, 2, sum(old), heads)
    cache.qdr_kv_write(pages, counts(torch, old), i32(torch, old), k0, v0)
    lead, tail = 3, 2
    T = lead + sum(lens) + tail
    rows = slice(lead, lead + sum(lens))
    qkv = torch.cat([vectors(torch, 3, T, q_heads), vectors(torch, 4, T, heads), vectors(torch, 5, T, heads)], 1)
    q, k, v = qkv[:, :q_heads], qkv[:, q_heads:q_heads + heads], qkv[:, q_heads + heads:]
    cu, ctx = counts(torch, lens, lead), i32(torch, contexts)
    q_out = torch.full((T, q_heads, D), 7, dtype=torch.bfloat16, device="cuda")
    cache.qdr_kv_write_rotary(rot, pages, cu, ctx, k, v, q=q, q_out=q_out)
    assert cache.qdr_kv_poll_device_error() == 0
    pos = [p for m, c in zip(lens, contexts) for p in range(c - m, c)]
    assert (q_out[:lead] == 7).all() and (q_out[rows.stop:] == 7).all()
    both = torch.empty((len(pos), q_heads, D), dtype=torch.bfloat16, device="cuda")
    rot.qdr_rotate_bf16(i32(torch, pos), q[rows].contiguous(), both)
    assert torch.equal(q_out[rows], both)
    got = [torch.full((T, heads, D), 7, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    cache.qdr_kv_read(pages, cu, ctx, *got)
    assert torch.equal(got[1][rows], held(torch, v[rows], kind).bfloat16())
    ref, e = turned(torch, k[rows], pos, freq, layout, 1.1)
    room = 2.0 ** -8 * (ref.abs() + e) + e
    if kind == INT8:
        most = e.amax(-1, keepdim=True)
        scale = (ref.abs().amax(-1, keepdim=True) + most) / 127 * (1 + 2 * U)
        step = (0.5 + 2.0 ** -14) * scale + most
        room = 2.0 ** -8 * (ref.abs() + step) + step
    assert ((got[0][rows].double() - ref).abs() <= room).all()
    if kind == BF16:       # the same as turning first and writing then
        first = torch.empty_like(k[rows].contiguous())
        rot.qdr_rotate_bf16(i32(torch, pos), k[rows], first)
        assert torch.equal(got[0][rows], first)
    k1, v1 = torch.empty_like(k0), torch.empty_like(v0)
    cache.qdr_kv_read(pages, counts(torch, old), i32(torch, old), k1, v1)
    assert torch.equal(k1, held(torch, k0, kind).bfloat16()) and torch.equal(v1, held(torch, v0, kind).bfloat16())
    # without queries, and with the queries in place
    cache.qdr_kv_write_rotary(rot, pages, cu, ctx, k, v)
    again = [torch.full_like(x, 7) for x in got]
    cache.qdr_kv_read(pages, cu, ctx, *again)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    whole = q.contiguous()
    cache.qdr_kv_write_rotary(rot, pages, cu, ctx, k, v, q=whole, q_out=whole)
    assert torch.equal(whole[rows], q_out[rows]) and torch.equal(whole[:lead], q[:lead]) and torch.equal(whole[rows.stop:], q[rows.stop:])


def test_write_rotary_extremes(torch_dev):
    """Zero, the smallest and the largest keys, infinity and NaN (8-bit: the whole vector reads back as NaN)."""
    torch = torch_dev
    freq, _ = qdr.qdr_rotary_frequencies(qdr.ROTARY_PLAIN, 64)
    rot = qdr.Rotary(freq, HALF)
    k = torch.zeros((8, 1, D), device="cuda")
    k[1, 0, 3] = 2.0 ** -130
    k[2, 0, 3], k[2, 0, 100] = 2.0 ** -120, 2.0 ** -121
    k[3, 0, 3], k[3, 0, 100] = 1e38, -2e38
    k[4, 0, 9] = float("inf")
    k[5, 0, 110] = float("nan")
    k[6, 0] = torch.linspace(-1, 1, D, device="cuda")
    k[7, 0, 3] = k[7, 0, 35] = 3.3e38       # the turned value leaves the range
    k = k.bfloat16()
    v = vectors(torch, 1, 8, 1)
    for kind in (INT8, BF16):
        cache = qdr.KVCache(1, 32, 1, kind)
        pages, cu, ctx = i32(torch, [[0]]), i32(torch, [0, 8]), i32(torch, [17])
        cache.qdr_kv_write_rotary(rot, pages, cu, ctx, k, v)
        a, b = torch.empty_like(k), torch.empty_like(v)
        cache.qdr_kv_read(pages, cu, ctx, a, b)
        assert torch.equal(b, held(torch, v, kind).bfloat16())
        ref, e = turned(torch, k, list(range(9, 17)), freq, HALF)
        some = [0, 2, 3, 6]
        scale = ref[some].abs().amax(-1, keepdim=True) / 127 if kind == INT8 else 0
        assert ((a[some].double() - ref[some]).abs() <= 2.0 ** -8 * ref[some].abs() + 0.52 * scale + e[some].amax(-1, keepdim=True)).all()
        if kind == INT8:
            assert (a[1] == 0).all() and a[4:6].isnan().all()
            over = (ref[7].abs() > 3.4028236e38).any()
            assert a[7].isnan().all() if over else torch.isfinite(a[7]).all()
        else:
            assert a[5, 0, 110].isnan() and torch.isfinite(a[5, 0, :110]).all() and not torch.isfinite(a[4, 0, [9, 41]]).all()


@pytest.mark.parametrize("kind", [INT8, BF16])
def test_write_rotary_bad_pages_and_counts(torch_dev, kind):
    torch = torch_dev
    H, Q, page = 2, 4, 32
    freq, _ = qdr.qdr_rotary_frequencies(qdr.ROTARY_PLAIN, 128)
    rot = qdr.Rotary(freq, HALF)
    cache = qdr.KVCache(3, page, H, kind)
    x, y, q = vectors(torch, 1, 70, H), vectors(torch, 2, 70, H), vectors(torch, 3, 70, Q)
    good, cu, ctx = i32(torch, [[0, 1, 2]]), i32(torch, [0, 70]), i32(torch, [70])
    cache.qdr_kv_write(good, cu, ctx, x, x)
    ref = torch.empty_like(q)
    rot.qdr_rotate_bf16(torch.arange(70, dtype=torch.int32, device="cuda"), q, ref)
    out = torch.full_like(q, 7)
    cache.qdr_kv_write_rotary(rot, i32(torch, [[-1, 3, 2 ** 31 - 1]]), cu, ctx, y, y, q=q, q_out=out)
    assert cache.qdr_kv_poll_device_error() == qdr.DEVERR_PAGE and torch.equal(out, ref)
    for c, t in (([0, 70], [69]), ([0, 70], [97]), ([0, 70], [-5]), ([0, 71], [71]), ([-1, 70], [71]), ([5, 3], [70])):
        out.fill_(7)
        cache.qdr_kv_write_rotary(rot, good, i32(torch, c), i32(torch, t), y, y, q=q, q_out=out)
        assert cache.qdr_kv_poll_device_error() == qdr.DEVERR_LENGTH, (c, t)
        if c == [0, 70]:
            assert (out == 0).all()
    k, v = torch.empty_like(x), torch.empty_like(x)
    cache.qdr_kv_read(good, cu, ctx, k, v)
    assert torch.equal(k, held(torch, x, kind).bfloat16()) and torch.equal(v, held(torch, x, kind).bfloat16())


def test_rotary_refusals(torch_dev):
    torch = torch_dev
    freq, _ = qdr.qdr_rotary_frequencies(qdr.ROTARY_PLAIN, 64)
    rot = qdr.Rotary(freq)
    x, p = torch.zeros((5, 2, D), device="cuda"), i32(torch, [0] * 5)
    for args, kind in (((p[:4], x, x), ValueError), ((p.long(), x, x), TypeError), ((p, x.half(), x), TypeError), ((p, x, x[:4]), ValueError),
                       ((p, x, x[:, :1]), ValueError), ((p, x[..., :64], x[..., :64]), ValueError),
                       ((p, x.transpose(0, 1).contiguous().transpose(0, 1), x), ValueError),
                       ((p, x[:1].expand(5, 2, D), x), qdr.QdrError)):
        with pytest.raises(kind):
            rot.qdr_rotate(*args)
    b = torch.zeros(5 * 257, dtype=torch.bfloat16, device="cuda")
    odd = b.as_strided((5, 2, D), (257, D, 1))
    even = torch.zeros((5, 2, D), dtype=torch.bfloat16, device="cuda")
    for args in ((p, odd, even), (p, even, odd), (p, b[1:1281].view(5, 2, D), even)):
        with pytest.raises(qdr.QdrError):
            rot.qdr_rotate_bf16(*args)
    rot.qdr_rotate(p[:0], x[:0], x[:0])
    cache = qdr.KVCache(2, 32, 2, INT8)
    pages, cu, ctx = i32(torch, [[0, 1]]), i32(torch, [0, 5]), i32(torch, [5])
    for kw, kind in ((dict(k=odd, v=even), qdr.QdrError), (dict(k=even, v=even[:4]), ValueError), (dict(k=even[:, :1], v=even), ValueError),
                     (dict(k=even, v=even, q=even), TypeError), (dict(k=even, v=even, q=even, q_out=even[:, :1]), ValueError),
                     (dict(k=even.float(), v=even), TypeError)):
        with pytest.raises((kind, AttributeError) if kind is TypeError else kind):
            cache.qdr_kv_write_rotary(rot, pages, cu, ctx, **kw)
    assert cache.qdr_kv_poll_device_error() == 0
