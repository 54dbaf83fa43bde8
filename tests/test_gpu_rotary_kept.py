"""Channels that a rotation does not turn stay as they are, bit for bit: also
bfloat16 NaN that a conversion to fp32 and back would quiet (0x7F81, 0xFFBF)."""
import pytest

from quantized_delta_rule_decode_amd import qdr
from test_gpu_kv import BF16, D, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch_dev():
    import torch
    assert torch.cuda.is_available(), "device tests need a HIP GPU"
    qdr.load()
    return torch


def rows(torch, T, heads, channels):
    """[T][heads][128] whose channels from `channels` on hold NaN, infinities and others."""
    x = torch.randn((T, heads, D), generator=torch.Generator("cuda").manual_seed(4), device="cuda").bfloat16()
    bits = x.view(torch.int16)
    kept = bits[..., channels:]
    odd = torch.tensor([0x7F81, 0xFFBF - 65536, 0x7FC0, 0xFFFF - 65536, 0x7F80, 0x8001 - 65536, 1, 0x3F80], dtype=torch.int16, device="cuda")
    kept.copy_(odd[torch.arange(kept.numel(), device="cuda") % 8].view(kept.shape))
    return x, kept.clone()


@pytest.mark.parametrize("layout", [qdr.ROTARY_HALF, qdr.ROTARY_PAIRS])
@pytest.mark.parametrize("channels", [16, 48, 64, 80, 112])
@pytest.mark.parametrize("T,heads", [(1, 1), (45, 3), (2, 130)])
def test_rotate(torch_dev, layout, channels, T, heads):
    torch = torch_dev
    rot = qdr.Rotary(qdr.qdr_rotary_frequencies(qdr.ROTARY_PLAIN, channels)[0], layout, 1.5)
    x, kept = rows(torch, T, heads, channels)
    pos = i32(torch, list(range(3, T + 3)))
    y = torch.empty_like(x)
    rot.qdr_rotate_bf16(pos, x, y)
    assert torch.equal(y.view(torch.int16)[..., channels:], kept)
    assert y[..., :channels].isfinite().all() and not torch.equal(y[..., :channels], x[..., :channels])
    f, g = x.view(torch.int16).int().bitwise_left_shift(16).view(torch.float32).clone(), torch.empty((T, heads, D), device="cuda")
    rot.qdr_rotate(pos, f, g)
    assert torch.equal(g.view(torch.int32)[..., channels:], f.view(torch.int32)[..., channels:])


@pytest.mark.parametrize("layout", [qdr.ROTARY_HALF, qdr.ROTARY_PAIRS])
@pytest.mark.parametrize("channels", [16, 48, 64, 80, 112])
def test_write_rotary(torch_dev, layout, channels):
    """Keys in a bfloat16 cache, and the queries beside them."""
    torch, T, heads, page = torch_dev, 41, 2, 32
    rot = qdr.Rotary(qdr.qdr_rotary_frequencies(qdr.ROTARY_PLAIN, channels)[0], layout, 1.5)
    x, kept = rows(torch, T, heads, channels)
    with qdr.KVCache(2, page, heads, BF16) as cache:
        pages, cu, context = i32(torch, [[1, 0]]), i32(torch, [0, T]), i32(torch, [T])
        q, k, v = (torch.empty_like(x) for _ in range(3))
        cache.qdr_kv_write_rotary(rot, pages, cu, context, x, x, q=x, q_out=q)
        cache.qdr_kv_read(pages, cu, context, k, v)
        assert torch.equal(q.view(torch.int16)[..., channels:], kept)
        assert torch.equal(k.view(torch.int16)[..., channels:], kept)
        assert torch.equal(v.view(torch.int16), x.view(torch.int16)) and torch.equal(k[..., :channels], q[..., :channels])
        assert cache.qdr_kv_poll_device_error() == 0
