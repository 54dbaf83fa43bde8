"""qdr_kv_assign where a row runs out of pages that another would share a page with."""
import pytest

from quantized_delta_rule_decode_amd import qdr
from test_gpu_kv import BF16, INT8, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", [INT8, BF16])
@pytest.mark.parametrize("fill", [0, 300])
def test_a_row_that_runs_out_counts_as_one_that_keeps(kind, fill):
    """Row 0 keeps page 1 as a full one and runs out; row 1 keeps it in part, wants a
    copy for that, and runs out too.  Without row 0, or where it fits, row 1 has what it asks for."""
    import torch
    with qdr.KVCache(8, 32, 2, kind) as cache:
        old, context = i32(torch, [[0, 1, -1, -1, -1, -1, -1, -1]]), i32(torch, [64])
        # (rows that begin and are empty: the same by the launch that more rows have)
        for parent, add, refs, tables, after, held, err in (
                ([0, 0], [96, -20], [1] * 7 + [0], [[], []], [0, 0], [0, 0] + [1] * 5 + [0], qdr.DEVERR_FULL),
                ([-1, 0], [0, -20], [1] * 7 + [0], [[], [0, 1]], [0, 44], [1] * 7 + [0], 0),
                ([0, 0], [96, -20], [1, 1, 1, 0, 0, 0, 0, 1], [[0, 1, 3, 4, 5], [0, 6]], [160, 44], [2, 1, 1, 1, 1, 1, 1, 1], 0)):
            m = len(parent) + fill
            new = [torch.full((m, 8), 9, dtype=torch.int32, device="cuda"), torch.full((m,), 9, dtype=torch.int32, device="cuda"), torch.full((8,), 9, dtype=torch.int32, device="cuda")]
            cache.qdr_kv_assign(old, context, i32(torch, parent + [-1] * fill), i32(torch, add + [0] * fill), i32(torch, refs), *new)
            assert new[0][:2].tolist() == [x + [-1] * (8 - len(x)) for x in tables] and (new[0][2:] == -1).all()
            assert new[1].tolist() == after + [0] * fill and new[2].tolist() == held
            assert cache.qdr_kv_poll_device_error() == err
