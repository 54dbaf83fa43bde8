"""Edges of qdr_kv_attend_shared."""
import numpy as np
import pytest

from quantized_delta_rule_decode_amd import qdr
from test_gpu_kv import BF16, INT8, i32
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
