"""The operators behind a router on the GPU at the ends of their ranges: broken plans, guard rows around outputs,
the choice of sums, and sizes at which each tile of ds_block_product is chosen. Tolerances as in
test_gpu_experts.py, where the definitions' helpers are from."""
import ctypes

import numpy as np
import pytest
import torch

import top_selection_amd as ts
from gpu_util import say
from oracle import experts as orc
from test_gpu_experts import E8, KEPT, _np

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [ts.BF16, ts.FP32])
@pytest.mark.parametrize("n", [64, 100])
@pytest.mark.parametrize("end", [128, 256, 2 ** 31 - 1])
def test_columns_of_a_plan_without_rows(dtype, n, end):
    """No row, so no x, and offsets that say otherwise: every position below the (clamped) end is padding."""
    say(f"columns of no rows, n {n}, end {end}")
    cap, experts = 384, 3
    i32 = dict(dtype=torch.int32, device="cuda")
    place, order = torch.zeros(4, **i32), torch.arange(cap, **i32)
    offsets = torch.tensor([0, 128, 128, end], **i32)
    plan = ts._binding.ds_expert_plan(place.data_ptr(), order.data_ptr(), offsets.data_ptr(), 0, cap, 8, experts, 128)
    q = torch.full((n, cap), 2.0, device="cuda").to(E8["e4m3"])
    s = torch.full((n, cap // 128), KEPT, device="cuda")
    torch.cuda.synchronize()
    st = ts.lib().ds_block_quantize(None, 0, n, n, dtype, ts.BLOCK_COLUMN, ctypes.byref(plan), q.data_ptr(), cap, ts.E4M3,
                                    s.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert st == 0
    torch.cuda.synchronize()
    end = min(end, cap)
    assert (_np(q.float())[:, :end] == 0).all() and (_np(q.float())[:, end:] == 2).all()
    least = np.float32(orc.LEAST) / np.float32(orc.LARGEST["e4m3"])
    assert (_np(s)[:, :end // 128] == least).all() and (_np(s)[:, end // 128:] == KEPT).all()
