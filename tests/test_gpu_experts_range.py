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


@pytest.mark.parametrize("padding", [100, 5])
def test_sort_next_to_the_largest_position(padding):
    """As many slots of one expert as 2^31 - 2 positions hold: neither the padded count nor the walk through the padding
    may pass 2^31 - 1 on the way."""
    rows, align = 2 ** 31 - 2 - padding, 126
    say(f"sort of {rows} slots")
    cap = ts.ds_expert_capacity(rows, 1, 1, align)
    assert cap == 2 ** 31 - 2
    idx = torch.zeros(rows, 1, dtype=torch.int32, device="cuda")
    plan = ts.ds_expert_sort(idx, 1, align)
    del idx
    assert _np(plan.offsets).tolist() == [0, cap]
    assert (plan.order[rows:] == -1).all()
    for lo in range(0, rows, 2 ** 28):
        hi = min(rows, lo + 2 ** 28)
        want = torch.arange(lo, hi, dtype=torch.int32, device="cuda")
        assert torch.equal(plan.place[lo:hi, 0], want) and torch.equal(plan.order[lo:hi], want)
    del plan, want
    torch.cuda.empty_cache()
