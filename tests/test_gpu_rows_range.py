"""Row operators at the ends of their arguments' ranges.

Floats are held to the tolerance that test_gpu_rows.py derives, with distances from the row's
maximum in units of the temperature: the derivation uses nothing else of the logits.
"""
import numpy as np
import pytest
import torch

import top_selection_amd as ts
from oracle import rows as orc
from test_gpu_rows import DT, _close, _gen, _np

pytestmark = pytest.mark.gpu

# rows, n: each row kernel (256 and 1024 threads, of 4 and 8 vectors, with several workgroups a row and
# with one; more vectors, and elements past those that a workgroup keeps) and rows in slices
SHAPES = {"fp32": [(9, 1000), (9, 5001), (9, 12003), (27, 30001), (5, 30001), (70, 30001), (9, 140003), (50, 130001)],
          "bf16": [(9, 2000), (9, 12003), (9, 30001), (27, 50001), (5, 50001), (70, 50001), (9, 140003), (50, 140003)]}
EACH = [(d, s) for d in SHAPES for s in SHAPES[d]]


@pytest.mark.parametrize("dtype,shape", EACH)
@pytest.mark.parametrize("mask", [-1e10, -1e30, "lowest"])
def test_softmax_finite_masks(dtype, shape, mask):
    """Masks that are large finite numbers: the row's tail, all but a few places, or its first half."""
    rows, n = shape
    low = torch.finfo(DT[dtype]).min if mask == "lowest" else mask
    x = 2 * torch.randn(rows, n, generator=_gen(n))
    x[::3, n // 2:] = low
    x[1::3] = low
    x[1::3, [0, n // 3, n - 1]] = torch.tensor([-1.0, 0.5, 1.0])
    x[2::3, :n // 2] = low
    x = x.to(DT[dtype])
    t = 0.3 + torch.rand(rows, generator=_gen(rows))
    for temp in (None, t):
        p = ts.ds_softmax(x.cuda(), temperature=None if temp is None else temp.cuda())
        _close(p, orc.softmax(_np(x), None if temp is None else _np(temp)), f"softmax {shape} {dtype} {mask} {temp is None}")
