"""The operators behind a router on the GPU against their 64-bit definitions (oracle/experts.py).

Integers, gathered bits, scales and 8-bit values have to be equal. Tolerances of the others, in units of
u = 2^-24, half a step of fp32 (bf16 results add half a step of bf16, 2^-8 relative):
  * combine: k fused multiply-adds, each off by u of a sum that the terms' magnitudes bound: k u of those.
  * the rows' gradient is one product: u (fp32), then the rounding to bf16.
  * the weights' gradient: a lane adds at most n / 64 + 16 products and 8 sums join them: (n / 64 + 24) u of
    the products' magnitudes.
  * products: 128 exact products of a block are added by the matrix unit in an order and with a rounding of
    its own, at most one step (2 u) of the magnitudes' sum for each addition: 256 u; the block's scale is a
    product (u), the blocks' sum adds u a block and the joining of 16 partial sums 16 u: (273 + blocks) u of
    the scaled magnitudes' sum. With a bf16 result the 8-bit unit may add: eight products at a time, each cut
    below 2^-13 of the largest one's leading bit (a power of two that 2^-13 of the largest product bounds), the
    largest itself not: at most 7 * 2^-13 < 2^-10 of the magnitudes' sum.
"""
import numpy as np
import pytest
import torch

import top_selection_amd as ts
from gpu_util import say
from oracle import experts as orc

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
E8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
KEPT = 77.0  # what outputs hold where nothing is written


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _np(t):
    t = t.detach().cpu()
    return t.double().numpy() if t.is_floating_point() else t.numpy()


def _choices(seed, rows, k, experts, dropped=0.1, hot=False):
    g = _gen(seed)
    idx = torch.randint(0, experts, (rows, k), generator=g, dtype=torch.int32)
    if hot:
        idx[torch.rand(rows, k, generator=g) < 0.7] = experts // 2
    if dropped:
        gone = torch.rand(rows, k, generator=g) < dropped
        idx[gone] = torch.where(torch.rand(rows, k, generator=g) < 0.5, -1, experts + 3)[gone].to(torch.int32)
    return idx


def _made(seed, rows, k, experts, align, dropped=0.1, hot=False):
    """A plan on the device and its arrays."""
    idx = _choices(seed, rows, k, experts, dropped, hot)
    plan = ts.ds_expert_sort(idx.cuda(), experts, align)
    return plan, _np(plan.place), _np(plan.order), _np(plan.offsets)


def _wide(t, pad, shift=0):
    """The same matrix on the device with rows `pad` elements longer and its start shifted."""
    rows, n = t.shape
    base = torch.full((rows * (n + pad) + shift + 8,), KEPT, dtype=t.dtype if t.element_size() > 1 else torch.float32)
    v = base.to(t.dtype).cuda()[shift:shift + rows * (n + pad)].view(rows, n + pad)[:, :n] if rows else t.cuda()
    v.copy_(t)
    return v


def _close(got, want, tol, label):
    got = _np(got)
    assert got.shape == want.shape, label
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{label}: {bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}: " \
                          f"{got[bad][0]} for {want[bad][0]}, allowed {np.broadcast_to(tol, bad.shape)[bad][0]}"


def _half(dtype, want):
    return 2.0 ** -8 * np.abs(want) + 2.0 ** -133 if dtype in ("bf16", torch.bfloat16) else 0


# ------------------------------------------------------------------------------------------ sort
@pytest.mark.parametrize("rows,k,experts", [
    (0, 8, 16), (1, 1, 1), (1, 64, 1024), (4, 8, 256), (31, 3, 5), (128, 8, 60), (1024, 8, 256), (1025, 8, 256),
    (2000, 6, 1000), (9001, 7, 129), (70000, 8, 256), (40000, 3, 1024)])
@pytest.mark.parametrize("align,dropped,hot", [(1, 0.0, False), (16, 0.1, True), (128, 0.5, False), (100, 1.0, False)])
def test_sort(rows, k, experts, align, dropped, hot):
    say(f"sort {rows} x {k} of {experts}, align {align}")
    idx = _choices(rows + align, rows, k, experts, dropped, hot)
    plan = ts.ds_expert_sort(idx.cuda(), experts, align)
    cap = ts.ds_expert_capacity(rows, k, experts, align)
    place, order, offsets = orc.sort(idx.numpy(), experts, align, cap)
    assert np.array_equal(_np(plan.offsets), offsets)
    assert np.array_equal(_np(plan.place), place)
    assert np.array_equal(_np(plan.order), order)


@pytest.mark.parametrize("rows,k,experts,align", [(400000, 8, 300, 128), (200000, 6, 1023, 1), (100, 64, 2, 16)])
def test_sort_of_many_and_of_equal_slots(rows, k, experts, align):
    """More slots than 256 chunks of 4096; an expert that fills most slots of every row."""
    say(f"sort many {rows} x {k} of {experts}")
    idx = _choices(rows, rows, k, experts, 0.05, hot=True)
    plan = ts.ds_expert_sort(idx.cuda(), experts, align)
    for got, want in zip(plan, orc.sort(idx.numpy(), experts, align, plan.order.numel())):
        assert np.array_equal(_np(got), want)


def test_sort_into_longer_arrays_and_a_dirty_workspace():
    say("sort into given arrays")
    idx = _choices(3, 20000, 4, 77).cuda()
    cap = ts.ds_expert_capacity(20000, 4, 77, 32) + 1000
    i32 = dict(dtype=torch.int32, device="cuda")
    out = ts.ExpertPlan(torch.full((20000, 4), 9, **i32), torch.full((cap,), 9, **i32), torch.full((78,), 9, **i32), 32)
    ws = torch.randint(0, 255, (ts.ds_expert_sort_workspace_size(20000, 4, 77),), dtype=torch.uint8, device="cuda")
    for _ in range(2):
        ts.ds_expert_sort(idx, 77, 32, out=out, workspace=ws)
        for got, want in zip(out, orc.sort(_np(idx), 77, 32, cap)):
            assert np.array_equal(_np(got), want)


# ------------------------------------------------------------------------ gather, combine, gradient
SHAPES = [(1, 1, 1, 1, 1), (3, 2, 4, 1, 7), (5, 8, 16, 16, 8), (4, 8, 256, 1, 2048), (40, 6, 9, 128, 33),
          (64, 3, 5, 100, 257), (33, 8, 8, 1, 1000), (130, 4, 31, 16, 1025), (9, 64, 64, 1, 515), (17, 2, 3, 128, 4096),
          (6, 3, 4, 1, 9001), (3, 2, 4, 16, 20011), (300, 1, 7, 1, 64)]


@pytest.mark.parametrize("rows,k,experts,align,n", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_gather(rows, k, experts, align, n, dtype):
    say(f"gather {rows} x {k} of {experts}, align {align}, n {n}, {dtype}")
    plan, place, order, offsets = _made(n, rows, k, experts, align)
    x = torch.randn(rows, n, generator=_gen(n)).to(DT[dtype])
    x[0, 0] = float("nan")
    x[-1, -1] = float("-inf")
    out = _wide(torch.full((order.size, n), KEPT, dtype=DT[dtype]), 3, 1)
    assert ts.ds_expert_gather(_wide(x, 5, 1), plan, out=out) is out
    bits = torch.int16 if dtype == "bf16" else torch.int32
    want = orc.gather(x.view(bits).numpy(), place, offsets,
                      torch.full((order.size, n), KEPT, dtype=DT[dtype]).view(bits).numpy())
    assert np.array_equal(out.contiguous().cpu().view(bits).numpy(), want)
    again = ts.ds_expert_gather(x.cuda(), plan).cpu().view(bits).numpy()
    assert np.array_equal(again[:offsets[-1]], want[:offsets[-1]])


@pytest.mark.parametrize("rows,k,experts,align,n", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("weighted", [True, False])
def test_combine(rows, k, experts, align, n, dtype, weighted):
    say(f"combine {rows} x {k} of {experts}, align {align}, n {n}, {dtype}, {weighted}")
    plan, place, order, offsets = _made(n, rows, k, experts, align)
    y = torch.randn(order.size, n, generator=_gen(n)).to(DT[dtype])
    y[torch.from_numpy(order) < 0] = float("nan")  # padding and what lies behind is not looked at
    w = torch.randn(rows, k, generator=_gen(n + 1))
    w[torch.from_numpy(place) < 0] = float("nan")  # neither are the weights of slots without a position
    out = ts.ds_expert_combine(_wide(y, 3, 1), plan, w.cuda() if weighted else None,
                               out=_wide(torch.zeros(rows, n, dtype=DT[dtype]), 7, 1))
    want, size = orc.combine(_np(y), place, w.double().numpy() if weighted else None)
    _close(out, want, k * U * size + _half(dtype, want), "combine")


def test_combine_of_infinite_and_missing_values():
    say("combine inf")
    plan, place, order, _ = _made(3, 6, 2, 4, 1, dropped=0)
    y = torch.randn(order.size, 40, generator=_gen(1))
    y[place[1, 0]] = float("inf")
    y[place[2, 1]] = float("nan")
    w = torch.ones(6, 2)
    w[3] = 0
    got = _np(ts.ds_expert_combine(y.cuda(), plan, w.cuda()))
    assert np.isposinf(got[1]).all() and np.isnan(got[2]).all() and (got[3] == 0).all()
    assert np.isfinite(got[[0, 4, 5]]).all()


@pytest.mark.parametrize("rows,k,experts,align,n", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("weighted", [True, False])
def test_combine_grad(rows, k, experts, align, n, dtype, weighted):
    say(f"combine grad {rows} x {k} of {experts}, align {align}, n {n}, {dtype}, {weighted}")
    plan, place, order, offsets = _made(n, rows, k, experts, align)
    g = torch.randn(rows, n, generator=_gen(n)).to(DT[dtype])
    y = torch.randn(order.size, n, generator=_gen(n + 1)).to(DT[dtype])
    y[torch.from_numpy(order) < 0] = float("nan")
    w = torch.randn(rows, k, generator=_gen(n + 2))
    w[torch.from_numpy(place) < 0] = float("nan")
    wd = w.cuda() if weighted else None
    kept = torch.full((order.size, n), KEPT, dtype=DT[dtype])
    want_y, want_w, size = orc.combine_grad(_np(g), _np(torch.nan_to_num(y)), place,
                                            w.double().numpy() if weighted else None, offsets, _np(kept))
    gd, yd = _wide(g, 1, 1), _wide(y, 3, 1)
    got_y, got_w = ts.ds_expert_combine_grad(gd, yd, plan, wd, out_y=_wide(kept, 5, 1))
    tol_y = U * np.abs(want_y) + _half(dtype, want_y)
    tol_w = (n / 64 + 24) * U * size
    _close(got_y, want_y, tol_y, "rows")
    _close(got_w, want_w, tol_w, "weights")
    # each alone, and over y itself
    only_w = ts.ds_expert_combine_grad(gd, yd, plan, wd, grad_y=False)
    assert only_w[0] is None and torch.equal(only_w[1], got_w)
    only_y = ts.ds_expert_combine_grad(gd, None, plan, wd, grad_weights=False, out_y=_wide(kept, 2))
    assert only_y[1] is None and torch.equal(only_y[0], got_y)
    over = ts.ds_expert_combine_grad(gd, yd, plan, wd, out_y=yd)
    assert over[0] is yd and torch.equal(over[1], got_w)
    assert torch.equal(yd[:offsets[-1]], got_y[:offsets[-1]])
    assert torch.equal(yd[offsets[-1]:].isnan().cpu(), y[offsets[-1]:].isnan())


def test_gradients_are_those_of_differences():
    """Central differences of the definitions in 64 bits."""
    say("differences")
    rows, k, n = 5, 3, 11
    plan, place, order, offsets = _made(7, rows, k, 4, 8)
    g, y = torch.randn(rows, n, generator=_gen(1)), torch.randn(order.size, n, generator=_gen(2))
    w, x = torch.randn(rows, k, generator=_gen(3)), torch.randn(rows, n, generator=_gen(4))
    grad_y, grad_w = ts.ds_expert_combine_grad(g.cuda(), y.cuda(), plan, w.cuda())
    gy = torch.randn(order.size, n, generator=_gen(5))
    gy[offsets[-1]:] = 0
    grad_x = ts.ds_expert_combine(gy.cuda(), plan)
    h, f = 2.0 ** -10, {}
    f["y"] = lambda v: (orc.combine(v, place, w.double().numpy())[0] * g.double().numpy()).sum()
    f["w"] = lambda v: (orc.combine(y.double().numpy(), place, v)[0] * g.double().numpy()).sum()
    f["x"] = lambda v: (orc.gather(v, place, offsets, np.zeros((order.size, n))) * gy.double().numpy()).sum()
    live = order >= 0
    for name, at, got in (("y", y, grad_y), ("w", w, grad_w), ("x", x, grad_x)):
        got, v = _np(got), at.double().numpy()
        for i in np.ndindex(*v.shape):
            if name == "y" and not live[i[0]]:
                continue
            up, down = v.copy(), v.copy()
            up[i] += h
            down[i] -= h
            slope = (f[name](up) - f[name](down)) / (2 * h)
            # the functions are linear in each: differences are exact up to 64-bit rounding
            assert abs(got[i] - slope) < 2.0 ** -18 * max(1, abs(slope)) * n, (name, i)


@pytest.mark.parametrize("rows", [0, 3])
def test_no_row_and_no_slot(rows):
    say(f"no slot, {rows} rows")
    plan = ts.ds_expert_sort(torch.full((rows, 2), -1, dtype=torch.int32, device="cuda"), 4, 16)
    cap = plan.order.numel()
    assert _np(plan.offsets).max() == 0
    x = torch.randn(rows, 9, device="cuda")
    out = torch.full((cap, 9), KEPT, device="cuda")
    assert (ts.ds_expert_gather(x, plan, out=out) == KEPT).all()
    assert (ts.ds_expert_combine(out, plan) == 0).all()
    gy, gw = ts.ds_expert_combine_grad(x, out, plan, out_y=out.clone())
    assert (gy == KEPT).all() and (gw == 0).all()
    q = torch.full((cap, 16), 1.0, device="cuda").to(torch.float8_e4m3fn)
    q, s = ts.ds_block_quantize(x, plan=plan, out=q, out_scales=torch.full((cap, 1), KEPT, device="cuda"))
    assert (q.float() == 1).all() and (s == KEPT).all()


def test_far_offsets():
    """Rows 2^27 elements apart: offsets past 32 bits in elements and bytes."""
    say("far offsets")
    rows, k, n, step = 9, 3, 130, 1 << 27
    plan, place, order, offsets = _made(2, rows, k, 4, 1, dropped=0)
    far = torch.empty((order.size - 1) * step + n, dtype=torch.bfloat16, device="cuda")
    out = far.as_strided((order.size, n), (step, 1))
    x = torch.randn(rows, n, generator=_gen(1)).bfloat16()
    ts.ds_expert_gather(x.cuda(), plan, out=out)
    assert torch.equal(out.cpu(), x[torch.from_numpy(order // k).long()])
    want, size = orc.combine(_np(out), place, None)
    _close(ts.ds_expert_combine(out, plan), want, k * U * size + _half("bf16", want), "combine")
    g = torch.randn(rows, n, generator=_gen(2)).bfloat16()
    _, gw = ts.ds_expert_combine_grad(g.cuda(), out, plan)
    _, want_w, size = orc.combine_grad(_np(g), _np(out), place, None, offsets, np.zeros((order.size, n)))
    _close(gw, want_w, (n / 64 + 24) * U * size, "weights")
    assert torch.equal(out.cpu(), x[torch.from_numpy(order // k).long()])
    q = far[:(4 * step - 16) // 2].view(torch.float8_e4m3fn).as_strided((3, 144), (step, 1))
    w = torch.randn(3, n, generator=_gen(3))
    got, s = ts.ds_block_quantize(w.cuda(), out=q)
    want_q, want_s = orc.quantize(w.numpy(), 1, "e4m3")
    assert np.array_equal(_np(got.float())[:, :n], want_q) and np.array_equal(_np(s), want_s)
    b, sb = ts.ds_block_quantize(w.cuda())
    assert torch.equal(ts.ds_block_product(q, s, b, sb), ts.ds_block_product(b, sb, b, sb))
    # (rows 2^24 bytes apart are past the tiles' 32-bit offsets)
    step = 1 << 24
    many = far.view(torch.uint8)[:299 * step + 144].view(torch.float8_e4m3fn).as_strided((300, 144), (step, 1))
    w = torch.randn(300, n, generator=_gen(4)).cuda()
    got, s = ts.ds_block_quantize(w, out=many)
    b, sb = ts.ds_block_quantize(w)
    assert torch.equal(got.view(torch.uint8), b.view(torch.uint8)) and torch.equal(s, sb)
    assert torch.equal(ts.ds_block_product(many, s, many, s, out_dtype=torch.float32),
                       ts.ds_block_product(b, sb, b, sb, out_dtype=torch.float32))


def test_broken_plans_stay_in_bounds():
    """Positions, slots and offsets out of range are skipped or clamped."""
    say("broken plans")
    rows, k, experts, align, n = 12, 3, 5, 16, 70
    plan, place, order, offsets = _made(1, rows, k, experts, align, dropped=0)
    bad = ts.ExpertPlan(plan.place.clone(), plan.order.clone(), plan.offsets.clone(), align)
    bad.place[::2] = 2 ** 31 - 1
    bad.place[1::4] = -5
    bad.order[::3] = 2 ** 31 - 1
    bad.order[1::7] = -9
    bad.offsets[-1] = 2 ** 31 - 1
    bad.offsets[0] = -7
    x, y = torch.randn(rows, n, device="cuda"), torch.randn(order.size, n, device="cuda")
    ts.ds_expert_gather(x, bad)
    got = ts.ds_expert_combine(y, bad)
    keep = np.where((_np(bad.place) >= 0) & (_np(bad.place) < order.size), _np(bad.place), -1)
    want, size = orc.combine(_np(y), keep, None)
    _close(got, want, k * U * size, "combine")
    ts.ds_expert_combine_grad(x, y, bad)
    ts.ds_block_quantize(x, plan=bad)
    wide = ts.ds_expert_sort(torch.randint(0, 5, (40, 3), dtype=torch.int32, device="cuda"), 5, 128)
    wide.offsets[-1] = 2 ** 31 - 1
    wide.order[5:90] = 2 ** 30
    ts.ds_block_quantize(torch.randn(40, n, device="cuda"), ts.BLOCK_COLUMN, plan=wide)
    a, sa = ts.ds_block_quantize(y)
    b, sb = ts.ds_block_quantize(torch.randn(experts, 20, n, device="cuda"), ts.BLOCK_TILE)
    ts.ds_block_product(a, sa, b, sb, offsets=torch.tensor([-4, 90, 20, 2 ** 31 - 1, 7, -3], dtype=torch.int32).cuda())
    t, st = ts.ds_block_quantize(y, ts.BLOCK_COLUMN)
    ts.ds_block_product(t, st, t, st, offsets=torch.tensor([-4, 90, 20, 2 ** 31 - 1, 7], dtype=torch.int32).cuda(),
                        inner=True)
    torch.cuda.synchronize()


# --------------------------------------------------------------------------------------- quantize
def _blocks_input(seed, rows, n, dtype):
    g = _gen(seed)
    x = torch.randn(rows, n, generator=g) * torch.exp(2 * torch.randn(n, generator=g))
    x[torch.rand(rows, n, generator=g) < 0.05] = 0
    return x.to(DT[dtype])


def _quantized(x, layout, to, plan=None, place=None, order=None, offsets=None):
    """The definition's values and scales for a layout, rows from the plan's end on left out."""
    v = x.float().numpy()
    if plan is not None:
        v = orc.gather(v, place, offsets, np.zeros((order.size, v.shape[1]), np.float32))[:offsets[-1]]
    if layout == ts.BLOCK_COLUMN:
        v = np.ascontiguousarray(v.T)
    return orc.quantize(v, 128 if layout == ts.BLOCK_TILE else 1, to)


@pytest.mark.parametrize("rows,n", [(1, 1), (3, 16), (7, 127), (128, 128), (130, 129), (5, 1000), (257, 300), (64, 4096)])
@pytest.mark.parametrize("dtype,to", [("bf16", "e4m3"), ("fp32", "e4m3"), ("bf16", "e5m2"), ("fp32", "e5m2")])
@pytest.mark.parametrize("layout", [0, 1, 2])
def test_quantize(rows, n, dtype, to, layout):
    say(f"quantize {rows} x {n} {dtype} to {to}, layout {layout}")
    x = _blocks_input(rows + n, rows, n, dtype)
    want, want_s = _quantized(x, layout, to)
    wide = -(-want.shape[1] // 16) * 16
    # an output with longer rows, whose rest stays as it was
    base = torch.full((want.shape[0], wide + 32), 2.0, device="cuda").to(E8[to])
    q, s = ts.ds_block_quantize(_wide(x, 3, 1), layout, dtype=E8[to], out=base[:, :wide])
    got = _np(base.float())
    assert np.array_equal(_np(s), want_s)
    assert np.array_equal(got[:, :want.shape[1]], want)
    assert (got[:, want.shape[1]:wide] == 0).all() and (got[:, wide:] == 2).all()
    again, s2 = ts.ds_block_quantize(x.cuda(), layout, dtype=E8[to])
    assert torch.equal(again.view(torch.uint8), q.view(torch.uint8)) and torch.equal(s2, s)


@pytest.mark.parametrize("rows,k,experts,align,n", [(1, 1, 1, 128, 1), (5, 8, 16, 128, 40), (40, 6, 9, 256, 129),
                                                    (70, 3, 5, 128, 1000), (4, 8, 64, 1, 2048), (33, 2, 7, 16, 300)])
@pytest.mark.parametrize("dtype,to", [("bf16", "e4m3"), ("fp32", "e5m2")])
def test_quantize_with_a_plan(rows, k, experts, align, n, dtype, to):
    plan, place, order, offsets = _made(n, rows, k, experts, align)
    x, end = _blocks_input(n, rows, n, dtype), int(offsets[-1])
    for layout in (ts.BLOCK_ROW, ts.BLOCK_COLUMN) if align % 128 == 0 else (ts.BLOCK_ROW,):
        say(f"quantize with a plan {rows} x {k} of {experts}, align {align}, n {n}, layout {layout}")
        P = order.size
        shape, sshape = ((P, -(-n // 16) * 16), (P, -(-n // 128))) if layout == 0 else \
            ((n, -(-P // 16) * 16), (n, -(-P // 128)))
        q, s = ts.ds_block_quantize(_wide(x, 3, 1), layout, dtype=E8[to], plan=plan,
                                    out=torch.full(shape, 2.0, device="cuda").to(E8[to]),
                                    out_scales=torch.full(sshape, KEPT, device="cuda"))
        want, want_s = _quantized(x, layout, to, plan, place, order, offsets)
        got, got_s = _np(q.float()), _np(s)
        if layout == ts.BLOCK_COLUMN:
            got, got_s, want, want_s = got.T, got_s.T, want.T, want_s.T
            assert np.array_equal(got[:end], want) and (got[end:P] == 2).all()
            assert np.array_equal(got_s[:end // 128], want_s) and (got_s[end // 128:] == KEPT).all()
        else:
            assert np.array_equal(got[:end, :n], want) and (got[:end, n:] == 0).all() and (got[end:] == 2).all()
            assert np.array_equal(got_s[:end], want_s) and (got_s[end:] == KEPT).all()


@pytest.mark.parametrize("to", ["e4m3", "e5m2"])
@pytest.mark.parametrize("layout", [0, 1, 2])
def test_quantize_extremes(to, layout):
    say(f"quantize extremes {to}, layout {layout}")
    big = 3.4028234663852886e38
    x = torch.zeros(128 * 12, 128)
    g = _gen(9)
    fill = [torch.zeros(128, 128), torch.full((128, 128), big), big * (2 * torch.rand(128, 128, generator=g) - 1),
            1e-45 * torch.randint(0, 9, (128, 128), generator=g), 2.0 ** -101 * torch.randn(128, 128, generator=g),
            2.0 ** -118 * torch.randn(128, 128, generator=g), 2.0 ** -90 * torch.randn(128, 128, generator=g),
            2.0 ** -61 * torch.randn(128, 128, generator=g), torch.randn(128, 128, generator=g),
            torch.randn(128, 128, generator=g), torch.randn(128, 128, generator=g), torch.randn(128, 128, generator=g)]
    # blocks at whose scale of 1 (the largest magnitude is the type's) every tie occurs
    every = torch.arange(256, dtype=torch.uint8).view(E8[to]).float()
    every = every[every.isfinite()].sort()[0]
    mid = ((every[1:].double() + every[:-1].double()) / 2).float()
    ties = torch.cat([every, mid]).repeat(64)[:128 * 128].view(128, 128)
    fill[8] = torch.where(torch.arange(128)[:, None] == torch.arange(128)[None], orc.LARGEST[to], ties)
    fill[9][3, 5] = float("inf")
    fill[10][127, 0] = float("nan")
    fill[11][0, 127] = float("-inf")
    for i, b in enumerate(fill):
        x[128 * i:128 * (i + 1)] = b
    if layout == 1:
        x = x.t().contiguous()
    q, s = ts.ds_block_quantize(x.cuda(), layout, dtype=E8[to])
    want, want_s = _quantized(x, layout, to)
    assert np.array_equal(_np(s), want_s, equal_nan=True)
    assert np.array_equal(_np(q.float()), want)


@pytest.mark.parametrize("to", ["e4m3", "e5m2"])
@pytest.mark.parametrize("layout", [0, 1, 2])
@pytest.mark.parametrize("exponent", [0, -70, -110])
def test_quantize_next_to_ties(to, layout, exponent):
    """Quotients within a few 2^-24 of every tie of 8-bit floats, on either side: fp32 makes many of them the tie."""
    say(f"quantize next to ties {to}, layout {layout}, 2^{exponent}")
    every = torch.arange(256, dtype=torch.uint8).view(E8[to]).float()
    every = every[every.isfinite()].sort()[0].double()
    mid = (every[1:] + every[:-1]) / 2
    x = torch.randn(128, 4 * 128, generator=_gen(exponent + 500)).double() * 2.0 ** exponent
    for r in range(128 if layout == 0 else 1):
        for b in range(4):
            at = (slice(r, r + 1), slice(128 * b, 128 * b + 128)) if layout == 0 else (slice(None), slice(128 * b, 128 * b + 128))
            for part in ([x[at]] if layout != 1 else [x[at][:, c:c + 1] for c in range(128)]):
                most = part.abs().max().float()
                scale = (most.clamp(min=2.0 ** -100) / orc.LARGEST[to]).double()
                flat = part.reshape(-1)
                n = flat.numel() - 1
                t = mid[torch.randint(0, mid.numel(), (n,), generator=_gen(r * 4 + b))]
                near = (t * scale).float()
                near = near * (1 + 2.0 ** -23 * torch.randint(-1, 2, (n,), generator=_gen(r + b)))
                new = torch.cat([most.double()[None], near.double()]).view(part.shape)
                part.copy_(new)
    x = x.float()
    q, s = ts.ds_block_quantize(x.cuda(), layout, dtype=E8[to])
    want, want_s = _quantized(x, layout, to)
    assert np.array_equal(_np(s), want_s)
    assert np.array_equal(_np(q.float()), want)


def test_quantize_a_stack_of_weights():
    say("quantize a stack")
    for rows in (128, 100):
        x = _blocks_input(rows, 3 * rows, 200, "bf16")
        q, s = ts.ds_block_quantize(x.cuda().view(3, rows, 200), ts.BLOCK_TILE)
        for g in range(3):
            want, want_s = _quantized(x[g * rows:(g + 1) * rows], ts.BLOCK_TILE, "e4m3")
            assert np.array_equal(_np(q[g].float())[:, :200], want) and np.array_equal(_np(s[g]), want_s)


# ---------------------------------------------------------------------------------------- product
def _operand(seed, rows, k, to, of=1):
    """Random 8-bit values of all exponents and scales of many sizes; and the numbers they stand for."""
    g = _gen(seed)
    v = torch.randn(rows, k, generator=g) * torch.exp2(torch.randint(-6, 3, (rows, k), generator=g).float())
    q = v.to(E8[to])
    s = torch.exp(torch.randn(-(-rows // of), -(-k // 128), generator=g))
    return q, s, orc.values(_np(q.float()), s.numpy(), of)


def _strided8(q, pad):
    """The same on the device with rows `pad` bytes longer, NaN in between."""
    rows, k = q.shape
    base = torch.full((rows, k + pad), 0x7F, dtype=torch.uint8, device="cuda")
    base[:, :k] = q.view(torch.uint8).cuda()
    return base.view(q.dtype)[:, :k]


def _product_tol(k, size, want, out):
    eight = 2.0 ** -10 if out in ("bf16", torch.bfloat16) else 0
    return (eight + (273 + -(-k // 128)) * U) * size + U * np.abs(want) + _half(out, want)


@pytest.mark.parametrize("m,n,k", [(1, 1, 16), (1, 128, 128), (3, 100, 144), (16, 64, 256), (17, 65, 1040), (64, 257, 512),
                                   (100, 333, 208), (128, 128, 2048), (200, 512, 384), (257, 1000, 1296), (511, 300, 640),
                                   (1024, 1024, 272)])
@pytest.mark.parametrize("a,of_b,out", [("e4m3", 128, "bf16"), ("e4m3", 1, "fp32"), ("e5m2", 128, "fp32"),
                                        ("e5m2", 1, "bf16")])
def test_product(m, n, k, a, of_b, out):
    say(f"product {m} x {n} x {k}, {a}, {of_b}, {out}")
    qa, sa, va = _operand(m, m, k, a)
    qb, sb, vb = _operand(n + 1, n, k, "e4m3", of_b)
    want, size = orc.product(va, vb)
    got = ts.ds_block_product(_strided8(qa, 32), sa.cuda(), _strided8(qb, 16), sb.cuda(),
                              out=_wide(torch.zeros(m, n, dtype=DT[out]), 3, 1))
    _close(got, want, _product_tol(k, size, want, out), "product")
    assert torch.equal(got, ts.ds_block_product(qa.cuda(), sa.cuda(), qb.cuda(), sb.cuda(), out_dtype=DT[out]))


def _exact_on_device(va, vb):
    """The definition in 64 bits for larger sizes: elementary products on the device."""
    a, b = torch.from_numpy(va).cuda(), torch.from_numpy(vb).cuda()
    return (a @ b.t()).cpu().numpy(), (a.abs() @ b.abs().t()).cpu().numpy()


# Sizes at which every kernel is chosen (the tile is noted), with fewer blocks of the inner axis than are under
# way at a time, as many, and more; with a rest and without; with rows and columns past the last tile.
LARGER = [(500, 2000, 16), (500, 1999, 128), (450, 2000, 640), (511, 1990, 1040), (512, 2048, 768),  # 64 x 128
          (1000, 4000, 144), (1023, 4001, 512), (1024, 4096, 1296),  # 128 x 128
          (2000, 2048, 272), (2047, 2050, 128), (1999, 2048, 400),  # exact sums: 128 x 128
          (4000, 4001, 144), (4096, 4096, 256), (4095, 4000, 416)]  # 256 x 256


@pytest.mark.parametrize("m,n,k", LARGER)
@pytest.mark.parametrize("a,of_b,out", [("e4m3", 128, "bf16"), ("e5m2", 1, "bf16"), ("e5m2", 128, "fp32"),
                                        ("e4m3", 1, "fp32")])
def test_larger_product(m, n, k, a, of_b, out):
    say(f"larger product {m} x {n} x {k}, {a}, {of_b}, {out}")
    qa, sa, va = _operand(m, m, k, a)
    qb, sb, vb = _operand(n + 1, n, k, "e4m3", of_b)
    want, size = _exact_on_device(va, vb)
    base = torch.full((m + 2, n + 8), KEPT, dtype=DT[out], device="cuda")
    got = ts.ds_block_product(_strided8(qa, 16), sa.cuda(), qb.cuda(), sb.cuda(), out=base[1:m + 1, 3:n + 3])
    _close(got, want, _product_tol(k, size, want, out), "product")
    got.fill_(KEPT)
    assert (base == KEPT).all()  # nothing was written around it


@pytest.mark.parametrize("m,n,k", [(500, 2000, 300), (1024, 4096, 300), (4096, 4096, 300)])
@pytest.mark.parametrize("out", ["bf16", "fp32"])
def test_larger_product_keeps_nan_in_its_rows(m, n, k, out):
    say(f"larger product nan {m} x {n}, {out}")
    k -= k % 16
    qa, sa, _ = _operand(1, m, k, "e5m2")
    qb, sb, _ = _operand(2, n, k, "e4m3", 128)
    clean = ts.ds_block_product(qa.cuda(), sa.cuda(), qb.cuda(), sb.cuda(), out_dtype=DT[out])
    assert clean.isfinite().all()
    sa[5, 1] = float("nan")
    qa.view(torch.uint8)[m - 1, k - 1] = 0x7C  # an infinity
    qb.view(torch.uint8)[n - 3, 7] = 0x7F  # a NaN
    got = ts.ds_block_product(qa.cuda(), sa.cuda(), qb.cuda(), sb.cuda(), out_dtype=DT[out])
    assert got[5].isnan().all() and got[:, n - 3].isnan().all() and not got[m - 1].isfinite().any()
    rest = torch.ones(m, n, dtype=torch.bool)
    rest[5], rest[m - 1], rest[:, n - 3] = False, False, False
    assert torch.equal(got.cpu()[rest], clean.cpu()[rest])


@pytest.mark.parametrize("loads", [[700, 0, 130, 64, 1, 400], [300] * 20, [1] * 1000 + [0] * 24, [2000, 3, 0, 900],
                                   [100, 3, 128, 0, 77] * 13, [40, 33] * 4],
                         ids=["few", "even", "many", "uneven", "short", "eight"])
@pytest.mark.parametrize("out", ["bf16", "fp32"])
def test_larger_product_of_segments(loads, out):
    n, k = (500, 272) if len(loads) > 100 else (2000, 400)
    say(f"larger product of segments, {len(loads)}, {out}")
    offsets = np.concatenate([[0], np.cumsum(loads)]).astype(np.int32)
    m, G = int(offsets[-1]) + 3, len(loads)
    qa, sa, va = _operand(m, m, k, "e4m3")
    qb, sb, vb = _operand(7, G * n, k, "e4m3")
    got = ts.ds_block_product(qa.cuda(), sa.cuda(), qb.cuda().view(G, n, k), sb.cuda().view(G, n, -1),
                              offsets=torch.from_numpy(offsets).cuda(),
                              out=torch.full((m, n), KEPT, dtype=DT[out], device="cuda"))
    assert (got[m - 3:] == KEPT).all()
    a, b = torch.from_numpy(va).cuda(), torch.from_numpy(vb).cuda().view(G, n, k)
    for g in range(G):
        lo, hi = int(offsets[g]), int(offsets[g + 1])
        if hi > lo:
            want, size = (a[lo:hi] @ b[g].t()).cpu().numpy(), (a[lo:hi].abs() @ b[g].abs().t()).cpu().numpy()
            _close(got[lo:hi], want, _product_tol(k, size, want, out), f"segment {g}")


@pytest.mark.parametrize("m,n", [(600, 1000), (2048, 1000)])
@pytest.mark.parametrize("out", ["bf16", "fp32"])
def test_larger_product_along_segments(m, n, out):
    say(f"larger product along segments {m} x {n}, {out}")
    ends, k = [0, 128, 128, 1024, 1152, 2560, 2704], 2704
    qa, sa, va = _operand(m, m, k, "e5m2")
    qb, sb, vb = _operand(n + 1, n, k, "e4m3")
    got = ts.ds_block_product(qa.cuda(), sa.cuda(), qb.cuda(), sb.cuda(), inner=True, out_dtype=DT[out],
                              offsets=torch.tensor(ends, dtype=torch.int32).cuda())
    for g in range(len(ends) - 1):
        lo, hi = ends[g], ends[g + 1]
        want, size = _exact_on_device(np.ascontiguousarray(va[:, lo:hi]), np.ascontiguousarray(vb[:, lo:hi]))
        _close(got[g], want, _product_tol(k, size, want, out), f"segment {g}")


LOADS = [[5], [0, 3, 0], [16, 16, 16, 16], [1] * 40, [130, 0, 7, 64, 1], [0] * 70 + [9] + [0] * 70 + [33], [300, 520, 2],
         [70, 60, 50, 90], [1000, 40]]


@pytest.mark.parametrize("loads", LOADS, ids=lambda v: str(len(v)) + "_" + str(sum(v)))
@pytest.mark.parametrize("n,k,a,of_b,out", [(100, 144, "e4m3", 128, "bf16"), (300, 1040, "e5m2", 1, "fp32"),
                                            (256, 512, "e4m3", 128, "fp32")])
def test_product_of_segments(loads, n, k, a, of_b, out):
    say(f"product of segments {loads[:8]}, {n} x {k}")
    G, before, behind = len(loads), 3, 5
    offsets = np.concatenate([[before], before + np.cumsum(loads)]).astype(np.int32)
    m = int(offsets[-1]) + behind
    qa, sa, va = _operand(m, m, k, a)
    parts = [_operand(50 + g, n, k, "e4m3", of_b) for g in range(G)]
    qb, sb = torch.stack([p[0].view(torch.uint8) for p in parts]).view(torch.float8_e4m3fn), torch.stack([p[1] for p in parts])
    out_t = _wide(torch.full((m, n), KEPT, dtype=DT[out]), 5, 1)
    got = ts.ds_block_product(qa.cuda(), sa.cuda(), qb.cuda(), sb.cuda(), offsets=torch.from_numpy(offsets).cuda(), out=out_t)
    assert (got[:before] == KEPT).all() and (got[m - behind:] == KEPT).all()
    for g in range(G):
        lo, hi = offsets[g], offsets[g + 1]
        if hi > lo:
            want, size = orc.product(va[lo:hi], parts[g][2])
            _close(got[lo:hi], want, _product_tol(k, size, want, out), f"segment {g}")


@pytest.mark.parametrize("ends,k", [([0, 128], 128), ([0, 0, 256, 256, 400], 400), ([128, 384, 512], 640),
                                    ([0, 1280, 1408, 2048], 2048), ([0, 16], 16), ([5, 200, 300], 512)])
@pytest.mark.parametrize("m,n", [(1, 1), (70, 100), (300, 257), (128, 512)])
@pytest.mark.parametrize("a,out", [("e4m3", "fp32"), ("e5m2", "bf16")])
def test_product_along_segments(ends, k, m, n, a, out):
    say(f"product along segments {ends} of {k}, {m} x {n}")
    qa, sa, va = _operand(m, m, k, a)
    qb, sb, vb = _operand(n + 1, n, k, "e4m3")
    got = ts.ds_block_product(qa.cuda(), sa.cuda(), qb.cuda(), sb.cuda(), inner=True, out_dtype=DT[out],
                              offsets=torch.tensor(ends, dtype=torch.int32).cuda())
    assert got.shape == (len(ends) - 1, m, n)
    up = [min(k, -(-e // 128) * 128) for e in ends]  # others count as the next multiple
    for g in range(len(ends) - 1):
        want, size = orc.product(va[:, up[g]:up[g + 1]], vb[:, up[g]:up[g + 1]])
        _close(got[g], want, _product_tol(k, size, want, out), f"segment {g}")


def test_product_without_an_inner_axis():
    say("product k 0")
    none = torch.empty(5, 0, device="cuda").to(torch.float8_e4m3fn)
    s, w = torch.empty(5, 0, device="cuda"), torch.empty(3, 0, device="cuda")
    b = torch.empty(3, 0, device="cuda").to(torch.float8_e4m3fn)
    assert (ts.ds_block_product(none, s, b, w) == 0).all()
    got = ts.ds_block_product(none, s, b, w, inner=True, offsets=torch.zeros(3, dtype=torch.int32, device="cuda"))
    assert got.shape == (2, 5, 3) and (got == 0).all()


def test_product_keeps_nan_and_infinity_in_their_rows():
    say("product nan")
    m, n, k = 150, 140, 300
    qa, sa, va = _operand(1, m, k - k % 16, "e5m2")
    qb, sb, vb = _operand(2, n, k - k % 16, "e4m3", 128)
    clean = ts.ds_block_product(qa.cuda(), sa.cuda(), qb.cuda(), sb.cuda(), out_dtype=torch.float32)
    sa[5, 1] = float("nan")
    bits = qa.view(torch.uint8)
    bits[77, 130] = 0x7C  # an infinity
    qb.view(torch.uint8)[33, 7] = 0x7F  # a NaN
    got = ts.ds_block_product(qa.cuda(), sa.cuda(), qb.cuda(), sb.cuda(), out_dtype=torch.float32)
    assert got[5].isnan().all() and got[:, 33].isnan().all() and not got[77].isfinite().any()
    rest = torch.ones(m, n, dtype=torch.bool)
    rest[5], rest[77], rest[:, 33] = False, False, False
    assert torch.equal(got.cpu()[rest], clean.cpu()[rest])


@pytest.mark.parametrize("a,b_of", [("e4m3", 128), ("e5m2", 1)])
def test_product_gradients(a, b_of):
    """a's and b's gradients by the same entry, against the formula on the operands' numbers and against
    differences of the definition (linear in each operand, so differences are exact up to 64 bits)."""
    say("product gradients")
    m, n, k = 96, 256, 384
    _, _, va = _operand(1, m, k, a)
    qb, sb, vb = _operand(2, n, k, "e4m3", b_of)
    g = torch.randn(m, n, generator=_gen(3))
    qg, sg = ts.ds_block_quantize(g.cuda(), dtype=E8[a])
    vg = orc.values(_np(qg.float()), _np(sg), 1)
    x = torch.from_numpy(va).float()
    if b_of == 128:
        bt, st = qb.view(torch.uint8).t().contiguous().view(torch.float8_e4m3fn), sb.t().contiguous()
        da = ts.ds_block_product(qg, sg, bt.cuda(), st.cuda(), out_dtype=torch.float32)
        want, size = orc.product(vg, vb.T)
        _close(da, want, _product_tol(n, size, want, "fp32"), "a's gradient")
        for i in ((0, 0), (50, 383), (95, 7)):
            up, down = va.copy(), va.copy()
            up[i] += 1
            down[i] -= 1
            slope = ((orc.product(up, vb)[0] - orc.product(down, vb)[0]) * vg).sum() / 2
            assert abs(_np(da)[i] - slope) <= _product_tol(n, size, want, "fp32")[i] + 2.0 ** -30 * size[i] * m
    gt, sgt = ts.ds_block_quantize(g.cuda(), ts.BLOCK_COLUMN, dtype=E8[a])
    xt, sxt = ts.ds_block_quantize(x.cuda(), ts.BLOCK_COLUMN)
    db = ts.ds_block_product(gt, sgt, xt, sxt, out_dtype=torch.float32)
    vgt, vxt = orc.values(_np(gt.float()), _np(sgt), 1), orc.values(_np(xt.float()), _np(sxt), 1)
    want, size = orc.product(vgt, vxt)
    _close(db, want, _product_tol(m, size, want, "fp32"), "b's gradient")
    for i in ((0, 0), (255, 100)):
        up = np.zeros((n, k))
        up[i] = 1
        slope = (orc.product(vxt.T, up)[0] * vgt.T).sum()
        assert abs(_np(db)[i] - slope) <= _product_tol(m, size, want, "fp32")[i] + 2.0 ** -30 * size[i]


def test_product_into_rows_apart():
    say("product into rows apart")
    m, n, k, ends = 70, 90, 384, [0, 128, 384]
    qa, sa, _ = _operand(1, m, k, "e4m3")
    qb, sb, _ = _operand(2, n, k, "e4m3")
    args = (qa.cuda(), sa.cuda(), qb.cuda(), sb.cuda(), torch.tensor(ends, dtype=torch.int32).cuda(), True)
    base = torch.full((2, m, n + 6), KEPT, device="cuda")
    got = ts.ds_block_product(*args, out=base[:, :, 3:n + 3])
    assert torch.equal(got, ts.ds_block_product(*args, out_dtype=torch.float32))
    got.fill_(KEPT)
    assert (base == KEPT).all()


# --------------------------------------------------------------------------------------- together
def test_every_call_on_a_given_stream():
    """Work that a stream still has to do before the calls on it: they see its result, not what was there before."""
    say("given stream")
    stream = torch.cuda.Stream()
    E, rows, n = 8, 500, 512
    idx = _choices(1, rows, 2, E, 0).cuda()
    x, w = torch.randn(rows, n, generator=_gen(1)).cuda(), torch.rand(rows, 2, generator=_gen(2)).cuda()
    wt = torch.randn(E, n, n, generator=_gen(3)).cuda() * n ** -0.5

    def all_of(x, **kw):
        plan = ts.ds_expert_sort(idx, E, 128, **kw)
        cap = plan.order.numel()
        rows_of = ts.ds_expert_gather(x, plan, out=torch.zeros(cap, n, device="cuda"), **kw)
        q, s = ts.ds_block_quantize(x, plan=plan, out=torch.zeros(cap, n, device="cuda").to(torch.float8_e4m3fn),
                                    out_scales=torch.zeros(cap, n // 128, device="cuda"), **kw)
        b, t = ts.ds_block_quantize(wt, ts.BLOCK_TILE, **kw)
        y = ts.ds_block_product(q, s, b, t, offsets=plan.offsets, out=torch.zeros(cap, n, device="cuda"), **kw)
        out = ts.ds_expert_combine(y, plan, w, **kw)
        gy, gw = ts.ds_expert_combine_grad(out, y, plan, w, out_y=torch.zeros(cap, n, device="cuda"), **kw)
        return rows_of, q.view(torch.uint8), s, y, out, gy, gw

    want = all_of(x)
    torch.cuda.synchronize()
    late = torch.zeros_like(x)
    with torch.cuda.stream(stream):
        torch.cuda._sleep(20_000_000)
        late.copy_(x)
        got = all_of(late)
    with torch.cuda.stream(stream):
        late.zero_()
        torch.cuda._sleep(20_000_000)
        late.copy_(x)
    stream.wait_stream(torch.cuda.current_stream())
    q2, s2 = ts.ds_block_quantize(late, stream=stream)
    out2 = ts.ds_expert_combine(ts.ds_expert_gather(late, ts.ds_expert_sort(idx, E, 128, stream=stream), stream=stream),
                                ts.ds_expert_sort(idx, E, 128, stream=stream), w, stream=stream)
    stream.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    q, s = ts.ds_block_quantize(x)
    assert torch.equal(q2.view(torch.uint8), q.view(torch.uint8)) and torch.equal(s2, s)
    plan = ts.ds_expert_sort(idx, E, 128)
    assert torch.equal(out2, ts.ds_expert_combine(ts.ds_expert_gather(x, plan), plan, w))


def _layer(x, logits, w1, w2, k, align, g=None):
    """A layer of experts as a program runs it: route, sort, quantise to the experts, two products with a
    rectifier between, combine; with g also every gradient."""
    E = logits.shape[1]
    weights, idx = ts.ds_route(logits, k, renormalize=True)
    plan = ts.ds_expert_sort(idx, E, align)
    a1, s1 = ts.ds_block_quantize(x, plan=plan)
    q1, t1 = ts.ds_block_quantize(w1, ts.BLOCK_TILE)
    q2, t2 = ts.ds_block_quantize(w2, ts.BLOCK_TILE)
    h = ts.ds_block_product(a1, s1, q1, t1, offsets=plan.offsets, out=x.new_zeros(plan.order.numel(), w1.shape[1]))
    act = torch.relu(h)
    a2, s2 = ts.ds_block_quantize(act)
    y = ts.ds_block_product(a2, s2, q2, t2, offsets=plan.offsets, out=x.new_zeros(plan.order.numel(), w2.shape[1]))
    out = ts.ds_expert_combine(y, plan, weights)
    if g is None:
        return out
    gy, gw = ts.ds_expert_combine_grad(g, y, plan, weights, out_y=torch.zeros_like(y))
    grad_logits = ts.ds_route_grad(logits, idx, gw, renormalize=True)
    turned = lambda q, s: (q.view(torch.uint8).transpose(1, 2).contiguous().view(q.dtype),  # noqa: E731
                           s.transpose(1, 2).contiguous())
    qg, sg = ts.ds_block_quantize(gy, dtype=torch.float8_e5m2)
    b2, u2 = turned(q2, t2)
    gh = ts.ds_block_product(qg, sg, b2, u2, offsets=plan.offsets, out=torch.zeros_like(h)) * (h > 0)
    c = ts.BLOCK_COLUMN
    gw2 = ts.ds_block_product(*ts.ds_block_quantize(gy, c, dtype=torch.float8_e5m2), *ts.ds_block_quantize(act, c),
                              offsets=plan.offsets, inner=True, out_dtype=torch.float32)
    qh, sh = ts.ds_block_quantize(gh, dtype=torch.float8_e5m2)
    b1, u1 = turned(q1, t1)
    gx = ts.ds_expert_combine(ts.ds_block_product(qh, sh, b1, u1, offsets=plan.offsets,
                                                  out=x.new_zeros(plan.order.numel(), x.shape[1])), plan)
    gw1 = ts.ds_block_product(*ts.ds_block_quantize(gh, c, dtype=torch.float8_e5m2),
                              *ts.ds_block_quantize(x, c, plan=plan, out=torch.zeros(x.shape[1], -(-plan.order.numel() // 16) * 16, device="cuda").to(torch.float8_e4m3fn),
                                                    out_scales=torch.zeros(x.shape[1], -(-plan.order.numel() // 128), device="cuda")),
                              offsets=plan.offsets, inner=True, out_dtype=torch.float32)
    return out, grad_logits, gx, gw1, gw2


def _layer_input(seed, rows, E, d, f):
    g = _gen(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return (r(rows, d).bfloat16().cuda(), r(rows, E).cuda(), (r(E, f, d) * d ** -0.5).bfloat16().cuda(),
            (r(E, d, f) * f ** -0.5).bfloat16().cuda(), r(rows, d).bfloat16().cuda())


def test_a_layer_of_experts_forward_and_backward():
    """Against the same layer in fp32 without quantisation. Every 8-bit rounding is at most 2^-4 (e4m3) or
    2^-3 (e5m2) of its value and rounds to either side; a result that m such roundings reach is off by at
    most the sum of their bounds relative to the 2-norm: forward four e4m3 roundings (4 * 2^-4), gradients
    those of their factors besides (two more e5m2: 2^-2). Norms, so half of the bound is ample."""
    say("layer")
    rows, E, d, f, k = 200, 6, 256, 384, 2
    x, logits, w1, w2, g = _layer_input(1, rows, E, d, f)
    got = _layer(x, logits, w1, w2, k, 128, g)
    leaves = [t.float().cpu().requires_grad_() for t in (logits, x, w1, w2)]
    p = torch.softmax(leaves[0], dim=1)
    top = p.topk(k, dim=1)
    w = top[0] / top[0].sum(dim=1, keepdim=True)
    want = 0
    for j in range(k):
        e = top[1][:, j]
        h = torch.relu((leaves[2][e] @ leaves[1][:, :, None])[:, :, 0])
        want = want + w[:, j:j + 1] * (leaves[3][e] @ h[:, :, None])[:, :, 0]
    want.backward(g.float().cpu())
    for name, a, b, bound in (("out", got[0], want, 0.125), ("logits", got[1], leaves[0].grad, 0.25),
                              ("x", got[2], leaves[1].grad, 0.25), ("w1", got[3], leaves[2].grad, 0.25),
                              ("w2", got[4], leaves[3].grad, 0.25)):
        a, b = _np(a), _np(b)
        assert np.linalg.norm(a - b) <= bound * np.linalg.norm(b), name


def test_a_layer_replayed_from_graphs_and_on_other_streams():
    """Two captured decode steps, replayed in turn with eager work between; a given stream."""
    say("graphs")
    eager, graphs = [], []
    for seed, rows in ((1, 4), (2, 1)):
        x, logits, w1, w2, _ = _layer_input(seed, rows, 16, 256, 128)
        want = _layer(x, logits, w1, w2, 4, 1).clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            _layer(x, logits, w1, w2, 4, 1)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = _layer(x, logits, w1, w2, 4, 1)
        graphs.append((graph, out))
        eager.append((want, x, logits, w1, w2))
    for turn in range(4):
        for (graph, out), (want, *args) in zip(graphs, eager):
            out.zero_()
            graph.replay()
            again = _layer(*args, 4, 1)
            torch.cuda.synchronize()
            assert torch.equal(out, want) and torch.equal(again, want), turn
    big = _choices(5, 30000, 4, 64).cuda()
    want = ts.ds_expert_sort(big, 64, 16)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    got = ts.ds_expert_sort(big, 64, 16, stream=stream)
    stream.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got[:3], want[:3]))
