"""The operators behind a router on the GPU at the ends of their ranges: broken plans, guard rows around outputs,
the choice of sums, and sizes at which each tile of ds_block_product is chosen. Tolerances as in
test_gpu_experts.py, where the definitions' helpers are from."""
import ctypes
import threading

import numpy as np
import pytest
import torch

import top_selection_amd as ts
from gpu_util import say
from oracle import experts as orc
from test_gpu_experts import E8, KEPT, U, _layer, _layer_input, _made, _np, _operand

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


# ------------------------------------------------------------------------------------ exact sums
def _small_beside_large(seed, rows, k, sign):
    """Runs of eight along k: two of 256 (the second with `sign`) and six small whole numbers."""
    v = torch.randint(-3, 4, (rows, k), generator=torch.Generator().manual_seed(seed)).float()
    v[:, 0::8], v[:, 1::8] = 256, 256 * sign
    return v


def _ones(q):
    return torch.ones(q.shape[0], -(-q.shape[1] // 128))


# one size for each kernel that exact sums choose: 16 x 16, 16 x 32, 32 x 32, 64 x 128, 128 x 128
EXACT = [(4, 300, 1296), (16, 16400, 272), (100, 333, 528), (500, 2000, 640), (511, 1990, 1040), (2000, 2048, 272),
         (4095, 4000, 144)]


@pytest.mark.parametrize("m,n,k", EXACT)
@pytest.mark.parametrize("a", ["e4m3", "e5m2"])
@pytest.mark.parametrize("of_b", [1, 128])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_exact_sums_keep_what_is_small(m, n, k, a, of_b, out):
    """In every eight products two of 2^16 cancel beside small whole numbers: all partial sums are whole and below
    2^24, so fp32 sums are exact in any order, and the result is the whole number, rounded once. (A sum that cuts
    below 2^-13 of the largest product loses what is below 8.)"""
    say(f"exact sums {m} x {n} x {k}, {a}, {of_b}, {out}")
    va, vb = _small_beside_large(1, m, k, 1), _small_beside_large(2, n, k, -1)
    want = (va.cuda() @ vb.cuda().t()).double()  # (whole numbers below 2^24: exact)
    qa, qb = va.to(E8[a]).cuda(), vb.to(E8["e4m3"]).cuda()
    sb = _ones(qb)[::of_b].contiguous().cuda()
    got = ts.ds_block_product(qa, _ones(qa).cuda(), qb, sb, out_dtype=out, exact=True)
    assert got.dtype == out and torch.equal(got, want.to(out))


@pytest.mark.parametrize("loads", [[4] * 6, [700, 0, 130, 64, 1, 400], [300] * 20, [2000, 3, 0, 900]],
                         ids=["few", "uneven", "even", "large"])
@pytest.mark.parametrize("of_b", [1, 128])
def test_exact_sums_of_segments(loads, of_b):
    n, k, G = 1000, 400, len(loads)
    say(f"exact sums of segments {loads[:4]}, {of_b}")
    offsets = np.concatenate([[0], np.cumsum(loads)]).astype(np.int32)
    va = _small_beside_large(3, int(offsets[-1]), k, 1)
    vb = _small_beside_large(4, G * n, k, -1).view(G, n, k)
    qa, qb = va.to(E8["e4m3"]).cuda(), vb.to(E8["e4m3"]).cuda()
    sb = torch.ones(G, -(-n // of_b), -(-k // 128), device="cuda")
    got = ts.ds_block_product(qa, _ones(qa).cuda(), qb, sb, offsets=torch.from_numpy(offsets).cuda(), exact=True)
    for g in range(G):
        lo, hi = int(offsets[g]), int(offsets[g + 1])
        assert torch.equal(got[lo:hi], (va[lo:hi].cuda() @ vb[g].cuda().t()).bfloat16()), g


def test_exact_sums_along_segments():
    say("exact sums along segments")
    m, n, k, ends = 700, 900, 1040, [0, 256, 256, 1040]
    va, vb = _small_beside_large(5, m, k, 1), _small_beside_large(6, n, k, -1)
    qa, qb = va.to(E8["e5m2"]).cuda(), vb.to(E8["e4m3"]).cuda()
    got = ts.ds_block_product(qa, _ones(qa).cuda(), qb, _ones(qb).cuda(), inner=True, exact=True,
                              offsets=torch.tensor(ends, dtype=torch.int32, device="cuda"))
    for g in range(3):
        want = va[:, ends[g]:ends[g + 1]].cuda() @ vb[:, ends[g]:ends[g + 1]].cuda().t()
        assert torch.equal(got[g], want.bfloat16()), g


def test_exact_sums_of_a_row_do_not_depend_on_its_batch():
    """The first rows alone and among many: with exact sums (of whole numbers) the same bits."""
    say("exact sums and batches")
    n, k = 2048, 1024
    va, vb = _small_beside_large(7, 2048, k, 1), _small_beside_large(8, n, k, -1)
    qa, qb = va.to(E8["e4m3"]).cuda(), vb.to(E8["e4m3"]).cuda()
    sa, sb = _ones(qa).cuda(), _ones(qb).cuda()
    all_of = ts.ds_block_product(qa, sa, qb, sb, exact=True)
    for m in (1, 16, 40, 256, 1000):
        assert torch.equal(ts.ds_block_product(qa[:m], sa[:m], qb, sb, exact=True), all_of[:m]), m


# ------------------------------------------------------------------- every tile, with tiles of scales
def _values(q, s, of):
    """What 8-bit values and scales for each `of` x 128 of them stand for, in 64 bits on the device."""
    full = s.double().repeat_interleave(of, dim=-2)[..., :q.shape[-2], :].repeat_interleave(128, dim=-1)
    return q.double() * full[..., :q.shape[-1]]


def _within(got, a, b, k, out, label, exact=False):
    want, size = a @ b.t(), a.abs() @ b.abs().t()
    eight = 0 if exact or out == torch.float32 else 2.0 ** -10
    tol = (eight + (273 + -(-k // 128)) * U) * size + U * want.abs()
    if out == torch.bfloat16:
        tol += 2.0 ** -8 * want.abs() + 2.0 ** -133
    off = ~((got.double() - want).abs() <= tol)
    assert not off.any(), f"{label}: {int(off.sum())} of {off.numel()} off, first at {off.nonzero()[0].tolist()}"


SEGMENTS = {"uneven": [700, 0, 130, 64, 1, 400], "even": [300] * 20, "large": [2000, 3, 0, 900],
            "short": [100, 3, 128, 0, 77] * 13, "eight": [40, 33] * 4}


@pytest.mark.parametrize("loads", SEGMENTS)
@pytest.mark.parametrize("a", ["e4m3", "e5m2"])
@pytest.mark.parametrize("out,exact", [(torch.bfloat16, False), (torch.bfloat16, True), (torch.float32, False)])
def test_segments_with_tiles_of_scales(loads, a, out, exact):
    """What a training step runs: every group has scales of its own for 128 x 128, of which the last cover fewer
    columns (2000 = 15 * 128 + 80). By size these take tiles of 64 x 128, 128 x 128 and 256 x 256."""
    say(f"segments with tiles of scales, {loads}, {a}, {out}, {exact}")
    n, k = 2000, 400
    loads = SEGMENTS[loads]
    offsets, G = np.concatenate([[0], np.cumsum(loads)]).astype(np.int32), len(loads)
    m = int(offsets[-1]) + 3
    qa, sa, _ = _operand(m, m, k, a)
    parts = [_operand(50 + g, n, k, "e4m3", 128)[:2] for g in range(G)]
    qa, sa = qa.cuda(), sa.cuda()
    qb = torch.stack([p[0].view(torch.uint8) for p in parts]).cuda().view(torch.float8_e4m3fn)
    sb = torch.stack([p[1] for p in parts]).cuda()
    got = ts.ds_block_product(qa, sa, qb, sb, offsets=torch.from_numpy(offsets).cuda(), exact=exact,
                              out=torch.full((m, n), KEPT, dtype=out, device="cuda"))
    assert (got[m - 3:] == KEPT).all()
    va = _values(qa, sa, 1)
    for g in range(G):
        lo, hi = int(offsets[g]), int(offsets[g + 1])
        if hi > lo:
            _within(got[lo:hi], va[lo:hi], _values(qb[g], sb[g], 128), k, out, f"segment {g}", exact)


@pytest.mark.parametrize("m,n", [(500, 2001), (1000, 4000), (4000, 4001)])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_products_of_many_blocks(m, n, out):
    """67 blocks of the inner axis: a lane holds the tile scales of 64, which are then read anew."""
    say(f"many blocks {m} x {n}, {out}")
    k = 8192 + 272
    qa, sa, _ = _operand(m, m, k, "e4m3")
    qb, sb, _ = _operand(n + 1, n, k, "e4m3", 128)
    qa, sa, qb, sb = qa.cuda(), sa.cuda(), qb.cuda(), sb.cuda()
    _within(ts.ds_block_product(qa, sa, qb, sb, out_dtype=out), _values(qa, sa, 1), _values(qb, sb, 128), k, out, "product")


@pytest.mark.parametrize("loads", ["uneven", "eight"])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_segments_of_many_blocks(loads, out):
    say(f"segments of many blocks, {loads}, {out}")
    n, k, loads = 2001, 8192 + 272, SEGMENTS[loads]
    offsets, G = np.concatenate([[0], np.cumsum(loads)]).astype(np.int32), len(loads)
    qa, sa, _ = _operand(1, int(offsets[-1]), k, "e5m2")
    parts = [_operand(70 + g, n, k, "e4m3", 128)[:2] for g in range(G)]
    qa, sa = qa.cuda(), sa.cuda()
    qb = torch.stack([p[0].view(torch.uint8) for p in parts]).cuda().view(torch.float8_e4m3fn)
    sb = torch.stack([p[1] for p in parts]).cuda()
    got = ts.ds_block_product(qa, sa, qb, sb, offsets=torch.from_numpy(offsets).cuda(), out_dtype=out)
    va = _values(qa, sa, 1)
    for g in range(G):
        lo, hi = int(offsets[g]), int(offsets[g + 1])
        if hi > lo:
            _within(got[lo:hi], va[lo:hi], _values(qb[g], sb[g], 128), k, out, f"segment {g}")


@pytest.mark.parametrize("m,n,k", [(8, 2048, 2048), (100, 333, 2048), (512, 2048, 768), (1000, 4000, 2048),
                                   (4096, 4096, 2048), (512, 2048, 8192)])
@pytest.mark.parametrize("of_b", [1, 128])
@pytest.mark.parametrize("exact", [False, True])
def test_mean_error_of_bf16_products(m, n, k, of_b, exact):
    """The mean error of normal data, a bound about twenty times tighter than that of single elements. It is at most
      * the mean rounding to bf16: half of half a step, 2^-9 of the value;
      * the fp32 sums' (273 + blocks) u of the products' magnitudes;
      * and where the 8-bit unit adds: it cuts seven of eight products towards zero by less than 2^-13 of the largest, so by
        errors with the products' signs, which are even and independent for such data: the mean of their sum's magnitude is
        at most the root of their squares' sum, over a block 112 (2^-13 of its largest |a| times its largest |b|)^2."""
    say(f"mean error {m} x {n} x {k}, {of_b}, {exact}")
    g = torch.Generator(device="cuda").manual_seed(m + n + k)
    a, sa = ts.ds_block_quantize(torch.randn(m, k, generator=g, device="cuda"))
    b, sb = ts.ds_block_quantize(torch.randn(n, k, generator=g, device="cuda"), ts.BLOCK_TILE if of_b == 128 else ts.BLOCK_ROW)
    va, vb = _values(a, sa, 1), _values(b, sb, of_b)
    want, size = va @ vb.t(), va.abs() @ vb.abs().t()
    bound = 2.0 ** -9 * want.abs() + (273 + k // 128) * U * size
    if not exact:
        top = lambda v: v.abs().view(v.shape[0], -1, 128).amax(dim=2) ** 2  # noqa: E731
        bound += 2.0 ** -13 * (112 * (top(va) @ top(vb).t())).sqrt()
    got = ts.ds_block_product(a, sa, b, sb, exact=exact).double()
    assert (got - want).abs().mean() <= bound.mean()
    # neither above nor below: the mean of n m such errors of either sign
    assert (got - want).mean().abs() <= 8 * bound.mean() / (m * n) ** 0.5 + 2.0 ** -13 * bound.mean()


# ---------------------------------------------------------------------- broken plans, guarded outputs
class _Guarded:
    """A device matrix in the middle of a larger one, all KEPT (8-bit: 2), and a check of what lies around it."""

    def __init__(self, rows, n, dtype, groups=1):
        self.fill = KEPT if dtype.itemsize > 1 else 2.0
        self.base = torch.full((groups * rows + 64, n + 32), self.fill, device="cuda").to(dtype)
        self.rows, self.n = groups * rows, n
        self.view = self.base[32:32 + groups * rows, 16:16 + n]
        if groups > 1:
            self.view = self.base[32:32 + groups * rows].view(groups, rows, n + 32)[:, :, 16:16 + n]

    def check(self):
        around = self.base.float().clone()
        around[32:32 + self.rows, 16:16 + self.n] = self.fill
        assert (around == self.fill).all()


def _broken(rows, k, experts, align, seed=1):
    """A plan with positions, slots and offsets out of range; the positions that still hold a slot both ways, and that
    slot's row."""
    plan, place, order, _ = _made(seed, rows, k, experts, align, dropped=0)
    bad = ts.ExpertPlan(plan.place.clone(), plan.order.clone(), plan.offsets.clone(), align)
    bad.place[::2] = 2 ** 31 - 1
    bad.place[1::4] = -5
    bad.order[::3] = 2 ** 31 - 1
    bad.order[1::7] = -9
    bad.offsets[-1] = 2 ** 31 - 1
    bad.offsets[0] = -7
    flat, order = _np(bad.place).reshape(-1), _np(bad.order)
    at = [p for p in range(order.size) if 0 <= order[p] < rows * k and flat[order[p]] == p]
    assert len(at) >= 4
    return bad, np.array(at), order[at] // k


@pytest.mark.parametrize("n", [70, 257])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_of_broken_plans(n, dtype):
    say(f"rows of broken plans, n {n}, {dtype}")
    rows, k = 40, 3
    plan, at, row = _broken(rows, k, 5, 16)
    cap = plan.order.numel()
    x, y = torch.randn(rows, n, device="cuda").to(dtype), torch.randn(cap, n, device="cuda").to(dtype)
    w = torch.rand(rows, k, device="cuda")
    out = _Guarded(cap, n, dtype)
    ts.ds_expert_gather(x, plan, out=out.view)
    out.check()
    assert torch.equal(out.view[at], x[row])
    # combining skips slots out of range, and its gradient gives them 0
    place = _np(plan.place)
    has = (place >= 0) & (place < cap)
    back = _Guarded(rows, n, dtype)
    ts.ds_expert_combine(y, plan, w, out=back.view)
    back.check()
    want, size = orc.combine(_np(y), np.where(has, place, -1), _np(w))
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 0
    assert (np.abs(_np(back.view) - want) <= k * U * size + half * np.abs(want)).all()
    grad = _Guarded(cap, n, dtype)
    _, gw = ts.ds_expert_combine_grad(x, y, plan, w, out_y=grad.view)
    grad.check()
    _, want_w, size = orc.combine_grad(_np(x), _np(y), np.where(has, place, -1), _np(w), np.array([0]), np.zeros((cap, n)))
    assert (np.abs(_np(gw) - want_w) <= (n / 64 + 24) * U * size).all() and (_np(gw)[~has] == 0).all()
    slot = _np(plan.order)[at]
    want = _np(x)[row] * _np(w).reshape(-1)[slot][:, None]
    assert (np.abs(_np(grad.view)[at] - want) <= (U + half) * np.abs(want)).all()


@pytest.mark.parametrize("n", [70, 257])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_blocks_of_broken_plans(n, dtype):
    say(f"blocks of broken plans, n {n}, {dtype}")
    rows, k = 40, 3
    x = torch.randn(rows, n, device="cuda").to(dtype)
    plan, at, row = _broken(rows, k, 5, 16)
    cap, wide = plan.order.numel(), -(-n // 16) * 16
    q, s = _Guarded(cap, wide, E8["e4m3"]), torch.full((cap + 64, -(-n // 128)), KEPT, device="cuda")
    ts.ds_block_quantize(x, plan=plan, out=q.view, out_scales=s[32:32 + cap])
    q.check()
    assert (s[:32] == KEPT).all() and (s[32 + cap:] == KEPT).all()
    want, want_s = ts.ds_block_quantize(x)
    assert torch.equal(q.view[at].view(torch.uint8), want[row].view(torch.uint8)) and torch.equal(s[32:][at], want_s[row])
    # columns go by the order alone: what it has out of range is padding, up to the end, here the capacity
    plan, _, _ = _broken(rows, k, 5, 128)
    order, cap = _np(plan.order), plan.order.numel()
    q, s = _Guarded(n, cap, E8["e5m2"]), torch.full((n + 64, cap // 128), KEPT, device="cuda")
    ts.ds_block_quantize(x, ts.BLOCK_COLUMN, dtype=E8["e5m2"], plan=plan, out=q.view, out_scales=s[32:32 + n])
    q.check()
    assert (s[:32] == KEPT).all() and (s[32 + n:] == KEPT).all()
    held = (order >= 0) & (order < rows * k)
    v = np.where(held[:, None], _np(x)[np.where(held, order, 0) // k], 0).astype(np.float32)
    want, want_s = orc.quantize(np.ascontiguousarray(v.T), 1, "e5m2")
    assert np.array_equal(_np(q.view.float()), want) and np.array_equal(_np(s[32:32 + n]), want_s)


@pytest.mark.parametrize("m,n,split", [(72, 20, 20), (1000, 2000, 200)])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_products_of_broken_offsets(m, n, split, out):
    """Offsets that fall, and lie below 0 and past the end: clamped, and segments that end before they start are empty.
    By rows the first segment has the first `split` rows to itself."""
    say(f"products of broken offsets {m} x {n}, {out}")
    k = 384
    far = torch.tensor([-4, m - 10, split, 2 ** 31 - 1, 7, -3], dtype=torch.int32, device="cuda")
    qa, sa, _ = _operand(1, m, k, "e4m3")
    qb, sb, _ = _operand(2, 5 * n, k, "e4m3")
    qa, sa, qb, sb = qa.cuda(), sa.cuda(), qb.cuda(), sb.cuda()
    o = _Guarded(m, n, out)
    ts.ds_block_product(qa, sa, qb.view(5, n, k), sb.view(5, n, -1), offsets=far, out=o.view)
    o.check()
    _within(o.view[:split], _values(qa, sa, 1)[:split], _values(qb[:n], sb[:n], 1), k, out, "rows")
    far = torch.tensor([-4, 90, 20, 2 ** 31 - 1, 7], dtype=torch.int32, device="cuda")
    o = _Guarded(m, n, out, groups=4)
    qb, sb = qb[:n], sb[:n]
    ts.ds_block_product(qa, sa, qb, sb, offsets=far, inner=True, out=o.view)
    o.check()
    va, vb = _values(qa, sa, 1), _values(qb, sb, 1)
    for g, (lo, hi) in enumerate([(0, 128), (128, 128), (128, k), (k, k)]):
        _within(o.view[g], va[:, lo:hi], vb[:, lo:hi], k, out, f"segment {g}")


# ------------------------------------------------------------------------- launches, graphs, threads
def _identity(rows):
    """A plan of one expert and one slot a row: positions are rows."""
    return ts.ds_expert_sort(torch.zeros(rows, 1, dtype=torch.int32, device="cuda"), 1)


def test_rows_of_more_than_one_launch():
    """A launch is at most 2^21 workgroups, of sixteen short rows (the gradient: four)."""
    say("rows past a launch")
    n = 8
    rows = 16 * 2 ** 21 + 5
    plan = _identity(rows)
    x = torch.randint(-1000, 1000, (rows, n), dtype=torch.int16, device="cuda").bfloat16()
    out = ts.ds_expert_gather(x, plan)
    assert torch.equal(out, x)
    assert torch.equal(ts.ds_expert_combine(out, plan, torch.full((rows, 1), 0.5, device="cuda")), x * 0.5)
    rows = 4 * 2 ** 21 + 5
    plan, x = _identity(rows), x[:rows]
    w = torch.randint(1, 4, (rows, 1), device="cuda").float()
    gy, gw = ts.ds_expert_combine_grad(x, x, plan, w)
    assert torch.equal(gy, (w * x.float()).bfloat16()) and torch.equal(gw[:, 0], (x.float() ** 2).sum(dim=1))


@pytest.mark.parametrize("layout,rows,n", [(0, 32 * 2 ** 21 + 40, 3), (1, 3, 64 * 2 ** 21 + 100), (2, 128 * 2 ** 21 + 130, 3)])
def test_blocks_of_more_than_one_launch(layout, rows, n):
    """As 2^21 workgroups take 32 blocks of a row, 64 columns, or a tile each: the same as in two calls."""
    say(f"blocks past a launch, layout {layout}")
    x = torch.randn(rows, n, device="cuda", dtype=torch.bfloat16)
    q, s = ts.ds_block_quantize(x, layout)
    half = 2 ** 26  # rows of q
    for part in (slice(0, half), slice(half, None)):
        want, want_s = ts.ds_block_quantize(x[:, part].contiguous() if layout == 1 else x[part], layout)
        assert torch.equal(q[part].view(torch.uint8), want.view(torch.uint8))
        assert torch.equal(s[slice(part.start // 128, part.stop and part.stop // 128) if layout == 2 else part], want_s)


def test_a_product_of_more_than_one_launch():
    say("product past a launch")
    m, n, k = 2, 32 * 2 ** 21 + 70, 16
    qb = torch.randint(0, 0x70, (n, k), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    sb = torch.rand(n, 1, device="cuda")
    qa, sa = torch.randn(m, k, device="cuda").to(torch.float8_e4m3fn), torch.rand(m, 1, device="cuda")
    got = ts.ds_block_product(qa, sa, qb, sb)
    for part in (slice(0, 1000), slice(n - 1000, n)):
        assert torch.equal(got[:, part], ts.ds_block_product(qa, sa, qb[part], sb[part]))
    assert got.isfinite().all()


def test_training_steps_replayed_from_graphs():
    """Two captured layers of experts with all gradients, one of them with a sort in two launches, replayed in turn with
    eager work and synchronisation between: every replay gives what eager work gives."""
    say("training steps from graphs")
    steps = []
    for seed, rows, k in ((1, 150, 2), (2, 2100, 4)):
        x, logits, w1, w2, g = _layer_input(seed, rows, 6, 128, 256)
        run = lambda a=(x, logits, w1, w2, k, 128, g): _layer(*a)  # noqa: E731
        want = [t.clone() for t in run()]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            run()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = run()
        steps.append((graph, out, want, run))
    for turn in range(4):
        for graph, out, want, run in steps:
            for t in out:
                t.zero_()
            graph.replay()
            again = run()
            torch.cuda.synchronize()
            for got in (out, again):
                assert all(torch.equal(a, b) for a, b in zip(got, want)), turn


def test_calls_from_several_threads():
    """Threads with streams of their own: plans, workspaces and outputs are each call's."""
    say("threads")
    jobs = []
    for i in range(6):
        idx = torch.randint(-1, 40, (3000 + 11 * i, 4), dtype=torch.int32, device="cuda")
        x = torch.randn(idx.shape[0], 96 + i, device="cuda")
        plan = ts.ds_expert_sort(idx, 40, 16)
        end = int(plan.offsets[-1])
        jobs.append((idx, x, end, [t.clone() for t in plan[:3]], ts.ds_expert_gather(x, plan)[:end].clone(),
                     ts.ds_expert_combine(ts.ds_expert_gather(x, plan), plan).clone()))
    torch.cuda.synchronize()
    wrong = []

    def work(idx, x, end, arrays, rows, back):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(20):
                plan = ts.ds_expert_sort(idx, 40, 16)
                got = ts.ds_expert_gather(x, plan)
                out = ts.ds_expert_combine(got, plan)
                if not (all(torch.equal(a, b) for a, b in zip(plan[:3], arrays)) and torch.equal(got[:end], rows)
                        and torch.equal(out, back)):
                    wrong.append(idx.shape)

    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
