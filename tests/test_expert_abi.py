"""Host-side checks of the operators behind a router (no GPU needed): constants and structs match the
header, capacities and workspaces, and invalid calls are refused before the device is touched."""
import ctypes
import re

import numpy as np
import pytest
import torch

import top_selection_amd as ts
from oracle import experts as orc

B = ts._binding
BAD, BIG, ALIGN, WS = ts.DS_ERR_INVALID_ARG, ts.DS_ERR_UNSUPPORTED, ts.DS_ERR_ALIGNMENT, ts.DS_ERR_WORKSPACE
# addresses far apart, never dereferenced by a refused call
P, O, F, X, Y, G, W, Q, S = (i << 40 for i in range(1, 10))


def _plan(place=P, order=O, offsets=F, rows=4, capacity=32, k=8, experts=64, align=1):
    return B.ds_expert_plan(place, order, offsets, rows, capacity, k, experts, align)


def _ref(p):
    return None if p is None else ctypes.byref(p)


def _sort(idx=X, plan=_plan(), ws=None, ws_bytes=0):
    return ts.lib().ds_expert_sort(idx, _ref(plan), ws, ws_bytes, None)


def _gather(x=X, n=100, stride=None, dtype=ts.BF16, plan=_plan(), out=Y, ostride=None):
    return ts.lib().ds_expert_gather(x, n, n if stride is None else stride, dtype, _ref(plan), out,
                                     n if ostride is None else ostride, None)


def _combine(y=X, n=100, stride=None, dtype=ts.BF16, plan=_plan(), w=W, out=Y, ostride=None):
    return ts.lib().ds_expert_combine(y, n, n if stride is None else stride, dtype, _ref(plan), w, out,
                                      n if ostride is None else ostride, None)


def _grad(g=G, gstride=None, y=X, ystride=None, n=100, dtype=ts.BF16, plan=_plan(), w=W, gy=Y, gystride=None, gw=Q):
    d = lambda s: n if s is None else s  # noqa: E731
    return ts.lib().ds_expert_combine_grad(g, d(gstride), y, d(ystride), n, dtype, _ref(plan), w, gy, d(gystride), gw,
                                           None)


def _quantize(x=X, rows=4, n=100, stride=None, dtype=ts.BF16, layout=ts.BLOCK_ROW, plan=None, q=Q, qstride=112,
              qtype=ts.E4M3, s=S):
    return ts.lib().ds_block_quantize(x, rows, n, n if stride is None else stride, dtype, layout, _ref(plan), q,
                                      qstride, qtype, s, None)


def _product(a=X, sa=W, astride=128, atype=ts.E4M3, arows=1, b=Y, sb=S, bstride=128, btype=ts.E4M3, brows=128, m=4,
             n=100, k=128, group=ts.GROUP_NONE, groups=1, offsets=None, out=Q, ostride=None, otype=ts.BF16):
    oa, ob = B.ds_block_operand(a, sa, astride, atype, arows), B.ds_block_operand(b, sb, bstride, btype, brows)
    return ts.lib().ds_block_product(ctypes.byref(oa), ctypes.byref(ob), m, n, k, group, groups, offsets, out,
                                     n if ostride is None else ostride, otype, None)


def test_names_are_declared_and_bound():
    new = {"ds_expert_capacity", "ds_expert_sort", "ds_expert_sort_workspace_size", "ds_expert_gather",
           "ds_expert_combine", "ds_expert_combine_grad", "ds_block_quantize", "ds_block_product"}
    assert new <= set(ts.header_functions())
    for n in new:
        assert callable(getattr(ts, n)) and hasattr(ts.lib(), n)


def test_constants_and_structs_match_the_header():
    text = open(B.HEADER_PATH).read()
    for c in ("DS_BLOCK", "DS_MAX_EXPERT_ALIGN", "DS_E4M3", "DS_E5M2", "DS_BLOCK_ROW", "DS_BLOCK_COLUMN",
              "DS_BLOCK_TILE", "DS_GROUP_NONE", "DS_GROUP_ROWS", "DS_GROUP_INNER"):
        have = getattr(ts, c, None)
        have = getattr(ts, c[3:]) if have is None else have
        assert int(re.search(rf"#define {c} (\d+)", text).group(1)) == have
    for name, cls, size in (("ds_expert_plan", B.ds_expert_plan, 56), ("ds_block_operand", B.ds_block_operand, 32)):
        body = re.search(rf"typedef struct {name} \{{(.*?)\}}", text, re.S).group(1)
        assert re.findall(r"(\w+);", body) == [f for f, _ in cls._fields_] and ctypes.sizeof(cls) == size
    # the binding's bytes are the structures'
    p, o = _plan(), B.ds_block_operand(X, W, 128, ts.E5M2, 1)
    assert B._pack_plan(P, O, F, 4, 32, 8, 64, 1, 0) == bytes(p)
    assert B._pack_operand(X, W, 128, ts.E5M2, 1) == bytes(o)


@pytest.mark.parametrize("align", [1, 16, 128, 100, 1024])
@pytest.mark.parametrize("rows,k,experts", [(0, 8, 64), (1, 1, 1), (4, 8, 256), (1000, 6, 7), (3, 64, 1024)])
def test_capacity_holds_every_choice(rows, k, experts, align):
    cap, slots = ts.ds_expert_capacity(rows, k, experts, align), rows * k
    # the most positions: as many segments as there can be, each one slot past a multiple
    ends = min(slots, experts)
    most = 0
    for segments in range(1, ends + 1):
        counts = np.ones(segments, int)
        counts[0] += slots - segments
        most = max(most, int((-(-counts // align) * align).sum()))
    assert most <= cap <= slots + ends * (align - 1) and cap % align == 0
    idx = np.random.default_rng(1).integers(-1, experts, (rows, k)).astype(np.int32)
    assert orc.sort(idx, experts, align, cap)[2][-1] <= cap


def test_workspaces():
    assert ts.ds_expert_sort_workspace_size(4, 8, 256) == 0
    big = ts.ds_expert_sort_workspace_size(65536, 8, 256)
    assert big > 0 and big % 4 == 0
    assert ts.ds_expert_sort_workspace_size(2 ** 31 // 64 - 1, 64, 1024) <= 256 * 1024 * 4
    assert _sort(plan=_plan(rows=65536, capacity=65536 * 8)) == WS
    assert _sort(plan=_plan(rows=65536, capacity=65536 * 8), ws=S, ws_bytes=63) == WS
    assert _sort(plan=_plan(rows=65536, capacity=65536 * 8), ws=S + 4, ws_bytes=1 << 30) == ALIGN


PLANS = [(dict(rows=-1), BAD), (dict(k=0), BAD), (dict(k=65, capacity=260), BIG), (dict(experts=0), BAD),
         (dict(experts=1025), BIG), (dict(align=0), BAD), (dict(align=1025, capacity=1 << 20), BIG),
         (dict(capacity=31), BAD), (dict(align=16, capacity=511), BAD), (dict(rows=2 ** 31 // 8, capacity=2 ** 31), BAD),
         (dict(capacity=2 ** 31), BAD), (dict(place=None), BAD), (dict(order=None), BAD), (dict(offsets=None), BAD),
         (dict(place=P + 2), ALIGN), (dict(order=O + 1), ALIGN), (dict(offsets=F + 2), ALIGN)]


@pytest.mark.parametrize("kw,code", PLANS)
def test_bad_plans_are_refused_by_every_entry(kw, code):
    p = _plan(**kw)
    assert _sort(plan=p) == code and _gather(plan=p) == code and _combine(plan=p) == code and _grad(plan=p) == code
    if "rows" not in kw:
        assert _quantize(plan=p) == code


def test_null_plans_are_refused():
    assert _sort(plan=None) == _gather(plan=None) == _combine(plan=None) == _grad(plan=None) == BAD


@pytest.mark.parametrize("kw,code", [
    (dict(idx=None), BAD), (dict(idx=X + 2), ALIGN), (dict(idx=P), BAD), (dict(idx=O + 4 * 31), BAD),
    (dict(idx=F - 4 * 31), BAD), (dict(plan=_plan(order=P + 4)), BAD), (dict(plan=_plan(offsets=O + 124)), BAD)])
def test_sort_refuses(kw, code):
    assert _sort(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), BAD), (dict(n=0), BAD), (dict(n=2 ** 31), BAD), (dict(stride=99), BAD), (dict(ostride=99), BAD),
    (dict(stride=2 ** 60), BAD), (dict(ostride=2 ** 60), BAD), (dict(x=None), BAD), (dict(out=None), BAD),
    (dict(x=X + 1), ALIGN), (dict(out=Y + 2, dtype=ts.FP32), ALIGN), (dict(out=X), BAD),
    (dict(out=X - 2 * 31 * 100 - 2), BAD), (dict(out=P), BAD), (dict(out=O), BAD), (dict(out=F), BAD)])
def test_gather_refuses(kw, code):
    assert _gather(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=-1), BAD), (dict(n=0), BAD), (dict(stride=99), BAD), (dict(ostride=99), BAD), (dict(y=None), BAD),
    (dict(out=None), BAD), (dict(y=X + 1), ALIGN), (dict(out=Y + 1), ALIGN), (dict(w=W + 2), ALIGN),
    (dict(out=X + 2 * 100 * 31), BAD), (dict(out=W), BAD), (dict(out=P), BAD)])
def test_combine_refuses(kw, code):
    assert _combine(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), BAD), (dict(n=0), BAD), (dict(gstride=99), BAD), (dict(ystride=99), BAD), (dict(gystride=99), BAD),
    (dict(g=None), BAD), (dict(y=None), BAD), (dict(gy=None, gw=None), BAD), (dict(g=G + 1), ALIGN),
    (dict(y=X + 1), ALIGN), (dict(gy=Y + 1), ALIGN), (dict(w=W + 1), ALIGN), (dict(gw=Q + 2), ALIGN),
    (dict(gy=G), BAD), (dict(gy=X, ystride=100, gystride=102), BAD), (dict(gy=X + 2), BAD), (dict(gw=W), BAD),
    (dict(gw=X), BAD), (dict(gw=Y), BAD), (dict(gw=P), BAD), (dict(gy=O), BAD)])
def test_combine_grad_refuses(kw, code):
    assert _grad(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), BAD), (dict(qtype=1), BAD), (dict(layout=3), BAD), (dict(rows=-1), BAD), (dict(n=0), BAD),
    (dict(stride=99), BAD), (dict(qstride=100), BAD), (dict(qstride=96), BAD), (dict(qstride=120), ALIGN),
    (dict(q=Q + 8), ALIGN), (dict(x=X + 1), ALIGN), (dict(s=S + 2), ALIGN), (dict(x=None), BAD), (dict(q=None), BAD),
    (dict(s=None), BAD), (dict(q=X), BAD), (dict(s=X), BAD), (dict(s=Q + 112), BAD), (dict(plan=_plan(), rows=5), BAD),
    (dict(plan=_plan(), layout=ts.BLOCK_TILE), BAD), (dict(plan=_plan(), layout=ts.BLOCK_COLUMN), BAD),
    (dict(plan=_plan(align=64, capacity=4096), layout=ts.BLOCK_COLUMN, qstride=4096), BAD),
    (dict(plan=_plan(), q=O), BAD), (dict(layout=ts.BLOCK_COLUMN, qstride=0), BAD)])
def test_quantize_refuses(kw, code):
    assert _quantize(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(atype=1), BAD), (dict(btype=0), BAD), (dict(btype=ts.E5M2), BIG), (dict(otype=2), BAD), (dict(group=3), BAD),
    (dict(groups=2), BAD), (dict(offsets=F), BAD), (dict(group=1, groups=2), BAD), (dict(group=1, groups=0, offsets=F), BAD),
    (dict(group=1, groups=1025, offsets=F), BIG), (dict(group=2, groups=1, offsets=F), BAD), (dict(arows=128), BAD),
    (dict(brows=2), BAD), (dict(m=-1), BAD), (dict(n=0), BAD), (dict(k=-16), BAD), (dict(m=2 ** 31), BAD),
    (dict(k=120), ALIGN), (dict(astride=112), BAD), (dict(bstride=112), BAD), (dict(astride=136), ALIGN),
    (dict(bstride=136), ALIGN), (dict(ostride=99), BAD), (dict(a=None), BAD), (dict(b=None), BAD), (dict(sa=None), BAD),
    (dict(sb=None), BAD), (dict(out=None), BAD), (dict(a=X + 8), ALIGN), (dict(b=Y + 4), ALIGN), (dict(sa=W + 1), ALIGN),
    (dict(sb=S + 2), ALIGN), (dict(out=Q + 1), ALIGN), (dict(group=1, offsets=F + 2), ALIGN), (dict(out=X), BAD),
    (dict(out=Y + 128), BAD), (dict(out=W), BAD), (dict(out=S), BAD), (dict(group=1, offsets=F, out=F), BAD),
    (dict(bstride=2 ** 60), BAD), (dict(ostride=2 ** 60), BAD)])
def test_product_refuses(kw, code):
    assert _product(**kw) == code


def test_calls_without_work_return_at_once():
    none = _plan(rows=0, capacity=0, place=None, order=None)
    assert _gather(plan=none, x=None, out=None) == 0 and _combine(plan=none, y=None, out=None) == 0
    assert _grad(plan=none, g=None) == 0
    assert _quantize(rows=0, x=None, q=None, s=None) == 0 and _quantize(rows=0, plan=none, x=None, q=None, s=None) == 0
    assert _product(m=0, a=None, out=None) == 0


def test_binding_refuses_host_tensors_and_wrong_shapes():
    x, idx = torch.zeros(4, 64), torch.zeros(4, 8, dtype=torch.int32)
    with pytest.raises(ValueError):
        ts.ds_expert_sort(idx, 64)
    plan = ts.ExpertPlan(idx, torch.zeros(32, dtype=torch.int32), torch.zeros(65, dtype=torch.int32))
    for call in (lambda: ts.ds_expert_gather(x, plan), lambda: ts.ds_expert_combine(x, plan),
                 lambda: ts.ds_expert_combine_grad(x, x, plan), lambda: ts.ds_block_quantize(x),
                 lambda: ts.ds_block_product(x, x, x, x), lambda: ts.ds_block_quantize(x[None], ts.BLOCK_ROW),
                 lambda: ts.ds_block_quantize(x[None], ts.BLOCK_TILE)):
        with pytest.raises((ValueError, TypeError)):
            call()
    with pytest.raises(ts.DSError):
        ts.ds_expert_capacity(4, 8, 64, 0)


def test_oracle_rounding_is_torchs():
    g = torch.Generator().manual_seed(5)
    for name, dt, top in (("e4m3", torch.float8_e4m3fn, 448.0), ("e5m2", torch.float8_e5m2, 57344.0)):
        every = torch.arange(256, dtype=torch.uint8).view(dt).double()
        every = every[every.isfinite()]
        mid = (every.sort()[0][1:] + every.sort()[0][:-1]) / 2  # ties
        v = torch.cat([every, mid, (2 * torch.rand(4000, generator=g).double() - 1) * top,
                       torch.randn(4000, generator=g).double() * 2.0 ** -8])
        want = v.float().to(dt).double()
        assert np.array_equal(orc.round8(v.float().double().numpy(), name), want.numpy())
