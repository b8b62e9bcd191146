"""Host-side checks of the row operators' C ABI and binding (no GPU needed): constants and
structs match the header, and invalid calls are refused before the device is touched. Valid
calls with no rows return at once."""
import ctypes
import random
import re

import pytest
import torch

import top_selection_amd as ts

FAKE = 0x10000  # aligned; never dereferenced by a refused call
BIG = ts.DS_ERR_UNSUPPORTED
BAD = ts.DS_ERR_INVALID_ARG
ALIGN = ts.DS_ERR_ALIGNMENT
CFG = ts._binding.ds_route_config


def _cfg(**kw):
    c = CFG(ts.SCORE_SOFTMAX, 1, 1, 1, 0, 1.0)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _route(x=FAKE, rows=4, experts=64, stride=None, k=6, dtype=ts.BF16, bias=None, cfg=None, w=FAKE, idx=FAKE,
           counts=None):
    c = ctypes.byref(cfg) if cfg is not None else None
    return ts.lib().ds_route(x, rows, experts, experts if stride is None else stride, k, dtype, bias, c, w, idx,
                             counts, None)


def _route_grad(x=FAKE, rows=4, experts=64, stride=None, k=6, dtype=ts.BF16, cfg=None, idx=FAKE, g=FAKE, out=FAKE,
                gstride=None):
    c = ctypes.byref(cfg) if cfg is not None else None
    return ts.lib().ds_route_grad(x, rows, experts, experts if stride is None else stride, k, dtype, c, idx, g, out,
                                  experts if gstride is None else gstride, None)


def _softmax(x=FAKE, rows=4, n=1000, stride=None, dtype=ts.BF16, t=None, out=2 * FAKE, ostride=None, odtype=ts.FP32,
             ws=FAKE, ws_bytes=1 << 40):
    return ts.lib().ds_softmax(x, rows, n, n if stride is None else stride, dtype, t, out,
                               n if ostride is None else ostride, odtype, ws, ws_bytes, None)


def _list(vals=FAKE, idx=FAKE, rows=4, k=50, dtype=ts.BF16, ks=None, t=None, p=None, n=1000, out=FAKE, ostride=None,
          odtype=ts.FP32, lists=None):
    return ts.lib().ds_topk_softmax(vals, idx, rows, k, dtype, ks, t, p, n, out, n if ostride is None else ostride,
                                    odtype, lists, None)


def _verify(target=FAKE, tstride=None, draft=FAKE, dstride=None, tokens=FAKE, lens=None, u=FAKE, v=FAKE, batch=4,
            drafts=3, n=1000, dtype=ts.BF16, out=FAKE, acc=FAKE, ws=FAKE, ws_bytes=1 << 40):
    return ts.lib().ds_verify(target, n if tstride is None else tstride, draft, n if dstride is None else dstride,
                              tokens, lens, u, v, batch, drafts, n, dtype, out, acc, ws, ws_bytes, None)


def test_names_are_declared_and_bound():
    names = set(ts.header_functions())
    new = {"ds_route", "ds_route_grad", "ds_softmax", "ds_softmax_workspace_size", "ds_topk_softmax", "ds_verify",
           "ds_verify_workspace_size"}
    assert new <= names
    for n in new:
        assert callable(getattr(ts, n)) and hasattr(ts.lib(), n)


def test_constants_and_struct_match_the_header():
    text = open(ts._binding.HEADER_PATH).read()
    for name in ("DS_MAX_EXPERTS", "DS_MAX_ROUTE_K", "DS_MAX_ROUTE_GROUPS", "DS_MAX_DRAFTS"):
        assert int(re.search(rf"#define {name} (\d+)", text).group(1)) == getattr(ts, name)
    for name, value in (("DS_SCORE_SOFTMAX", ts.SCORE_SOFTMAX), ("DS_SCORE_SIGMOID", ts.SCORE_SIGMOID)):
        assert int(re.search(rf"#define {name} (\d+)", text).group(1)) == value
    body = re.search(r"typedef struct ds_route_config \{(.*?)\}", text, re.S).group(1)
    assert re.findall(r"(?:int32_t|float)\s+(\w+);", body) == [f for f, _ in CFG._fields_]
    assert ctypes.sizeof(CFG) == 24


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), BAD), (dict(rows=-1), BAD), (dict(experts=0), BAD), (dict(stride=63), BAD), (dict(k=0), BAD),
    (dict(k=65), BAD), (dict(experts=1025), BIG), (dict(experts=512, k=65), BIG), (dict(x=None), BAD),
    (dict(w=None, idx=None), BAD), (dict(idx=None, counts=FAKE), BAD), (dict(cfg=_cfg(score=2)), BAD), (dict(cfg=_cfg(groups=-1)), BAD),
    (dict(cfg=_cfg(groups=5)), BAD), (dict(cfg=_cfg(groups=4, topk_groups=5)), BAD),
    (dict(cfg=_cfg(groups=16, topk_groups=1)), BAD),  # four experts for k = 6
    (dict(cfg=_cfg(groups=4, topk_groups=2, group_top=3)), BAD), (dict(cfg=_cfg(groups=64, topk_groups=64, group_top=2)), BAD),
    (dict(experts=128, cfg=_cfg(groups=128, topk_groups=128)), BIG), (dict(cfg=_cfg(scale=float("inf"))), BAD),
    (dict(cfg=_cfg(scale=float("nan"))), BAD), (dict(x=FAKE + 1), ALIGN), (dict(x=FAKE + 2, dtype=ts.FP32), ALIGN),
    (dict(bias=FAKE + 2), ALIGN), (dict(w=FAKE + 2), ALIGN), (dict(idx=FAKE + 1), ALIGN),
    (dict(counts=FAKE + 3), ALIGN), (dict(rows=1 << 60, stride=1 << 20), BAD),
])
def test_route_refusals(kw, code):
    assert _route(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), BAD), (dict(k=0), BAD), (dict(gstride=63), BAD), (dict(stride=63), BAD), (dict(x=None), BAD),
    (dict(idx=None), BAD), (dict(g=None), BAD), (dict(out=None), BAD), (dict(experts=2048), BIG),
    (dict(out=FAKE + 1), ALIGN), (dict(g=FAKE + 2), ALIGN), (dict(idx=FAKE + 2), ALIGN), (dict(cfg=_cfg(score=-1)), BAD),
])
def test_route_grad_refusals(kw, code):
    assert _route_grad(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), BAD), (dict(odtype=-1), BAD), (dict(rows=-1), BAD), (dict(n=0), BAD), (dict(n=1 << 31), BAD),
    (dict(stride=999), BAD), (dict(ostride=999), BAD), (dict(x=None), BAD), (dict(out=None), BAD),
    (dict(x=FAKE + 1), ALIGN), (dict(out=FAKE + 2), ALIGN), (dict(t=FAKE + 2), ALIGN),
    (dict(x=FAKE, out=FAKE), BAD),  # in place
])
def test_softmax_refusals(kw, code):
    assert _softmax(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), BAD), (dict(odtype=2), BAD), (dict(k=0), BAD), (dict(k=1001), BAD), (dict(k=4097, n=10000), BIG),
    (dict(n=0), BAD), (dict(rows=-1), BAD), (dict(ostride=999), BAD), (dict(vals=None), BAD), (dict(idx=None), BAD),
    (dict(out=None), BAD), (dict(idx=FAKE + 2), ALIGN), (dict(ks=FAKE + 1), ALIGN), (dict(p=FAKE + 1), ALIGN),
    (dict(lists=FAKE + 2), ALIGN), (dict(out=FAKE + 2), ALIGN),
])
def test_list_softmax_refusals(kw, code):
    assert _list(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), BAD), (dict(batch=-1), BAD), (dict(drafts=-1), BAD), (dict(drafts=65), BIG), (dict(n=0), BAD),
    (dict(tstride=999), BAD), (dict(dstride=999), BAD), (dict(target=None), BAD), (dict(tokens=None), BAD),
    (dict(u=None), BAD), (dict(v=None), BAD), (dict(out=None), BAD), (dict(acc=None), BAD),
    (dict(target=FAKE + 1), ALIGN), (dict(draft=FAKE + 1), ALIGN), (dict(lens=FAKE + 2), ALIGN),
    (dict(ws=FAKE + 4, n=200000), ALIGN), (dict(ws=None, n=200000), ts.DS_ERR_WORKSPACE),
    (dict(ws_bytes=8, n=200000), ts.DS_ERR_WORKSPACE),
])
def test_verify_refusals(kw, code):
    assert _verify(**kw) == code


def test_no_rows_is_a_no_op():
    assert _route(rows=0, x=None) == ts.DS_OK
    assert _route_grad(rows=0, x=None) == ts.DS_OK
    assert _softmax(rows=0, x=None) == ts.DS_OK
    assert _list(rows=0, vals=None) == ts.DS_OK
    assert _verify(batch=0, target=None) == ts.DS_OK


def test_workspace_sizes():
    for f in (ts.ds_softmax_workspace_size, ts.ds_verify_workspace_size):
        assert f(0, 1000, ts.FP32) >= 0
        assert f(1, 129280, ts.FP32) <= 1 << 20
        assert f(4096, 129280, ts.BF16) <= 1 << 24
        for bad in ((-1, 10, ts.FP32), (1, 0, ts.FP32), (1, 10, 5)):
            with pytest.raises(ts.DSError) as e:
                f(*bad)
            assert e.value.status == BAD


def test_binding_refuses_host_tensors_and_wrong_shapes():
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        ts.ds_route(x, 4)
    with pytest.raises(ValueError):
        ts.ds_route_grad(x, torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2))
    with pytest.raises(ValueError):
        ts.ds_softmax(x)
    with pytest.raises(ValueError):
        ts.ds_topk_softmax(x, torch.zeros(4, 64, dtype=torch.int32), 100)
    with pytest.raises(ValueError):
        ts.ds_verify(torch.zeros(2, 3, 10), None, torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 2), torch.zeros(2))
    for dim in (1, 3):
        with pytest.raises(ValueError):
            ts.ds_softmax(torch.zeros([2] * dim))


@pytest.mark.parametrize("dtype,odtype", [(ts.FP32, ts.FP32), (ts.BF16, ts.BF16), (ts.BF16, ts.FP32)])
def test_softmax_refuses_shared_memory_and_nothing_else(dtype, odtype):
    """Against every pair of rows, one by one. Rows this long need a workspace, and without one a valid call is
    refused for that: none gets as far as the device."""
    rows, n = 3, 140000
    xb, ob = (2 if d == ts.BF16 else 4 for d in (dtype, odtype))
    rng = random.Random(dtype + 2 * odtype)
    seen = set()
    for case in range(400):
        stride = n + rng.choice([0, 1, 9, n, 2 * n, 5 * n])
        ostride = stride * xb // ob if case % 2 and stride * xb >= n * ob else n + rng.choice([0, 3, n, 3 * n])
        x = 1 << 30
        out = x + ob * rng.choice([-1, 0, 1, n, -n, n - 1, 1 - n, rng.randint(-6 * n, 6 * n), stride, -stride, stride + n])
        meet = any(x + i * stride * xb < out + j * ostride * ob + n * ob and out + j * ostride * ob < x + i * stride * xb + n * xb
                   for i in range(rows) for j in range(rows))
        got = _softmax(x=x, out=out, rows=rows, n=n, stride=stride, ostride=ostride, dtype=dtype, odtype=odtype, ws=None)
        assert got == (BAD if meet else ts.DS_ERR_WORKSPACE), (stride, ostride, out - x)
        seen.add((meet, stride * xb == ostride * ob))
    assert len(seen) == 4


@pytest.mark.parametrize("dtype", [ts.FP32, ts.BF16])
def test_route_grad_refuses_shared_memory(dtype):
    """Everything but x itself with its own stride."""
    b = 2 if dtype == ts.BF16 else 4
    x = 1 << 30
    for out, stride, gstride in ((x + b, 64, 64), (x - 63 * b, 64, 64), (x + 101 * b, 164, 164), (x, 64, 65), (x, 100, 64),
                                 (x + 4 * 64 * b - b, 64, 64), (x + 3 * 100 * b, 100, 64)):
        assert _route_grad(x=x, out=out, stride=stride, gstride=gstride, dtype=dtype) == BAD, (out - x, stride, gstride)
