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


def _softmax(x, t):
    """The definition with an infinite temperature as the limit: no mass at -inf, else as much at any logit."""
    x, t = _np(x), np.broadcast_to(np.asarray(t, np.float64), len(x))[:, None]
    m = x.max(axis=1, keepdims=True)
    with np.errstate(over="ignore", invalid="ignore"):
        e = np.where(x == -np.inf, 0.0, np.exp(np.where(x == m, 0.0, x - m) / t))
    return e / np.maximum(e.sum(axis=1, keepdims=True), 1e-300)


@pytest.mark.parametrize("dtype,shape", EACH)
def test_softmax_small_temperatures(dtype, shape):
    """Temperatures by decades from 1e-4 to 1e-30: the mass moves to the maxima."""
    rows, n = shape
    for first in ((4, 13, 22) if rows < 27 else (4,)):
        t = torch.tensor([10.0 ** -(first + r % (9 if rows < 27 else 27)) for r in range(rows)])
        x = 10 + 4 * torch.randn(rows, n, generator=_gen(n + first))
        x[1::2] -= 50  # maxima on both sides of zero
        x = x.to(DT[dtype])
        x[:, n - 2] = x.max(dim=1)[0]  # a tie
        p = ts.ds_softmax(x.cuda(), temperature=t.cuda())
        _close(p, _softmax(x, _np(t)), f"softmax {shape} {dtype} t from 1e-{first}")


@pytest.mark.parametrize("dtype,shape", EACH)
def test_softmax_logits_far_from_zero(dtype, shape):
    """Rows whose logits are all near one number of either sign, from 1e9 to 1e37, a few steps of their type
    apart, at temperature 1 and at one of about a step; and rows of a mask alone."""
    rows, n = shape
    step = 2.0 ** (-7 if dtype == "bf16" else -22)
    base = torch.tensor([(-1.0) ** r * 10.0 ** (9 + 3.5 * (r % 9)) for r in range(rows)])
    x = (base[:, None] * (1 + step * torch.randint(0, 3, (rows, n), generator=_gen(n)))).to(DT[dtype])
    x[3] = -1e10
    x[4] = torch.finfo(DT[dtype]).min
    for t in (torch.ones(rows), base.abs() * step):
        p = ts.ds_softmax(x.cuda(), temperature=t.cuda())
        _close(p, _softmax(x, _np(t)), f"softmax {shape} {dtype} t[0]={float(t[0])}")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("n,k,groups,tg,top", [(100, 7, 5, 3, 2), (256, 8, 8, 4, 2), (64, 6, 4, 2, 1)])
def test_route_groups_beside_large_biases(score, n, k, groups, tg, top):
    """Biases beside which scores vanish, in sums as in single ones: groups tie in double and the smaller ones are
    chosen; ranges of biases that fp32 does not hold."""
    x = (1.5 * torch.randn(40, n, generator=_gen(n))).cuda()
    size = n // groups
    ends = torch.zeros(n)
    ends[-size:] = 3e38
    ends[:size] = -3e38
    near = 3e38 * (1 - 2.0 ** -20 * torch.rand(n, generator=_gen(k)))
    near[:size] = -3e38
    one = torch.zeros(n)
    one[size] = -3e38
    one[-1] = 3e38
    for label, bias in (("1e12", torch.full((n,), 1e12)), ("1e15", torch.full((n,), 1e15)), ("1e20", torch.full((n,), 1e20)),
                        ("-1e17", torch.full((n,), -1e17)), ("ends", ends), ("near", near), ("one", one)):
        for dtype in DT.values():
            kw = dict(groups=groups, topk_groups=tg, group_top=top, renormalize=True)
            code = ts.SCORE_SIGMOID if score == "sigmoid" else ts.SCORE_SOFTMAX
            w, i = ts.ds_route(x.to(dtype), k, bias=bias.cuda(), score=code, **kw)
            ww, wi = orc.route(_np(x.to(dtype)), k, _np(bias), score, **kw)
            assert np.array_equal(_np(i), wi), f"{label} {dtype}"
            _close(w, ww, f"{label} {dtype}")


@pytest.mark.parametrize("dtype,shape", EACH)
def test_softmax_large_temperatures(dtype, shape):
    """Temperatures up to infinity against logits up to the type's ends: what is finite keeps its share."""
    rows, n = shape
    top = torch.finfo(DT[dtype]).max
    x = torch.randn(rows, n, generator=_gen(n))
    x[1::3] *= 2e37
    x[2::3, ::5] = -top
    x[3::6, 1::7] = top
    x[4::6, 2::7] = -np.inf
    x = x.clamp(-top, top).to(DT[dtype])
    x[4::6, 2::7] = -np.inf
    t = torch.tensor([(float("inf"), 3e38, 1.2e38, 1e38, 2e37, 1e36, 1e30)[r % 7] for r in range(rows)])
    p = ts.ds_softmax(x.cuda(), temperature=t.cuda())
    _close(p, _softmax(x, _np(t)), f"softmax {shape} {dtype}")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,n,k", [(21, 5000, 300), (21, 5000, 1000), (260, 70001, 64)])
def test_list_softmax_large_temperatures(dtype, rows, n, k):
    top = torch.finfo(DT[dtype]).max
    x = 1e37 * torch.randn(rows, k, generator=_gen(k))
    x[:, ::5] = -top
    x[1::3, ::7] = top
    x = x.clamp(-top, top).to(DT[dtype])
    x[2::3, 3::4] = -np.inf
    vals, at = x.sort(dim=1, descending=True, stable=True)
    t = torch.tensor([(float("inf"), 3e38, 1.2e38, 1e38, 2e37, 1e36, 1.0)[r % 7] for r in range(rows)])
    idx = (at * (n // k)).to(torch.int32)
    lists = torch.empty(rows, k, device="cuda")
    p = ts.ds_topk_softmax(vals.cuda(), idx.cuda(), n, temperature=t.cuda(), out_list=lists)
    want = _softmax(vals, _np(t))
    _close(lists, want, f"list {dtype}")
    _close(p.gather(1, idx.cuda().long()), want, f"rows {dtype}")
    assert (p != 0).sum().item() == (lists != 0).sum().item()


@pytest.mark.parametrize("dtype,shape", EACH)
def test_softmax_equal_logits_have_equal_probabilities(dtype, shape):
    """A row's probabilities are a function of its logits that never falls: one sum divides all of them."""
    rows, n = shape
    t = 0.3 + torch.rand(rows, generator=_gen(rows))
    x = torch.randn(rows, n, generator=_gen(n))
    x = ((x * 8).round() / 8).to(DT[dtype]).cuda()
    s, order = x.sort(dim=1)
    p = ts.ds_softmax(x, temperature=t.cuda()).gather(1, order)
    assert (p[:, 1:] >= p[:, :-1]).all()
    assert torch.equal(p[:, 1:] == p[:, :-1], s[:, 1:] == s[:, :-1])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,n", [(48, 1 << 25), (47, 1 << 26)])
def test_softmax_sums_of_very_long_rows(rows, n, dtype):
    """Rows of two values, so that every thread adds thousands of equal terms below its maximum's: one by one
    in fp32 they would all be rounded to one side. (In one workgroup, in slices.)"""
    c = -(torch.arange(rows) + 1) / 32  # exact in both types
    x = c.to(DT[dtype]).cuda()[:, None].repeat(1, n)
    x.view(rows, -1, 1 << 19)[:, :, :8192] = 0.0
    p = ts.ds_softmax(x)
    del x
    e, ones = np.exp(_np(c)), (n >> 19) * 8192
    total = ones + (n - ones) * e
    _close(p[:, [0, 8192, n - 1]], np.stack([1 / total, e / total, e / total], axis=1), f"softmax {rows}x{n} {dtype}")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_scales_past_the_scores(dtype, score):
    """Renormalised weights whose scale divided by the scores' sum is past fp32 (the weights are not)."""
    x = torch.randn(20, 48, generator=_gen(7))
    bias = None
    if score == "sigmoid":
        x -= torch.tensor([20.0, 40.0, 60.0, 66.0]).repeat(5)[:, None]
    else:  # the experts with mass are masked by their biases
        x[:, :8] += torch.tensor([20.0, 40.0, 60.0, 66.0]).repeat(5)[:, None]
        bias = torch.zeros(48)
        bias[:8] = -np.inf
    x = x.to(DT[dtype])
    for scale in (1.0, 1e12, 3e38, -1e30, 1e-30):
        w, i = ts.ds_route(x.cuda(), 5, bias=None if bias is None else bias.cuda(), score=ts.SCORE_SIGMOID if score == "sigmoid" else ts.SCORE_SOFTMAX,
                           renormalize=True, scale=scale)
        scale = float(np.float32(scale))
        ww, wi = orc.route(_np(x), 5, None if bias is None else _np(bias), score, renormalize=True)
        assert np.array_equal(_np(i), wi)
        _close(w.double() / scale, ww, f"scale {scale}")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("k", [6, 700])
def test_top_p_of_one_keeps_every_entry(dtype, k):
    """The prefix that holds all of the mass is the list, entries below a double's step of it included."""
    vals = torch.cat([torch.tensor([3.0, 2.0, -37.0, -40.0, -60.0]), -70 - torch.arange(k - 5) / 64]).to(DT[dtype])
    vals = vals.repeat(4, 1).cuda()
    idx = torch.arange(k, dtype=torch.int32, device="cuda").repeat(4, 1)
    ks = torch.tensor([k, 5, 3, 1], dtype=torch.int32, device="cuda")
    top_p = torch.tensor([1.0, 1.0, 1.5, 1.0], device="cuda")
    got, want = (ts.ds_topk_softmax(vals, idx, 1000, ks=ks, top_p=q, rows_out=False) for q in (top_p, None))
    assert torch.equal(got, want) and (got > 0).sum(dim=1).tolist() == ks.tolist()


def test_softmax_between_its_logits():
    """Logits and probabilities as columns of one matrix share no memory; anything else is refused."""
    wide = torch.randn(70, 1300, generator=_gen(3)).cuda()
    want = ts.ds_softmax(wide[:, :640].clone())
    got = ts.ds_softmax(wide[:, :640], out=wide[:, 650:1290])
    assert torch.equal(got, want)
    for out in (wide[:, :640], wide[:, 639:1279], wide[:, 1:641]):
        with pytest.raises(ts.DSError):
            ts.ds_softmax(wide[:, :640], out=out)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,n,k", [(1, 9, 2), (300, 61, 6), (130, 256, 8), (50, 1024, 64)])
def test_route_grad_over_its_logits(rows, n, k, dtype):
    """The gradient may go over the logits: every row is read before it is written."""
    full = torch.randn(rows, n + 3, generator=_gen(n)).to(DT[dtype]).cuda()
    idx = torch.rand(rows, n, generator=_gen(k)).argsort(dim=1)[:, :k].to(torch.int32).contiguous().cuda()
    g = torch.randn(rows, k, generator=_gen(k)).cuda()
    for score in (ts.SCORE_SOFTMAX, ts.SCORE_SIGMOID):
        for renorm in (False, True):
            wide = full.clone()
            x = wide[:, 2:n + 2]
            want = ts.ds_route_grad(x, idx, g, score=score, renormalize=renorm)
            got = ts.ds_route_grad(x, idx, g, score=score, renormalize=renorm, out=x)
            assert got is x and torch.equal(got, want)
            assert torch.equal(wide[:, :2], full[:, :2]) and torch.equal(wide[:, n + 2:], full[:, n + 2:])


def test_route_grad_between_its_logits():
    wide = torch.randn(100, 140, generator=_gen(5)).cuda()
    x = wide[:, 3:64]
    _, idx = ts.ds_route(x, 6)
    g = torch.randn(100, 6, generator=_gen(6)).cuda()
    want = ts.ds_route_grad(x, idx, g)
    assert torch.equal(ts.ds_route_grad(x, idx, g, out=wide[:, 64:125]), want)
    with pytest.raises(ts.DSError):
        ts.ds_route_grad(x, idx, g, out=wide[:, 63:124])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n", [700, 40001, 129280])
def test_verify_past_a_drafts_end(dtype, n):
    """What lies past a sequence's length takes no part: rows of NaN, tokens and numbers of any value."""
    g = _gen(n)
    B, K = 6, 4
    target = torch.softmax(2 * torch.randn(B, K + 1, n, generator=g), dim=2).to(DT[dtype])
    draft = torch.softmax(2 * torch.randn(B, K, n, generator=g), dim=2).to(DT[dtype])
    tokens = draft.float().argmax(dim=2).to(torch.int32)
    u, v = 0.3 * torch.rand(B, K, generator=g), torch.rand(B, generator=g)
    lens = torch.tensor([0, 1, 2, 3, 4, 0], dtype=torch.int32)
    want, wacc = orc.verify(_np(target), _np(draft), _np(tokens), _np(u), _np(v), _np(lens))
    certain, cacc = orc.verify(_np(target), None, _np(tokens), _np(u), _np(v), _np(lens))
    for b, m in enumerate(lens.tolist()):
        target[b, m + 1:] = draft[b, m:] = u[b, m:] = float("nan")
        tokens[b, m:] = torch.tensor([-2 ** 31, 2 ** 31 - 1, -1, n][:K - m], dtype=torch.int32)
    got, acc = ts.ds_verify(target.cuda(), draft.cuda(), tokens.cuda(), u.cuda(), v.cuda(), draft_lens=lens.cuda())
    assert np.array_equal(_np(got), want) and np.array_equal(_np(acc), wacc)
    got, acc = ts.ds_verify(target.cuda(), None, tokens.cuda(), u.cuda(), v.cuda(), draft_lens=lens.cuda())
    assert np.array_equal(_np(got), certain) and np.array_equal(_np(acc), cacc)


@pytest.mark.parametrize("shape", SHAPES["fp32"])
def test_softmax_of_fp32s_least_differences(shape):
    """Logits a few of fp32's least numbers apart, at temperatures that tell them apart and at ones whose inverse
    is past fp32 (the limit: the maxima share the mass)."""
    rows, n = shape
    x = (2.0 ** -149 * torch.randint(-3, 1, (rows, n), generator=_gen(n)).double()).float()
    t = torch.tensor([(1e-37, 2e-38, 1e-39, 1e-40, 1e-44)[r % 5] for r in range(rows)])
    p = ts.ds_softmax(x.cuda(), temperature=t.cuda())
    _close(p, _softmax(x, np.where(_np(t) < 4e-39, 1e-300, _np(t))), f"softmax {shape}")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_route_logits_of_a_finite_mask(dtype):
    """Sigmoid scores that vanish in double: rows of masks alone have no weights and no gradient, rows with
    some experts left have those. And the last scores that double holds."""
    n, k = 48, 6
    x = torch.randn(24, n, generator=_gen(71))
    lows = [torch.finfo(DT[dtype]).min, -1e30, -1e10, -1000.0, -760.0, -720.0]
    for r in range(24):
        x[r, torch.randperm(n, generator=_gen(r))[(0, 3, 8, 48)[r // 6] if r % 6 < 5 else 0:]] = lows[r % 6]
    x[5::6] += (4 * torch.rand(4, n, generator=_gen(72))).to(DT[dtype]).float()  # -720 to -716
    x = x.to(DT[dtype])
    g = torch.randn(24, k, generator=_gen(73))
    for bias in (None, 0.1 * torch.randn(n, generator=_gen(74))):
        w, i = ts.ds_route(x.cuda(), k, bias=None if bias is None else bias.cuda(), score=ts.SCORE_SIGMOID, renormalize=True)
        ww, wi = orc.route(_np(x), k, None if bias is None else _np(bias), "sigmoid", renormalize=True)
        assert np.array_equal(_np(i), wi)
        _close(w, ww, "weights")
        at = [r for r in range(24) if r % 6 < 5]  # (a division by the least of doubles overflows in the definition)
        dx = _np(ts.ds_route_grad(x.cuda(), i, g.cuda(), score=ts.SCORE_SIGMOID, renormalize=True))
        want, size = orc.route_grad(_np(x)[at], wi[at], _np(g)[at], "sigmoid", True, 1.0)
        _close(torch.from_numpy(dx[at]), want, "gradient", size=4 * size, bf16=dtype == "bf16")
        # (from the weights where the scores are ratios: dx_e = w_e (g_e - sum g w), 1 - s is 1)
        for r in range(5, 24, 6):
            d = np.zeros(n)
            v = np.exp(_np(x)[r][wi[r]] + 720.0)
            v = v / v.sum()
            d[wi[r]] = v * (_np(g)[r] - (_np(g)[r] * v).sum())
            _close(torch.from_numpy(dx[r:r + 1]), d[None], "gradient", size=np.full((1, n), 8.0), bf16=dtype == "bf16")


MEAN = 2.0 ** -19  # 32 u, u = 2^-24 as in test_gpu_rows.py


def _mean_close(got, want, label):
    """The mean relative error of a row's fp32 numbers. The roundings are independent of each other and at most
    u, so their squares' mean is at most u^2 / 3, and errors add as their squares: 3 in an exponent, 8 at most
    here with its distance from the maximum (3 * 64 / 3 = 64 u^2), 140 additions on the path of a sum (47), the
    sum's own exponents (64 again, were they all alike), exp2, two divisions and a product (4): 180 u^2, the
    square of 13.4 u. The mean is not above the root of the mean square; 32 u is 2.4 times that."""
    got, want = _np(got), np.asarray(want)
    live = want > 0
    err = np.where(live, np.abs(got - want) / np.where(live, want, 1), 0).sum(axis=1) / np.maximum(live.sum(axis=1), 1)
    assert err.max() < MEAN, f"{label}: {err.max() * 2 ** 24} u"


@pytest.mark.parametrize("dtype,shape", EACH)
def test_softmax_mean_error(dtype, shape):
    rows, n = shape
    x = torch.randn(rows, n, generator=_gen(n)).clamp(-4, 4).to(DT[dtype])
    _mean_close(ts.ds_softmax(x.cuda()), _softmax(x, 1.0), f"softmax {shape} {dtype}")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n,k,groups,tg", [(256, 8, 8, 4), (61, 6, 1, 1), (1024, 16, 1, 1), (256, 20, 1, 1)])
def test_route_mean_error(n, k, groups, tg, dtype):
    """The chosen experts' weights, over all rows at once (a row has few)."""
    x = torch.randn(300, n, generator=_gen(n)).clamp(-4, 4).to(DT[dtype])
    for name, code in (("softmax", ts.SCORE_SOFTMAX), ("sigmoid", ts.SCORE_SIGMOID)):
        for renorm in (False, True):
            w, i = ts.ds_route(x.cuda(), k, score=code, groups=groups, topk_groups=tg, renormalize=renorm, scale=2.5)
            ww, wi = orc.route(_np(x), k, None, name, groups, tg, 1, renorm, 2.5)
            assert np.array_equal(_np(i), wi)
            _mean_close(w.reshape(1, -1), ww.reshape(1, -1), f"route {name} {renorm}")
