"""Row operators on the GPU against their 64-bit definitions (oracle/rows.py).

Integers (experts, tokens, counts) have to be equal. Tolerances of floats, derived for the
inputs used here (finite logits within 16 of their row's maximum where a relative bound is
used; in units of u = 2^-24, half a step of fp32):
  * exp of d: the argument d * log2(e) / t carries 3 roundings, which move exp by 3 |d| u
    relative (at most 48 u), the exp2 instruction 2 u, so a score before its division has
    at most 50 u; sums of scores carry their terms' error plus half a step per addition on
    a path (at most 300 here), divisions 4 u. Quotients: (50 + 50 + 300 + 4) u < 2^-15.
  * an element d below that range has exp(d) 3 |d| u < 3 e^-1 u of the row's maximum: 2^-22
    of the row's largest value, as an absolute term.
  * exp below fp32's least normal number, 2^-126, is held as 0; it is multiplied by gradients
    and scales below 2^6 here: 2^-120, whatever the row's largest value.
  * a result held in bf16 adds half a step, 2^-8 relative (fp32: 2^-24, contained above).
"""
import numpy as np
import pytest
import torch

import top_selection_amd as ts
from gpu_util import say
from oracle import rows as orc

pytestmark = pytest.mark.gpu

RTOL, ATOL, LEAST = 2.0 ** -15, 2.0 ** -22, 2.0 ** -120
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
NEG = float("-inf")


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _np(t):
    t = t.detach().cpu()
    return t.double().numpy() if t.is_floating_point() else t.numpy()


def _close(got, want, label, size=None, bf16=False):
    """|got - want| within the module's tolerance; size: the values' magnitude before they cancel."""
    got = _np(got)
    assert np.isfinite(got).all(), label
    big = np.abs(want) if size is None else size
    top = np.abs(big).max(axis=-1, keepdims=True) if big.size else 0
    tol = RTOL * big + ATOL * top + LEAST + (2.0 ** -8 * np.abs(want) if bf16 else 0)
    bad = np.abs(got - want) > tol
    assert not bad.any(), f"{label}: {bad.sum()} of {bad.size} off, worst {np.max(np.abs(got - want) - tol)}"


def _logits(seed, rows, n, dtype, kind="normal"):
    g = _gen(seed)
    x = 1.5 * torch.randn(rows, n, generator=g)
    if kind == "ties":
        x = (x * 2).round() / 2 + 0.125  # a grid without a and -a: sigmoid(a) + sigmoid(-a) is 1 for every a
    elif kind == "masked":
        x[torch.rand(rows, n, generator=g) < 0.6] = NEG
        x[::3] = NEG  # rows that the mask leaves empty
        if rows > 1:
            x[1] = NEG
            x[1, n // 2] = 0.25  # one expert left
    elif kind == "far":
        x = 60 * x
    elif kind == "inf":
        x[::2, 0] = float("inf")
        x[::2, n - 1] = float("inf")
        x[1::2, n // 3] = NEG
    return x.to(dtype).cuda()


# ------------------------------------------------------------------------------ routing
ROUTES = [  # rows, experts, k, groups, topk_groups, group_top
    (1, 1, 1, 1, 1, 1), (3, 2, 2, 1, 1, 1), (5, 7, 3, 1, 1, 1), (4, 64, 64, 1, 1, 1), (37, 61, 6, 1, 1, 1),
    (33, 256, 8, 8, 4, 2), (64, 160, 6, 8, 3, 1), (9, 63, 5, 3, 2, 2), (17, 384, 9, 1, 1, 1), (6, 1024, 64, 64, 32, 2),
    (5, 1000, 10, 8, 1, 2), (11, 512, 16, 64, 5, 1), (130, 16, 4, 16, 8, 1), (2, 130, 20, 2, 2, 2), (3, 8, 2, 4, 1, 2),
    (66, 32, 5, 4, 2, 2), (21, 128, 1, 1, 1, 1), (19, 100, 12, 5, 3, 2), (40, 384, 8, 8, 4, 2), (7, 300, 9, 6, 3, 2),
    (9, 96, 8, 32, 9, 2), (5, 600, 7, 1, 1, 1), (3, 250, 24, 10, 4, 1), (12, 3, 3, 1, 1, 1),
]


def _check_route(x, k, bias=None, label="", **kw):
    w, i = ts.ds_route(x, k, bias=None if bias is None else bias.cuda(), **kw)
    okw = dict(kw, score="sigmoid" if kw.get("score") == ts.SCORE_SIGMOID else "softmax")
    ww, wi = orc.route(_np(x), k, None if bias is None else _np(bias), **okw)
    assert np.array_equal(_np(i), wi), f"{label}: {np.argwhere(_np(i) != wi)[:4]}"
    _close(w, ww, label)
    return w, i


@pytest.mark.parametrize("shape", ROUTES)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("score", [ts.SCORE_SOFTMAX, ts.SCORE_SIGMOID])
def test_route_matches_definition(shape, dtype, score):
    rows, n, k, groups, tg, top = shape
    for kind in ("normal", "ties", "masked", "far", "inf"):
        for with_bias in (False, True):
            x = _logits(7 * n + k, rows, n, DT[dtype], kind)
            bias = 0.2 * torch.randn(n, generator=_gen(n)) if with_bias else None
            label = f"route {shape} {dtype} score={score} {kind} bias={with_bias}"
            _check_route(x, k, bias, label, score=score, groups=groups, topk_groups=tg, group_top=top,
                         renormalize=(k + with_bias) % 2 == 0, scale=2.5 if with_bias else 1.0)


@pytest.mark.parametrize("score", [ts.SCORE_SOFTMAX, ts.SCORE_SIGMOID])
@pytest.mark.parametrize("n,k,groups,tg,top", [(256, 8, 8, 4, 2), (64, 6, 1, 1, 1), (96, 10, 4, 2, 1)])
def test_route_near_ties_are_decided_exactly(score, n, k, groups, tg, top):
    """Biases that bring every selection score to within about 1e-7 of the others: orders that
    fp32 scores cannot tell apart."""
    rows = 40
    x = _logits(3 + n, 1, n, torch.float32).repeat(rows, 1)
    x += 1e-4 * torch.randn(rows, 1, generator=_gen(5)).cuda()
    name = "sigmoid" if score == ts.SCORE_SIGMOID else "softmax"
    bias = torch.from_numpy(0.5 - orc.scores(_np(x)[0], name)).float()
    _check_route(x, k, bias, f"near ties {name} {n}", score=score, groups=groups, topk_groups=tg, group_top=top,
                 renormalize=True)


@pytest.mark.parametrize("scale", [0.002, 0.2, 1.0, 2.0, 6.0, 20.0])
def test_route_constant_bias_and_tied_bf16_logits(scale):
    """One bias for all and bf16 logits, of which many are equal: around zero, where different
    logits give closer scores than fp32 tells apart, and where the sigmoid saturates."""
    x = (scale * torch.randn(150, 256, generator=_gen(int(10 * scale)))).to(torch.bfloat16)
    x[::5] = x[::5].abs()
    for bias in (None, torch.zeros(256), torch.full((256,), -0.375)):
        for groups, tg, top in ((8, 4, 2), (1, 1, 1), (8, 3, 1)):
            _check_route(x.cuda(), 8, bias, f"flat {scale} {bias is None} {groups}", score=ts.SCORE_SIGMOID, groups=groups,
                         topk_groups=tg, group_top=top, renormalize=True)


@pytest.mark.parametrize("score", [ts.SCORE_SOFTMAX, ts.SCORE_SIGMOID])
def test_route_large_biases(score):
    """Biases beside which scores lose bits even in double, and ranges that no key holds."""
    x = _logits(17, 30, 100, torch.bfloat16)
    r = torch.randn(100, generator=_gen(18))
    for bias in (torch.full((100,), 1e12), 1e9 + 64 * r.round(), 1e6 * r, 1e20 * r, 3e38 * r.clamp(-1, 1), -1e12 + 0 * r):
        _check_route(x, 7, bias, f"large {float(bias[0])}", score=score, groups=5, topk_groups=3, group_top=2)


def test_route_zero_bias_and_equal_logits_give_the_smaller_expert():
    x = torch.zeros(5, 200, device="cuda", dtype=torch.bfloat16)
    x[1] = 3.0
    for score in (ts.SCORE_SOFTMAX, ts.SCORE_SIGMOID):
        for bias in (None, torch.zeros(200)):
            _, i = _check_route(x, 7, bias, "equal", score=score, groups=4, topk_groups=2, group_top=2)
            assert (_np(i) == np.arange(7)).all()


def test_route_masked_by_bias():
    x = _logits(11, 20, 40, torch.float32)
    bias = torch.full((40,), NEG)
    bias[[3, 30, 31]] = torch.tensor([0.1, -0.2, 0.0])
    _, i = _check_route(x, 5, bias, "bias mask", score=ts.SCORE_SIGMOID, renormalize=True, groups=4, topk_groups=2)
    assert (_np(i)[:, 3:] == -1).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_route_strides_counts_and_single_outputs(dtype):
    full = _logits(2, 70, 137, DT[dtype])
    x = full[1::2, 3:64]  # an odd offset, a row stride above the experts
    counts = torch.full((61,), 5, dtype=torch.int32, device="cuda")
    w, i = ts.ds_route(x, 4, counts=counts)
    w2, i2 = _check_route(x, 4, None, "strided")
    assert torch.equal(w, w2) and torch.equal(i, i2)
    want = 5 + np.bincount(_np(i).ravel(), minlength=61)
    assert np.array_equal(_np(counts), want)
    none, i3 = ts.ds_route(x, 4, weights=False)
    assert none is None and torch.equal(i3, i)
    ts.ds_route(x, 4, counts=counts)  # counts add up
    assert np.array_equal(_np(counts), 2 * want - 5)


def test_route_many_rows_counts():
    x = _logits(4, 20011, 64, torch.bfloat16, "ties")
    counts = torch.zeros(64, dtype=torch.int32, device="cuda")
    bias = 0.1 * torch.randn(64, generator=_gen(1))
    w, i = ts.ds_route(x, 6, bias=bias.cuda(), score=ts.SCORE_SIGMOID, renormalize=True, counts=counts)
    pick = torch.randperm(20011, generator=_gen(2))[:300]
    ww, wi = orc.route(_np(x[pick.cuda()]), 6, _np(bias), score="sigmoid", renormalize=True)
    assert np.array_equal(_np(i)[pick], wi)
    _close(w[pick.cuda()], ww, "many rows")
    assert np.array_equal(_np(counts), np.bincount(_np(i).ravel(), minlength=64))


# ----------------------------------------------------------------------------- its gradient
@pytest.mark.parametrize("shape", ROUTES)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_route_grad_matches_definition(shape, dtype):
    rows, n, k, groups, tg, top = shape
    for score in (ts.SCORE_SOFTMAX, ts.SCORE_SIGMOID):
        for renorm in (False, True):
            for kind in ("normal", "masked", "far"):
                x = _logits(3 * n + k, rows, n, DT[dtype], kind)
                _, idx = ts.ds_route(x, k, score=score, groups=groups, topk_groups=tg, group_top=top)
                g = torch.randn(rows, k, generator=_gen(n + 1)).cuda()
                dx = ts.ds_route_grad(x, idx, g, score=score, renormalize=renorm, scale=1.5)
                name = "sigmoid" if score == ts.SCORE_SIGMOID else "softmax"
                want, size = orc.route_grad(_np(x), _np(idx), _np(g), name, renorm, 1.5)
                assert dx.dtype == x.dtype
                # every element is a sum of terms of total magnitude `size`, each with the scores' error
                _close(dx, want, f"grad {shape} {dtype} {name} renorm={renorm} {kind}", size=4 * size,
                       bf16=dtype == "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_route_far_below_zero(dtype):
    """Sigmoid scores that fp32 does not hold: weights and gradients are those of their ratios."""
    x = (_logits(61, 20, 48, torch.float32) - torch.tensor([90.0, 120.0, 300.0, 600.0]).repeat(5)[:, None].cuda()).to(DT[dtype])
    w, i = _check_route(x, 5, None, "far below", score=ts.SCORE_SIGMOID, renormalize=True, scale=2.0)
    assert (w.sum(dim=1) - 2).abs().max() < 1e-5
    g = torch.randn(20, 5, generator=_gen(62)).cuda()
    dx = ts.ds_route_grad(x, i, g, score=ts.SCORE_SIGMOID, renormalize=True, scale=2.0)
    want, size = orc.route_grad(_np(x), _np(i), _np(g), "sigmoid", True, 2.0)
    _close(dx, want, "far below", size=4 * size, bf16=dtype == "bf16")
    assert np.abs(want).max() > 0.1


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_grad_matches_differences(score, renorm):
    """Central differences of the 64-bit weights, step 1e-5: truncation below 1e-10 times the
    third derivative (at most 1 here), rounding 1e-16 / 1e-5; both far below the fp32 bound."""
    x = _logits(21, 6, 24, torch.float32)
    code = ts.SCORE_SIGMOID if score == "sigmoid" else ts.SCORE_SOFTMAX
    _, idx = ts.ds_route(x, 5, score=code)
    g = torch.randn(6, 5, generator=_gen(22))
    dx = _np(ts.ds_route_grad(x, idx, g.cuda(), score=code, renormalize=renorm, scale=2.0))
    xn, i, h = _np(x), _np(idx), 1e-5
    for e in range(24):
        up, dn = xn.copy(), xn.copy()
        up[:, e] += h
        dn[:, e] -= h
        d = (orc.route_weights(up, i, score, renorm, 2.0) - orc.route_weights(dn, i, score, renorm, 2.0)) / (2 * h)
        want = (d * _np(g)).sum(axis=1)
        assert np.abs(dx[:, e] - want).max() < 4 * RTOL * 2.0 * np.abs(_np(g)).max() * 5


def test_route_grad_slots_without_an_expert_strides_and_repeats():
    n, k = 70, 6
    x = _logits(31, 40, n + 5, torch.float32)[:, 2:n + 2]
    idx = torch.stack([torch.randperm(n, generator=_gen(r))[:k] for r in range(40)]).to(torch.int32)
    idx[::2, 3] = -1
    idx[1, :] = -1                     # a row without any
    idx[2, 1], idx[2, 2] = n, 1 << 30  # outside the experts: no expert
    idx[4, 5] = idx[4, 0]              # one expert in two slots
    g = torch.randn(40, k, generator=_gen(8))
    for score, name in ((ts.SCORE_SOFTMAX, "softmax"), (ts.SCORE_SIGMOID, "sigmoid")):
        for renorm in (False, True):
            guard = torch.full((40, n + 9), 7.0, device="cuda")
            out = guard[:, 3:n + 3]
            ts.ds_route_grad(x, idx.cuda(), g.cuda(), score=score, renormalize=renorm, out=out)
            want, size = orc.route_grad(_np(x), idx.numpy(), _np(g), name, renorm, 1.0)
            _close(out, want, f"grad holes {name} {renorm}", size=4 * size)
            assert (guard[:, :3] == 7).all() and (guard[:, n + 3:] == 7).all()  # around the rows: as they were


# ----------------------------------------------------------------------------- probabilities
SOFT = [(1, 1), (3, 2), (2, 63), (5, 1000), (4, 4097), (3, 12289), (2, 50001), (70, 515), (300, 333), (1, 129280), (9, 32000)]


@pytest.mark.parametrize("rows,n", SOFT)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("odt", ["bf16", "fp32"])
def test_softmax_matches_definition(rows, n, dtype, odt):
    for kind in ("normal", "masked", "far", "inf", "ties"):
        x = _logits(n + rows, rows, n, DT[dtype], kind)
        t = 0.5 + torch.rand(rows, generator=_gen(rows))
        t[1::3] = 0.0
        t[2::5] = -1.0
        for temp in (None, t):
            p = ts.ds_softmax(x, temperature=None if temp is None else temp.cuda(), out_dtype=DT[odt])
            want = orc.softmax(_np(x), None if temp is None else _np(temp))
            assert p.dtype == DT[odt]
            _close(p, want, f"softmax {rows}x{n} {dtype}->{odt} {kind} t={temp is not None}", bf16=odt == "bf16")


@pytest.mark.parametrize("rows,n", [(50, 130001), (48, 140003), (49, 40000)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_softmax_long_rows(rows, n, dtype):
    """Rows past what a workgroup holds on chip, with and without a temperature."""
    t = 0.5 + torch.rand(rows, generator=_gen(rows))
    t[1::5] = 0.0
    t[2] = 1e-40
    for kind in ("normal", "inf", "masked", "ties"):
        x = _logits(n, rows, n, DT[dtype], kind)
        p = ts.ds_softmax(x, temperature=t.cuda())
        want = orc.softmax(_np(x), _np(t))
        _close(p, want, f"softmax {rows}x{n} {dtype} {kind}")


@pytest.mark.parametrize("rows,n", [(50, 130001), (48, 300007), (3, 140003), (2, 30001)])
def test_softmax_far_from_zero(rows, n):
    """Logits whose common part is thousands of times their spread: it takes no part in the result."""
    t = 0.3 + torch.rand(rows, generator=_gen(rows))
    for shift in (-3000.0, 3000.0):
        x = (shift + torch.randn(rows, n, generator=_gen(n))).cuda()
        _close(ts.ds_softmax(x, temperature=t.cuda()), orc.softmax(_np(x), _np(t)), f"softmax {rows}x{n} {shift}")


@pytest.mark.parametrize("rows", [1, 8, 9, 17, 32, 33, 47])
@pytest.mark.parametrize("n,dtype", [(8193, "fp32"), (16385, "fp32"), (32001, "fp32"), (16387, "bf16"), (50005, "bf16")])
def test_softmax_few_rows(rows, n, dtype):
    """Rows that several workgroups work out, each for its part of the output, and those that one does."""
    t = 0.5 + torch.rand(rows, generator=_gen(rows))
    t[1::4] = 0.0
    t[2::7] = 1e-40
    for kind in ("normal", "inf", "masked", "ties"):
        x = _logits(n + rows, rows, n, DT[dtype], kind)
        out = torch.full((rows, n + 6), 7.0, device="cuda")
        ts.ds_softmax(x, temperature=t.cuda(), out=out[:, 3:n + 3])
        _close(out[:, 3:n + 3], orc.softmax(_np(x), _np(t)), f"softmax {rows}x{n} {dtype} {kind}")
        assert (out[:, :3] == 7).all() and (out[:, n + 3:] == 7).all()


def test_softmax_extreme_temperatures_spread_or_keep_the_mass():
    """An infinite temperature is uniform over what is not masked; a NaN one counts as not above 0."""
    x = torch.randn(3, 20000, generator=_gen(9))
    x[:, ::4] = NEG
    t = torch.tensor([float("inf"), float("nan"), 1e30])
    want = np.where(np.isinf(x.double().numpy()), 0, 1 / 15000)
    for n in (20000, 40000):  # in one workgroup, in slices
        y = torch.full((3, n), NEG)
        y[:, :20000] = x
        p = _np(ts.ds_softmax(y.cuda(), temperature=t.cuda()))
        assert np.abs(p[[0, 2], :20000] - want[[0, 2]]).max() < 1e-8 and not p[:, 20000:].any()
        assert p[1].sum() == 1 and p[1].argmax() == int(x[1].argmax())
    v, i = x.sort(dim=1, descending=True)
    q = _np(ts.ds_topk_softmax(v[:, :4000].contiguous().cuda(), i[:, :4000].to(torch.int32).contiguous().cuda(), 20000,
                               temperature=t.cuda()))
    assert np.abs(q.max(axis=1) - [1 / 4000, 1, 1 / 4000]).max() < 1e-8


def test_more_rows_than_a_launch_takes():
    """Rows past the workgroups of one launch, and routing past the turns that a wave keeps."""
    rows = (1 << 22) + 5
    x = torch.randn(rows, 3, generator=_gen(2)).to(torch.bfloat16).cuda()
    p = ts.ds_softmax(x)
    assert (p - torch.softmax(x.float(), dim=1)).abs().max() < 1e-6
    v, i = ts.ds_topk_softmax, torch.arange(3, dtype=torch.int32, device="cuda").repeat(rows, 1)
    s = x.float().sort(dim=1, descending=True)
    assert torch.equal(v(s[0].to(torch.bfloat16), s[1].to(torch.int32), 3) > 0, p > 0)
    got, acc = ts.ds_verify(p.view(rows, 1, 3), None, None, None, torch.zeros(rows, device="cuda"))
    assert not got.any() and not acc.any()  # the first element that has mass
    y = torch.randn(rows, 8, generator=_gen(3)).cuda()
    y[-4000::3, 5] = y[-4000::3, 2]  # ties: decided in double
    bias = torch.tensor([0.1, 0.0, 0.2, -0.1, 0.05, 0.2, 0.0, 0.0]).cuda()
    w, e = ts.ds_route(y, 2, bias=bias, score=ts.SCORE_SIGMOID, renormalize=True)
    pick = torch.cat([torch.arange(0, rows, 9001), torch.arange(rows - 4000, rows)])
    ww, we = orc.route(_np(y[pick.cuda()]), 2, _np(bias), score="sigmoid", renormalize=True)
    assert np.array_equal(_np(e[pick.cuda()]), we)
    _close(w[pick.cuda()], ww, "many turns")


@pytest.mark.parametrize("off", [0, 1, 3])
def test_softmax_unaligned_rows_and_untouched_surroundings(off):
    x = _logits(5, 6, 5000, torch.bfloat16)[:, off:off + 4501]
    guard = torch.full((6, 4600), 3.0, device="cuda")
    out = guard[:, 7 + off:7 + off + 4501]
    ts.ds_softmax(x, out=out)
    _close(out, orc.softmax(_np(x)), "unaligned")
    assert (guard[:, :7 + off] == 3).all() and (guard[:, 7 + off + 4501:] == 3).all()


def test_softmax_tiny_temperatures():
    """Temperatures whose inverse overflows fp32: the limit, ties sharing the mass."""
    x = torch.tensor([[1.0, 2.0, 2.0, -3.0], [0.0, -1e-3, 5.0, 4.0]], device="cuda")
    p = ts.ds_softmax(x, temperature=torch.tensor([1e-40, 1e-42], device="cuda"))
    assert torch.equal(p.cpu(), torch.tensor([[0.0, 0.5, 0.5, 0.0], [0.0, 0.0, 1.0, 0.0]]))


@pytest.mark.parametrize("rows,n,k", [(1, 5, 1), (3, 100, 100), (7, 5000, 50), (2, 129280, 512), (5, 8191, 4096),
                                      (300, 777, 13), (4, 40000, 1000)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("odt", ["bf16", "fp32"])
def test_list_softmax_matches_definition(rows, n, k, dtype, odt):
    for kind in ("normal", "masked", "ties"):
        x = _logits(n + k, rows, n, DT[dtype], kind)
        vals, idx = x.sort(dim=1, descending=True, stable=True)
        vals, idx = vals[:, :k].contiguous(), idx[:, :k].to(torch.int32).contiguous()
        g = _gen(k)
        ks = torch.randint(0, k + 2, (rows,), generator=g, dtype=torch.int32)
        t = 0.5 + torch.rand(rows, generator=g)
        t[1::4] = 0.0
        top_p = 1.1 * torch.rand(rows, generator=g)
        for opts in (dict(), dict(ks=ks), dict(ks=ks, temperature=t), dict(top_p=top_p),
                     dict(ks=ks, temperature=t, top_p=top_p)):
            lists = torch.full((rows, k), 9.0, device="cuda")
            p = ts.ds_topk_softmax(vals, idx, n, out_dtype=DT[odt], out_list=lists,
                                   **{a: b.cuda() for a, b in opts.items()})
            want, wl = orc.list_softmax(_np(vals), _np(idx), n, **{a: _np(b) for a, b in opts.items()})
            label = f"lists {rows}x{n} k={k} {dtype}->{odt} {kind} {sorted(opts)}"
            assert np.array_equal(_np(lists) > 0, wl > 0), label  # the same prefix
            _close(lists, wl, label)
            _close(p, want, label, bf16=odt == "bf16")
        only = ts.ds_topk_softmax(vals, idx, n, rows_out=False)
        _close(only, orc.list_softmax(_np(vals), _np(idx), n)[1], "list only")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_list_softmax_many_long_rows(dtype):
    """Rows whose clearing takes longer than their list."""
    rows, n, k = 520, 66001, 40
    x = _logits(12, rows, 400, DT[dtype], "ties")
    vals, at = x.sort(dim=1, descending=True, stable=True)
    vals = vals[:, :k].contiguous()
    idx = (at[:, :k] * 165 + torch.arange(rows, device="cuda")[:, None] % 165).to(torch.int32).contiguous()
    g = _gen(4)
    ks = torch.randint(1, k + 1, (rows,), generator=g, dtype=torch.int32)
    t, top_p = 0.5 + torch.rand(rows, generator=g), torch.rand(rows, generator=g)
    t[::7] = 0.0
    idx[5, 3:] = -1
    lists = torch.empty(rows, k, device="cuda")
    p = ts.ds_topk_softmax(vals, idx, n, ks=ks.cuda(), temperature=t.cuda(), top_p=top_p.cuda(), out_dtype=DT[dtype],
                           out_list=lists)
    _, want = orc.list_softmax(_np(vals), _np(idx), n, _np(ks), _np(t), _np(top_p))
    _close(lists, want, "long rows")
    got = torch.gather(p.float(), 1, idx.clamp(min=0).long())
    _close(torch.where(idx < 0, 0, got), want, "long rows", bf16=dtype == "bf16")
    assert ((p != 0).sum(dim=1).cpu() == torch.from_numpy((want > 0).sum(axis=1))).all()


def test_list_softmax_padding_and_ragged_rows():
    """ds_topk_ex's padding (index -1, a NaN pattern as value) has no mass; an empty list gives zeros."""
    x = torch.randn(4, 1000, generator=_gen(1)).cuda()
    lens = torch.tensor([1000, 3, 0, 1], dtype=torch.int32, device="cuda")
    cfg = {"slices": 1}
    v, i = ts.ds_topk_ex(x, 20, cfg=cfg, lens=lens)
    p = ts.ds_topk_softmax(v, i, 1000, top_p=torch.full((4,), 0.9, device="cuda"))
    want, _ = orc.list_softmax(np.nan_to_num(_np(v)), _np(i), 1000, top_p=np.full(4, np.float64(np.float32(0.9))))
    _close(p, want, "padding")
    assert p[2].sum() == 0 and p[3].max() == 1


# ----------------------------------------------------------------------------- verification
def _verify_inputs(seed, batch, K, n, dtype, kind="probs"):
    g = _gen(seed)
    base = 2.5 * torch.randn(batch, K + 1, n, generator=g)
    target = torch.softmax(base, dim=2)
    draft = torch.softmax(base[:, :K] + 0.6 * torch.randn(batch, K, n, generator=g), dim=2)
    if kind == "sparse":  # rows that a top-k list left mostly at zero
        target = torch.where(target > target.topk(min(n, 4), dim=2)[0][..., -1:], target, 0)
        draft = torch.where(draft >= draft.topk(min(n, 3), dim=2)[0][..., -1:], draft, 0)
    tokens = torch.multinomial(draft.reshape(-1, n), 1, generator=g).view(batch, K).to(torch.int32) if K else \
        torch.empty(batch, 0, dtype=torch.int32)
    u, v = torch.rand(batch, K, generator=g), torch.rand(batch, generator=g)
    return target.to(dtype), draft.to(dtype), tokens, u, v


def _check_verify(target, draft, tokens, u, v, lens=None, label=""):
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    got, acc = ts.ds_verify(dev(target), dev(draft), dev(tokens), dev(u), dev(v), draft_lens=dev(lens))
    want, wacc = orc.verify(_np(target), None if draft is None else _np(draft), _np(tokens), _np(u), _np(v),
                            None if lens is None else _np(lens))
    assert np.array_equal(_np(acc), wacc), label
    assert np.array_equal(_np(got), want), f"{label}: {np.argwhere(_np(got) != want)[:4]}"
    return got, acc


@pytest.mark.parametrize("batch,K,n", [(1, 0, 1), (1, 1, 2), (3, 2, 17), (2, 3, 4096), (5, 1, 12289), (40, 4, 1000),
                                       (1, 64, 300), (3, 7, 32003), (300, 2, 257), (2, 2, 129280),
                                       (66, 1, 70001)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_verify_matches_definition(batch, K, n, dtype):
    for kind in ("probs", "sparse"):
        target, draft, tokens, u, v = _verify_inputs(batch + n, batch, K, n, DT[dtype], kind)
        lens = torch.randint(-1, K + 2, (batch,), generator=_gen(n), dtype=torch.int32)
        for q in (draft, None):
            for ln in (None, lens):
                _check_verify(target, q, tokens, u, v, ln, f"verify {batch}x{K}x{n} {dtype} {kind} {q is None} {ln is None}")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_verify_edges(dtype):
    n = 9001
    target, draft, tokens, u, v = _verify_inputs(77, 16, 3, n, DT[dtype])
    target[0] = 0                      # a target row without mass: no token
    draft[1] = target[1, :3]           # the same distributions: every draft accepted
    target[2, 0] = draft[2, 0]
    u[2, 0], tokens[2, 0] = 1.0, 5     # refused although the residual is empty: falls back to the target
    tokens[3, 1], tokens[4, 0] = -1, n  # tokens outside the vocabulary
    v[5], v[6] = 0.0, 1 - 2.0 ** -24   # the ends of the unit interval
    u[7] = 0.0
    target[8] = 0
    target[8, :, n - 1] = 1            # all mass on the last element
    target[9] = 0
    target[9, :, 0] = 1
    for q in (draft, None):
        got, _ = _check_verify(target, q, tokens, u, v, None, f"edges {dtype}")
        assert _np(got)[0, 0] == -1


def test_verify_samples_the_target_rows_when_nothing_is_drafted():
    """drafts = 0 is plain sampling: over many given numbers each token comes up as often as its
    share says (the counts are a function of the numbers: u = (i + 1/2) / N hits token t in
    its N p_t of them, one off at most at each end)."""
    n, N = 50, 4000
    p = torch.softmax(torch.randn(n, generator=_gen(5)), 0)
    target = p.repeat(N, 1).view(N, 1, n).cuda()
    u = ((torch.arange(N) + 0.5) / N).cuda()
    got, acc = ts.ds_verify(target, None, None, None, u)
    count = np.bincount(_np(got)[:, 0], minlength=n)
    assert np.abs(count - N * _np(p)).max() <= 2 and not _np(acc).any()


@pytest.mark.parametrize("batch", [64, 128, 129])
def test_verify_of_many_long_rows(batch):
    """Either side of the number of sequences that a workgroup each is enough for."""
    n, K = 33001, 1
    target, draft, tokens, u, v = _verify_inputs(batch, batch, K, n, torch.float32)
    _check_verify(target, draft, tokens, u, v, None, f"verify {batch}")


@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 7, 8, 9, 15, 17, 1023, 1024, 1025, 1027, 1031, 2047, 2048, 2049, 2055,
                               4097, 33001])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_verify_draws_each_place(n, dtype):
    """Equal masses, and numbers that aim at the middle of an element's share: (i + 1/2) of n shares
    is half a share (2^-17 of all, at the least) from the next element, the number is rounded by 2^-25
    and the sums by n 2^-53 of all. With a
    refused certain draft t the same over the other elements."""
    near = sorted({i for c in (0, 1024, 2048, n // 2, n) for i in range(c - 18, c + 18) if 0 <= i < n})
    at = torch.tensor(near)
    B = len(near)
    target = torch.full((1, 1, n), 2.0 ** -10, dtype=DT[dtype]).expand(B, 1, n)
    v = ((at.double() + 0.5) / n).float()
    got, acc = ts.ds_verify(target.contiguous().cuda(), None, None, None, v.cuda())
    assert _np(got)[:, 0].tolist() == near and not _np(acc).any()
    if n == 1:
        return
    for t in (0, n // 2, n - 1):
        others = at[at < n - 1]
        target = torch.full((1, 1, 1), 2.0 ** -10, dtype=DT[dtype]).expand(len(others), 2, n).contiguous()
        tokens = torch.full((len(others), 1), t, dtype=torch.int32)
        v = ((others.double() + 0.5) / (n - 1)).float()
        got, acc = ts.ds_verify(target.cuda(), None, tokens.cuda(), torch.ones(len(others), 1).cuda(), v.cuda())
        assert _np(got)[:, 0].tolist() == [i + (i >= t) for i in others.tolist()] and not _np(acc).any()


def test_verify_strided_inputs():
    target, draft, tokens, u, v = _verify_inputs(9, 4, 3, 1001, torch.float32)
    wide = torch.zeros(4, 4, 1103)
    wide[:, :, 5:1006] = target
    wq = torch.zeros(4, 3, 1050)
    wq[:, :, 1:1002] = draft
    got, acc = ts.ds_verify(wide.cuda()[:, :, 5:1006], wq.cuda()[:, :, 1:1002], tokens.cuda(), u.cuda(), v.cuda())
    want, wacc = orc.verify(_np(target), _np(draft), _np(tokens), _np(u), _np(v))
    assert np.array_equal(_np(got), want) and np.array_equal(_np(acc), wacc)
    with pytest.raises(ValueError):  # sequences that do not lie evenly apart
        ts.ds_verify(wide.cuda()[:, :3, 5:1006], wq.cuda()[:, :2], tokens[:, :2].contiguous().cuda(),
                     u[:, :2].contiguous().cuda(), v.cuda())


# ----------------------------------------------------------------------------- together
def test_sampler_run():
    """Logits -> ds_topk -> ds_topk_softmax for the target and ds_softmax for the draft ->
    ds_verify, as a sampler runs them; each step against the definition on the step's inputs."""
    B, K, n, k = 6, 3, 20000, 200
    g = _gen(44)
    base = 2 * torch.randn(B * (K + 1), n, generator=g)
    x = base.cuda()
    xq = (base + 0.3 * torch.randn(B * (K + 1), n, generator=g))[:B * K].contiguous().cuda()
    t = 0.5 + 0.5 * torch.rand(B * (K + 1), generator=g)
    t[3] = 0.0
    vals, idx = ts.ds_topk(x, k, seed=3)
    top_p = torch.full((B * (K + 1),), 0.95)
    p = ts.ds_topk_softmax(vals, idx, n, temperature=t.cuda(), top_p=top_p.cuda())
    q = ts.ds_softmax(xq, temperature=t[:B * K].cuda())
    want, _ = orc.list_softmax(_np(vals), _np(idx), n, temperature=_np(t), top_p=_np(top_p))
    _close(p, want, "target")
    _close(q, orc.softmax(_np(xq), _np(t[:B * K])), "draft")
    tokens = q.argmax(dim=1).to(torch.int32).view(B, K)
    u, v = torch.rand(B, K, generator=g), torch.rand(B, generator=g)
    got, acc = ts.ds_verify(p.view(B, K + 1, n), q.view(B, K, n), tokens, u.cuda(), v.cuda())
    want, wacc = orc.verify(_np(p).reshape(B, K + 1, n), _np(q).reshape(B, K, n), _np(tokens), _np(u), _np(v))
    assert np.array_equal(_np(got), want) and np.array_equal(_np(acc), wacc)
    # every drawn token has mass in its row
    a = _np(acc)
    assert (_np(p).reshape(B, K + 1, n)[np.arange(B), a, want[np.arange(B), a]] > 0).all()


def test_training_step_of_a_router():
    """Forward with counts, a bias moved against the load, forward again, gradient."""
    x = _logits(91, 500, 64, torch.float32)
    bias = torch.zeros(64, device="cuda")
    kw = dict(score=ts.SCORE_SIGMOID, renormalize=True, scale=2.0)
    for _ in range(2):
        counts = torch.zeros(64, dtype=torch.int32, device="cuda")
        w, i = ts.ds_route(x, 6, bias=bias, groups=8, topk_groups=4, group_top=2, counts=counts, **kw)
        ww, wi = orc.route(_np(x), 6, _np(bias), "sigmoid", 8, 4, 2, True, 2.0)
        assert np.array_equal(_np(i), wi)
        _close(w, ww, "forward")
        assert int(counts.sum()) == 3000
        bias -= 0.01 * torch.sign(counts - counts.float().mean())
    g = torch.randn(500, 6, generator=_gen(3)).cuda()
    dx = ts.ds_route_grad(x, i, g, **kw)
    want, size = orc.route_grad(_np(x), _np(i), _np(g), "sigmoid", True, 2.0)
    _close(dx, want, "gradient", size=4 * size)


def _everything(d):
    w, i = ts.ds_route(d["x"], 6, bias=d["bias"], score=ts.SCORE_SIGMOID, groups=8, topk_groups=4, group_top=2,
                       renormalize=True)
    dx = ts.ds_route_grad(d["x"], i, d["g"], score=ts.SCORE_SIGMOID, renormalize=True)
    p = ts.ds_softmax(d["logits"], temperature=d["t"])
    l = ts.ds_topk_softmax(d["vals"], d["idx"], 30011, top_p=d["top_p"])
    tok, acc = ts.ds_verify(p.view(2, 3, 30011), l.view(3, 2, 30011)[:2], d["tokens"], d["u"], d["v"])
    return w, i, dx, p, l, tok, acc


def _operands(seed):
    g = _gen(seed)
    x = torch.randn(200, 64, generator=g)
    logits = 3 * torch.randn(6, 30011, generator=g)
    v, i = logits.sort(dim=1, descending=True)
    d = dict(x=x, bias=0.1 * torch.randn(64, generator=g), g=torch.randn(200, 6, generator=g), logits=logits,
             t=0.5 + torch.rand(6, generator=g), vals=v[:, :99].contiguous(), idx=i[:, :99].to(torch.int32).contiguous(),
             top_p=torch.rand(6, generator=g), tokens=torch.randint(0, 30011, (2, 2), generator=g, dtype=torch.int32),
             u=torch.rand(2, 2, generator=g) * 1e-3, v=torch.rand(2, generator=g))
    return {k: t.cuda() for k, t in d.items()}


def test_graph_replays_with_other_work_between():
    d = _operands(1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _everything(d)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = _everything(d)
    for seed in (2, 3, 4):
        new = _operands(seed)
        for k in d:
            d[k].copy_(new[k])
        want = [t.clone() for t in _everything(new)]
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)
        _everything(_operands(seed + 10))


def test_streams_and_repeats_give_the_same_bits():
    """Two streams at once, each with its own operands, and an explicit stream argument."""
    d1, d2 = _operands(5), _operands(6)
    w1, w2 = _everything(d1), _everything(d2)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got1, got2 = [], []
    for _ in range(5):
        with torch.cuda.stream(s1):
            got1.append(_everything(d1))
        with torch.cuda.stream(s2):
            got2.append(_everything(d2))
    p = ts.ds_softmax(d1["logits"], temperature=d1["t"], stream=s1)
    dx = ts.ds_route_grad(d1["x"], w1[1], d1["g"], score=ts.SCORE_SIGMOID, renormalize=True, stream=s2)
    w, _ = ts.ds_route(d1["x"], 6, bias=d1["bias"], score=ts.SCORE_SIGMOID, groups=8, topk_groups=4, group_top=2,
                       renormalize=True, stream=s1)
    l = ts.ds_topk_softmax(d1["vals"], d1["idx"], 30011, top_p=d1["top_p"], stream=s2)
    t, _ = ts.ds_verify(w1[3].view(2, 3, 30011), None, d1["tokens"], d1["u"], d1["v"], stream=s2)
    torch.cuda.synchronize()
    t2, _ = ts.ds_verify(w1[3].view(2, 3, 30011), None, d1["tokens"], d1["u"], d1["v"])
    assert torch.equal(p, w1[3]) and torch.equal(t, t2)
    assert torch.equal(w, w1[0]) and torch.equal(dx, w1[2]) and torch.equal(l, w1[4])
    for got, want in ((got1, w1), (got2, w2)):
        for outs in got:
            for a, b in zip(outs, want):
                assert torch.equal(a, b)


def test_offsets_past_32_bits():
    """Rows whose elements lie more than 2^32 apart."""
    n, stride = 5000, (1 << 31) + 8
    buf = torch.empty(2 * stride + n, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(buf, (3, n), (stride, 1))
    x.copy_(_logits(8, 3, n, torch.bfloat16))
    say(f"[gpu] rows {stride * 2} bytes apart")
    _close(ts.ds_softmax(x), orc.softmax(_np(x)), "far rows")
    r = x[:, :64]
    w, i = ts.ds_route(r, 5)
    ww, wi = orc.route(_np(r), 5)
    assert np.array_equal(_np(i), wi)
    _close(w, ww, "far route")
    target = torch.as_strided(buf, (1, 3, n), (3 * stride, stride, 1))
    target.copy_(torch.softmax(target.float(), 2))
    tok = torch.tensor([[1, 2]], dtype=torch.int32, device="cuda")
    u = torch.tensor([[0.0, 0.0]], device="cuda")
    v = torch.tensor([0.7], device="cuda")
    got, acc = ts.ds_verify(target, None, tok, u, v)
    want, wacc = orc.verify(_np(target), None, _np(tok), _np(u), _np(v))
    assert np.array_equal(_np(got), want) and np.array_equal(_np(acc), wacc)
