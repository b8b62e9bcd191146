"""Plain 64-bit definitions of the row operators beside top-k (tests only; no code shared with
the kernels): routing to experts and its gradient, softmax of rows and of top-k lists, and the
verification of drafted tokens. Inputs are float64 copies of what the kernels are given."""
from __future__ import annotations

import numpy as np

NEG = -np.inf


def scores(x: np.ndarray, score: str) -> np.ndarray:
    """Scores of one row of logits; an expert at -inf scores 0, +inf is the limit."""
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "sigmoid":
            return np.where(x >= 0, 1 / (1 + np.exp(-np.abs(x))), np.exp(-np.abs(x)) / (1 + np.exp(-np.abs(x))))
        m = x.max()
        if m == NEG:
            return np.zeros_like(x)
        e = np.where(x == m, 1.0, np.exp(np.where(x == m, 0.0, x - m)))
        return e / e.sum()


def _best(c: np.ndarray, k: int) -> list:
    """Positions of the k largest entries above -inf, larger first, then smaller position."""
    order = sorted((i for i in range(len(c)) if c[i] > NEG), key=lambda i: (-c[i], i))
    return order[:k]


def route(x, k, bias=None, score="softmax", groups=1, topk_groups=0, group_top=1, renormalize=False, scale=1.0):
    rows, n = x.shape
    w = np.zeros((rows, k))
    idx = np.full((rows, k), -1, np.int32)
    topk_groups = topk_groups or groups
    size = n // groups
    for r in range(rows):
        s = scores(x[r], score)
        c = x[r].copy() if bias is None else np.where(x[r] == NEG, NEG, s + bias)
        if topk_groups < groups:
            add = np.where(c == NEG, NEG, s) if bias is None and group_top > 1 else c
            per = []
            for g in range(groups):
                top = [add[g * size + i] for i in _best(add[g * size:(g + 1) * size], group_top)]
                per.append(sum(top) if top else NEG)
            chosen = sorted(range(groups), key=lambda g: (-per[g], g))[:topk_groups]
            for g in range(groups):
                if g not in chosen:
                    c[g * size:(g + 1) * size] = NEG
        at = _best(c, k)
        idx[r, :len(at)] = at
        total = s[at].sum() if renormalize else 1.0
        if total > 0:
            w[r, :len(at)] = scale * s[at] / total
    return w, idx


def route_weights(x, idx, score, renormalize, scale):
    """The weights of a fixed choice idx (for differences)."""
    w = np.zeros(idx.shape)
    for r in range(len(x)):
        s = scores(x[r], score)
        live = (idx[r] >= 0) & (idx[r] < x.shape[1])
        v = np.where(live, s[np.where(live, idx[r], 0)], 0.0)
        total = v.sum() if renormalize else 1.0
        if total > 0:
            w[r] = scale * v / total
    return w


def route_grad(x, idx, g, score, renormalize, scale):
    """(dx, the size each element's terms have before they cancel)."""
    dx, size = np.zeros_like(x), np.zeros_like(x)
    for r in range(len(x)):
        s = scores(x[r], score)
        h, hits = np.zeros(x.shape[1]), np.zeros(x.shape[1])
        for j in range(idx.shape[1]):
            if 0 <= idx[r, j] < x.shape[1]:
                h[idx[r, j]] += scale * g[r, j]
                hits[idx[r, j]] += 1
        ds, mag = h, np.abs(h)
        if renormalize:
            S = (hits * s).sum()
            ds = (h - hits * (h * s).sum() / S) / S if S > 0 else np.zeros_like(h)
            mag = (np.abs(h) + hits * (np.abs(h) * s).sum() / S) / S if S > 0 else np.zeros_like(h)
        if score == "sigmoid":
            dx[r], size[r] = ds * s * (1 - s), mag * s
        elif renormalize:
            dx[r], size[r] = ds * s, mag * s
        else:
            dx[r], size[r] = s * (ds - (ds * s).sum()), s * (mag + (mag * s).sum())
    return dx, size


def softmax(x, temperature=None):
    out = np.zeros_like(x)
    for r in range(len(x)):
        m = x[r].max()
        if m == NEG:
            continue
        if temperature is not None and not temperature[r] > 0:
            out[r, int(np.argmax(x[r]))] = 1
            continue
        t = 1.0 if temperature is None else temperature[r]
        with np.errstate(over="ignore", invalid="ignore"):
            e = np.where(x[r] == m, 1.0, np.exp(np.where(x[r] == m, 0.0, x[r] - m) / t))
        out[r] = e / e.sum()
    return out


def list_softmax(vals, idx, n, ks=None, temperature=None, top_p=None):
    """(whole rows [rows, n], lists [rows, k])."""
    rows, k = vals.shape
    out, lists = np.zeros((rows, n)), np.zeros((rows, k))
    for r in range(rows):
        used = k if ks is None else min(max(int(ks[r]), 1), k)
        at = [i for i in range(used) if 0 <= idx[r, i] < n]
        if not at or vals[r, at[0]] == NEG:
            continue
        t = 1.0 if temperature is None else temperature[r]
        if not t > 0:
            at = at[:1]
            e = np.ones(1)
        else:
            v = vals[r, at]
            with np.errstate(over="ignore", invalid="ignore"):
                e = np.where(v == v[0], 1.0, np.exp(np.where(v == v[0], 0.0, v - v[0]) / t))
        if top_p is not None:
            before = np.concatenate([[0.0], np.cumsum(e)[:-1]])
            keep = before < top_p[r] * e.sum()
            keep[0] = True
            e = e * keep
        lists[r, at] = e / e.sum()
        out[r, idx[r, at]] = lists[r, at]
    return out, lists


def verify(target, draft, tokens, accept_u, sample_u, lens=None):
    batch, m, n = target.shape
    K = m - 1
    out, got = np.full((batch, m), -1, np.int32), np.zeros(batch, np.int32)
    for b in range(batch):
        length = K if lens is None else min(max(int(lens[b]), 0), K)
        j = 0
        while j < length:
            t = int(tokens[b, j])
            if not 0 <= t < n:
                break
            q = 1.0 if draft is None else draft[b, j, t]
            if not accept_u[b, j] * q < target[b, j, t]:
                break
            out[b, j] = t
            j += 1
        got[b] = j
        p = target[b, j]
        mass = p.copy()
        if j < length:
            if draft is None:
                if 0 <= int(tokens[b, j]) < n:
                    mass[int(tokens[b, j])] = 0.0
            else:
                mass = np.maximum(p - draft[b, j], 0.0)
        if not mass.sum() > 0:
            mass = p
        total = mass.sum()
        if total > 0:
            at = int(np.searchsorted(np.cumsum(mass), sample_u[b] * total, side="right"))
            out[b, j] = min(at, int(np.nonzero(mass > 0)[0][-1]))
    return out, got
