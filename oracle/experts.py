"""The definitions of the operators behind a router in 64 bits (numpy); test infrastructure only.

Bad positions and slots of a plan are taken as the header says: skipped.
"""
import numpy as np

LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}
LEAST = 2.0 ** -100


def sort(idx, experts, align, capacity):
    """place [rows, k], order [capacity], offsets [experts + 1]."""
    flat = idx.reshape(-1)
    place, order = np.full(flat.size, -1, np.int32), np.full(capacity, -1, np.int32)
    offsets = np.zeros(experts + 1, np.int32)
    for e in range(experts):
        mine = np.flatnonzero(flat == e)
        at = offsets[e] + np.arange(mine.size)
        place[mine], order[at] = at, mine
        offsets[e + 1] = offsets[e] + -(-mine.size // align) * align
    return place.reshape(idx.shape), order, offsets


def gather(x, place, offsets, out):
    """x's rows at their slots' positions in out [capacity, n] (rows from the end on as they are)."""
    out = out.copy()
    out[:offsets[-1]] = 0
    rows, slots = np.nonzero(place >= 0)
    out[place[rows, slots]] = x[rows]
    return out


def combine(y, place, weights):
    """(the sums, the sums of the terms' magnitudes)"""
    out, size = np.zeros((place.shape[0], y.shape[1])), np.zeros((place.shape[0], y.shape[1]))
    for j in range(place.shape[1]):
        has = place[:, j] >= 0
        term = y[place[has, j]] * (1.0 if weights is None else weights[has, j, None])
        out[has] += term
        size[has] += np.abs(term)
    return out, size


def combine_grad(g, y, place, weights, offsets, out_y):
    """grad_y, grad_weights, and the sums of the magnitudes that grad_weights is made of."""
    out_y = out_y.copy()
    out_y[:offsets[-1]] = 0
    rows, slots = np.nonzero(place >= 0)
    at = place[rows, slots]
    out_y[at] = g[rows] * (1.0 if weights is None else weights[rows, slots, None])
    out_w, size = np.zeros(place.shape), np.zeros(place.shape)
    out_w[rows, slots] = (g[rows] * y[at]).sum(axis=1)
    size[rows, slots] = np.abs(g[rows] * y[at]).sum(axis=1)
    return out_y, out_w, size


def round8(v, to):
    """The 8-bit float nearest to v (float64, up to the largest), ties to even."""
    bits, least = (3, -6) if to == "e4m3" else (2, -14)
    exponent = np.maximum(np.frexp(np.abs(v))[1] - 1, least)
    step = np.ldexp(1.0, exponent - bits)
    return np.rint(v / step) * step


def quantize(x, rows, to):
    """x [r, n] float32 in blocks of rows x 128: (values [r, n], scales). Blocks that are not finite have
    scale NaN and values 0."""
    r, n = x.shape
    q, scales = np.zeros((r, n)), np.zeros((-(-r // rows), -(-n // 128)), np.float32)
    for i in range(scales.shape[0]):
        for j in range(scales.shape[1]):
            at = (slice(i * rows, (i + 1) * rows), slice(j * 128, (j + 1) * 128))
            part = x[at]
            if not np.isfinite(part).all():
                scales[i, j] = np.nan
                continue
            most = np.float32(max(float(np.abs(part).max()), LEAST))
            scales[i, j] = most / np.float32(LARGEST[to])
            q[at] = round8(part.astype(np.float64) / np.float64(scales[i, j]), to)
    return q, scales


def values(q, scales, rows):
    """What 8-bit values and scales stand for."""
    full = np.repeat(np.repeat(scales.astype(np.float64), rows, axis=0)[:q.shape[0]], 128, axis=1)[:, :q.shape[1]]
    return q * full


def product(a, b):
    """a b^T, and the same of the magnitudes."""
    return a @ b.T, np.abs(a) @ np.abs(b).T
