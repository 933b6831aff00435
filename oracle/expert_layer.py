"""fp64 oracle of the expert layer's operators and of the 8-bit products
(include/expert_layer.h, include/int8_gemm.h): plain numpy, written from the
definitions, choice by choice and row by row, sharing no code with the CUDA
path.  Every function that returns a computed sum also returns (or has beside
it) the sum of the absolute values of its terms, the scale of its rounding
bounds.  Test infrastructure only.
"""
from __future__ import annotations

import numpy as np

TINY = 2.0 ** -100


def sort(ids, E):
    """(offsets, slots, positions) of the stable sort by expert; ids outside
    0 .. E-1 go last."""
    flat = [int(e) for e in np.asarray(ids).reshape(-1)]
    lists = [[] for _ in range(E + 1)]
    for s, e in enumerate(flat):
        lists[e if 0 <= e < E else E].append(s)
    offsets = np.zeros(E + 1, np.int32)
    for e in range(E):
        offsets[e + 1] = offsets[e] + len(lists[e])
    slots = np.array([s for one in lists for s in one], np.int32)
    positions = np.empty(len(flat), np.int32)
    positions[slots] = np.arange(len(flat), dtype=np.int32)
    return offsets, slots, positions


def dispatch(x, positions, total, k):
    T, H = x.shape
    rows = np.zeros((T * k, H))
    for t in range(T):
        for j in range(k):
            p = positions[t * k + j]
            if p < total:
                rows[p] = x[t]
    return rows


def combine(rows, positions, total, weights, T, k):
    """(out, sum of magnitudes); weights None: 1."""
    H = rows.shape[1]
    out, mag = np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        for j in range(k):
            p = positions[t * k + j]
            if p < total:
                w = 1.0 if weights is None else float(weights[t, j])
                out[t] += w * rows[p]
                mag[t] += np.abs(w * rows[p])
    return out, mag


def dispatch_grad(drows, positions, total, T, k):
    return combine(drows, positions, total, None, T, k)


def combine_grad(dout, rows, positions, total, weights, k):
    """(drows, dw, sum of dw's magnitudes)."""
    T, H = dout.shape
    drows = np.zeros((T * k, H))
    dw, mag = np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            p = positions[t * k + j]
            if p < total:
                w = 1.0 if weights is None else float(weights[t, j])
                drows[p] = w * dout[t]
                dw[t, j] = np.sum(rows[p] * dout[t])
                mag[t, j] = np.sum(np.abs(rows[p] * dout[t]))
    return drows, dw, mag


def gated(x):
    """silu(gate) * value of rows that hold K gates and then K values."""
    K = x.shape[1] // 2
    with np.errstate(over="ignore", invalid="ignore"):
        g, u = x[:, :K], x[:, K:]
        return g / (1.0 + np.exp(-g)) * u


def quantize(x):
    """(x * 127 / max|x| before rounding, scale); the code is its nearest
    integer.  Rows below 2^-100 are zero, rows with an infinity or NaN have
    scale NaN and codes 0."""
    M, K = x.shape
    y, scale = np.zeros((M, K)), np.zeros(M)
    for r in range(M):
        if K == 0:
            continue
        if not np.all(np.isfinite(x[r])):
            scale[r] = np.nan
            continue
        a = np.max(np.abs(x[r]))
        if a >= TINY:
            y[r] = x[r] * 127.0 / a
            scale[r] = a / 127.0
    return y, scale


def product(a, sa, b, sb):
    """(C, its magnitude sum |a||b| sa sb, the unscaled sum |a||b|)."""
    a, b = a.astype(np.float64), b.astype(np.float64)
    s = np.asarray(sa, np.float64)[:, None] * np.asarray(sb, np.float64)[None, :]
    raw = np.abs(a) @ np.abs(b).T
    return (a @ b.T) * s, raw * np.abs(s), raw


def product_experts(offsets, a, sa, b, sb, N):
    """C of all rows (rows from offsets[-1] on: zero), as product()."""
    M = a.shape[0]
    out = [np.zeros((M, N)) for _ in range(3)]
    for e in range(len(offsets) - 1):
        lo, hi = offsets[e], offsets[e + 1]
        if hi > lo:
            for o, v in zip(out, product(a[lo:hi], sa[lo:hi], b[e], sb[e])):
                o[lo:hi] = v
    return out
