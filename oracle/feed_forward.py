"""Oracle of the norm, of the 4-bit format and of the few-token expert layer
(include/rms_norm.h, include/fp4_gemm.h, include/expert_layer.h): plain numpy,
written from the definitions, sharing no code with the CUDA path.  Sums are
fp64; what the definition does in fp32 (codes and scales of a row) is done in
fp32, operation by operation, so that codes can be compared exactly.  Test
infrastructure only.
"""
from __future__ import annotations

import numpy as np

TINY = np.float32(2.0 ** -100)
LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BLOCK = {"mx": 32, "nv": 16}
F32 = np.float32


# ---------------------------------------------------------------------- norm

def rms_norm(s, weight, eps):
    """(y, rho) of rows s (fp64) in fp64."""
    rho = 1.0 / np.sqrt((s * s).mean(axis=1) + float(F32(eps)))
    return s * rho[:, None] * weight, rho


def rms_norm_grad(s, weight, dy, dsum, eps):
    """(dx, dweight) and the magnitudes of their rounding bounds."""
    H = s.shape[1]
    _, rho = rms_norm(s, weight, eps)
    r = rho[:, None]
    g = weight * dy
    m = (g * s).sum(axis=1, keepdims=True) / H
    dx = dsum + r * (g - s * r * r * m)
    mag = np.abs(dsum) + np.abs(r * g) + \
        np.abs(s) * r ** 3 * (np.abs(g * s).sum(axis=1, keepdims=True) / H)
    return dx, (dy * s * r).sum(axis=0), mag, np.abs(dy * s * r).sum(axis=0)


def quantize8(v):
    """(codes, scales) of fp32 rows, in fp32 as the definition says."""
    a = np.abs(v).max(axis=1, initial=0).astype(F32)
    ok = np.isfinite(v).all(axis=1)
    on = ok & (a >= TINY)
    safe = np.where(on, a, F32(1))
    q = np.rint(np.where(on[:, None], v, F32(0)) * (F32(127) / safe)[:, None]).astype(np.int64)
    return q, np.where(ok, np.where(on, a / F32(127), F32(0)), F32(np.nan)).astype(F32)


# ------------------------------------------------------------- 4-bit format

def round_e4m3(x):
    """The nearest e4m3 value of x >= 0 (ties to even, at most 448)."""
    x = np.asarray(x, np.float64)
    e = np.floor(np.log2(np.where(x > 0, x, 1.0)))
    step = np.exp2(np.maximum(e, -6.0) - 3.0)
    return np.minimum(np.rint(x / step) * step, 448.0)


def e4m3_byte(v):
    """The byte of an e4m3 value >= 0."""
    v = np.asarray(v, np.float64)
    e = np.floor(np.log2(np.where(v > 0, v, 1.0)))
    sub = v < 2.0 ** -6
    byte = np.where(sub, v * 512, (e + 7) * 8 + (v / np.exp2(e) - 1) * 8)
    return byte.astype(np.uint8)


def e4m3_value(b):
    b = np.asarray(b, np.int64)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m / 512.0, np.exp2(e - 7.0) * (1 + m / 8.0))
    return np.where((b & 127) == 127, np.nan, v)


def scale_value(b, format_):
    if format_ == "nv":
        return e4m3_value(b)
    return np.where(np.asarray(b) == 255, np.nan, np.exp2(np.asarray(b, np.float64) - 127))


def round_code(u):
    """Codes (0 .. 15) of the nearest 4-bit values, ties to the even code."""
    a = np.abs(u).astype(np.float64)
    border = (LEVELS[1:] + LEVELS[:-1]) / 2
    lo = np.searchsorted(border, a, side="left")   # a border itself goes down
    hi = np.searchsorted(border, a, side="right")  # and up
    return np.where(lo % 2 == 0, lo, hi) + 8 * np.signbit(u)


def code_value(c):
    c = np.asarray(c, np.int64)
    return LEVELS[c & 7] * np.where(c & 8, -1.0, 1.0)


def quantize4(v, format_):
    """(codes (M, K), block scale bytes (M, blocks), row scales) of fp32 rows."""
    v = np.asarray(v, F32)
    M, K = v.shape
    n = BLOCK[format_]
    blocks = -(-K // n)
    pad = np.zeros((M, blocks * n), F32)
    pad[:, :K] = v
    ok = np.isfinite(v).all(axis=1)
    pad = np.where(ok[:, None], pad, F32(0))
    b = pad.reshape(M, blocks, n)
    top = np.abs(b).max(axis=2, initial=0)
    if format_ == "mx":
        _, e = np.frexp(np.where(top > 0, top, F32(1)).astype(np.float64))
        e = np.where(top > 0, e - 3, -127)  # floor(log2) - 2
        byte = np.maximum(e + 127, 0)
        u = np.ldexp(b.astype(np.float64), (127 - byte)[:, :, None])
        row = np.ones(M, F32)
    else:
        a = np.abs(pad).max(axis=1, initial=0)
        on = a >= TINY
        safe = np.where(on, a, F32(1))
        s = round_e4m3((top * np.where(on, F32(448) / safe, F32(0))[:, None]).astype(F32))
        byte = e4m3_byte(s)
        up = np.where(on, F32(2688) / safe, F32(0))[:, None] / np.where(s > 0, s, 1).astype(F32)
        up = np.where(s > 0, up, F32(0)).astype(F32)
        u = (b * up[:, :, None]).astype(F32)
        row = np.where(on, a / F32(2688), F32(0)).astype(F32)
    codes = round_code(u).reshape(M, -1)[:, :K].astype(np.uint8)
    codes[~ok] = 0
    byte = np.where(ok[:, None], byte, 0).astype(np.uint8)
    return codes, byte, np.where(ok, row, F32(np.nan)).astype(F32)


def values4(codes, byte, format_):
    """What codes and block scales stand for (without the row scale), fp64."""
    s = np.repeat(scale_value(byte, format_), BLOCK[format_], axis=1)[:, :codes.shape[1]]
    return code_value(codes) * s


def scale_offset(r, j, blocks):
    """Byte of row r's block j, from the layout's definition."""
    return ((r // 128) * (-(-blocks // 4)) + j // 4) * 512 + (r % 32) * 16 + \
        (r % 128) // 32 * 4 + j % 4


def pack_codes(codes, ld):
    M, K = codes.shape
    full = np.zeros((M, ld), np.uint8)
    full[:, :K] = codes
    return full[:, 0::2] | (full[:, 1::2] << 4)


def unpack_codes(packed, K):
    both = np.stack([packed & 15, packed >> 4], axis=2).reshape(packed.shape[0], -1)
    return both[:, :K]


def pack_scales(byte, fill=0):
    """The tiled layout; bytes of rows past the last are `fill`."""
    M, blocks = byte.shape
    out = np.full((-(-M // 128)) * (-(-blocks // 4)) * 512, fill, np.uint8)
    r, j = np.meshgrid(np.arange(M), np.arange(-(-blocks // 4) * 4), indexing="ij")
    full = np.zeros(r.shape, np.uint8)
    full[:, :blocks] = byte
    out[scale_offset(r, j, blocks)] = full
    return out


def unpack_scales(tiled, M, blocks):
    r, j = np.meshgrid(np.arange(M), np.arange(blocks), indexing="ij")
    return tiled[scale_offset(r, j, blocks)]


def product4(a, sa, b, sb):
    """(C, sum of magnitudes) from values without row scales and row scales."""
    scale = sa.astype(np.float64)[:, None] * sb.astype(np.float64)[None, :]
    return (a @ b.T) * scale, (np.abs(a) @ np.abs(b).T) * np.abs(scale)


# ------------------------------------------------------- few-token expert layer

def experts_layer(x, ids, weights, W1, s1, W2, s2, u, least=2.0 ** -24):
    """(out, error bound without out's own rounding) of the layer; u: half a
    unit in the last place of the row type, in which h is kept as a rounded value
    and the rounded rest; e: of a fp32 operation; least: what h may be off by however
    small it is."""
    T, k = ids.shape
    E, F2, H = W1.shape
    F = F2 // 2
    e24 = 2.0 ** -24
    out, err = np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            if not 0 <= e < E:
                continue
            w1 = W1[e] if s1 is None else W1[e] * s1[e][:, None]
            w2 = W2[e] if s2 is None else W2[e] * s2[e][:, None]
            gu, mag = w1 @ x[t], np.abs(w1) @ np.abs(x[t])
            g, up = gu[:F], gu[F:]
            gm, um = mag[:F], mag[F:]
            silu = g / (1 + np.exp(-g))
            h = silu * up
            # |silu'| <= 1.1; fp32 sums of H terms, a few operations for silu
            dh = u * u * np.abs(h) + e24 * ((H + 16) * (1.1 * gm * np.abs(up) + np.abs(silu) * um) +
                                        8 * np.abs(h)) + least
            wt = 1.0 if weights is None else float(weights[t, j])
            out[t] += wt * (w2 @ h)
            err[t] += abs(wt) * (np.abs(w2) @ (dh + e24 * (F + k + 16) * np.abs(h)))
    return out, err
