"""The gated activation that the 4-bit quantiser makes (include/fp4_gemm.h) at
gates whose exponential is very small, against the definition in 64 bits.

silu(x) = x / (1 + exp(-x)) is small there, and a large up value makes its product
the largest of a block or row.  Bound of an element: 8 units of 2^-23 of it for silu
and its product, and 2^-141 of the up value where exp(x) is subnormal in fp32 (off by
2^-148 at most, times |x| <= 104).  What a scale or code adds: a row scale one
rounding, a block scale half its step, a code half the distance of its neighbours
and four fp32 operations."""
import numpy as np
import pytest

from oracle import feed_forward as ff
from test_gpu_fp4 import FORMATS, gpu_ready, quantize, rows  # noqa: F401

pytestmark = pytest.mark.gpu
E23 = 2.0 ** -23
# gates of a row; from -87.3 to -88.7 the divisor 1 + exp(-x) is beyond 2^126, below
# that exp(-x) is no fp32 number
BANDS = [(-35, -25), (-60, -50), (-87.2, -80), (-88.7, -87.4), (-91, -88.8), (-103, -92), (-1, 1)]


def values(K, type_, rng):
    largest = 60000.0 if type_ == "fp16" else 2.0 ** 126
    v = np.empty((2 * len(BANDS), 2 * K))
    for r, (lo, hi) in enumerate(BANDS):
        up = largest * (0.25 + 0.75 * rng.random(K)) * rng.choice([-1, 1], K)
        if lo == -1:
            up = rng.standard_normal(K)
        v[r] = np.concatenate([rng.uniform(lo, hi, K), up])
        # ordinary gates and small up values, but for one product in a few blocks
        few = rng.random(K) < 1 / 40
        few[K // 2] = True
        mixed = np.concatenate([rng.standard_normal(K), rng.standard_normal(K) * 1e-4])
        v[len(BANDS) + r] = np.where(np.concatenate([few, few]), v[r], mixed)
    return v


@pytest.mark.parametrize("format_", FORMATS)
@pytest.mark.parametrize("type_", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("K,pad,offset", [(64, 0, 0), (201, 0, 1), (8200, 8, 0)])
def test_very_negative_gates(type_, format_, K, pad, offset):
    rng = np.random.default_rng(K)
    x = rows(2 * len(BANDS), 2 * K, type_, pad, offset, values(K, type_, rng))
    q, _, sf, sc = quantize(x, K, format_, "swiglu")
    xv = x.np()
    g, u = xv[:, :K], xv[:, K:]
    t = np.exp(-np.abs(g))
    want = np.where(g < 0, g * t, g) / (1 + t) * u
    err = 8 * E23 * np.abs(want) + 2.0 ** -141 * np.abs(u)
    n, blocks = ff.BLOCK[format_], -(-K // ff.BLOCK[format_])

    def by_block(a):
        full = np.zeros((a.shape[0], blocks * n))
        full[:, :K] = a
        return full.reshape(a.shape[0], blocks, n).max(2)

    top, off_top = np.abs(want).max(1), err.max(1)
    block, off_block = by_block(np.abs(want)), by_block(err)
    codes = ff.unpack_codes(q.cpu().numpy(), K)
    s = ff.scale_value(ff.unpack_scales(sf.cpu().numpy(), x.R, blocks), format_)
    row = sc.double().cpu().numpy()
    if format_ == "nv":
        # (fp16's largest up values leave some rows below the least one that counts)
        tiny = top + off_top < 2.0 ** -100
        assert np.all(tiny | (top - off_top > 2.0 ** -100))
        assert not row[tiny].any() and not s[tiny].any() and not ff.code_value(codes)[tiny].any()
        top, off_top = np.where(tiny, np.inf, top), np.where(tiny, 0, off_top)
        want, block = np.where(tiny[:, None], 0, want), np.where(tiny[:, None], 0, block)
        assert np.all((np.abs(row - top / 2688) <= off_top / 2688 + E23 * top)[~tiny])
        ideal = block * 448 / top[:, None]
        step = np.exp2(np.floor(np.log2(np.maximum(ideal, 2.0 ** -6))) - 3)
        slack = 448 / top[:, None] * (off_block + block * (off_top / top)[:, None]) + 4 * E23 * ideal
        assert np.all(np.abs(s - ideal) <= step / 2 + slack)
    else:
        assert np.all(row == 1)
        on = block > 2.0 ** -124  # (below that the scale is its least)
        assert np.all((block + off_block)[on] >= 4 * s[on])
        assert np.all((block - off_block)[on] <= 8 * s[on])
    unit = np.repeat(s, n, axis=1)[:, :K] * row[:, None]
    on = unit > 0
    a, e = np.abs(np.where(on, want / np.where(on, unit, 1), 0)), np.where(on, err / np.where(on, unit, 1), 0)
    half = np.where(a <= 2, 0.25, np.where(a <= 4, 0.5, 1.0))
    got = ff.code_value(codes)
    assert np.all(np.abs(np.minimum(a, 6.0) - np.abs(got)) <= half + e + 4 * E23 * a)
    signed = (got != 0) & (np.abs(want) > err)
    assert np.all(np.sign(got[signed]) == np.sign(want[signed]))


@pytest.mark.parametrize("format_", FORMATS)
@pytest.mark.parametrize("g,u", [(-np.inf, 1.0), (np.inf, 0.0), (np.inf, -2.0), (np.nan, 0.0),
                                 (-3.0, np.inf), (-200.0, np.inf), (0.0, np.nan), (3e38, 1e10)])
def test_gated_rows_that_are_no_numbers(format_, g, u):
    """The row's scale says so; its codes and block scales are zeros."""
    K = 70
    v = np.ones((3, 2 * K))
    v[1, 11], v[1, K + 11] = g, u
    x = rows(3, 2 * K, "fp32", 0, 0, v)
    q, _, sf, sc = quantize(x, K, format_, "swiglu")
    assert np.array_equal(np.isnan(sc.cpu().numpy()), [False, True, False])
    assert not ff.unpack_codes(q.cpu().numpy(), K)[1].any()
    assert not ff.unpack_scales(sf.cpu().numpy(), 3, -(-K // ff.BLOCK[format_]))[1].any()
