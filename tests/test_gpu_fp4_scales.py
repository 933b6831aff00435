"""The 4-bit products (include/fp4_gemm.h) with MX block scales from 2^-127 to
2^127 in both operands, on every kernel: a product of two scales may leave fp32's
range where the value that it scales is zero or small."""
import numpy as np
import pytest

from oracle import feed_forward as ff
from test_gpu_fp4 import Operand, forced, gpu_ready, product  # noqa: F401

pytestmark = pytest.mark.gpu
K = 640


def operand(codes, byte):
    import torch
    o = Operand(codes.shape[0], K, "mx", np.random.default_rng(0), row_scale=False)
    o.codes = torch.from_numpy(ff.pack_codes(codes.astype(np.uint8), o.ld)).cuda()
    o.sf = torch.from_numpy(ff.pack_scales(byte.astype(np.uint8))).cuda()
    o.values = ff.values4(codes, byte, "mx")
    return o


@pytest.mark.parametrize("M", [1, 2, 4])
@pytest.mark.parametrize("forced", ["few", "slim", "narrow", "wide"], indirect=True)  # noqa: F811
def test_large_scales_of_values_that_do_not_meet(forced, M):  # noqa: F811
    """Where one operand holds values the other holds zeros: the product is zero,
    whatever the scales."""
    rng = np.random.default_rng(M)
    ca, cb = rng.integers(0, 16, (M, K)), rng.integers(0, 16, (140, K))
    ca[:, 1::2], cb[:, 0::2] = 0, 0
    a = operand(ca, rng.integers(0, 255, (M, K // 32)))
    b = operand(cb, rng.integers(0, 255, (140, K // 32)))
    assert not product("fp32", a, b).any()


@pytest.mark.parametrize("forced", ["few", "slim", "narrow", "wide"], indirect=True)  # noqa: F811
@pytest.mark.parametrize("ea,eb,code", [(64, 64, 1), (127, 1, 1), (1, 127, 9), (63, 63, 3),
                                        (127, -127, 7), (-127, 127, 6), (127, 0, 1), (-70, -70, 5),
                                        (-127, -15, 2), (-74, -74, 7)])
def test_products_at_the_ends_are_exact(forced, ea, eb, code):  # noqa: F811
    """One code in each operand: the result is an fp32 number, kept exactly."""
    ca, cb = np.zeros((3, K), int), np.zeros((140, K), int)
    ca[:, 333], cb[:, 333] = code, 1
    a = operand(ca, np.full((3, K // 32), ea + 127))
    b = operand(cb, np.full((140, K // 32), eb + 127))
    ref = a.values @ b.values.T
    assert np.all(ref.astype(np.float32) == ref) and ref.all()
    assert np.array_equal(product("fp32", a, b), ref)


@pytest.mark.parametrize("forced", ["few", "slim", "narrow", "wide"], indirect=True)  # noqa: F811
def test_results_past_the_range_are_infinite(forced):  # noqa: F811
    ca, cb = np.zeros((2, K), int), np.zeros((140, K), int)
    ca[:, 7], cb[:, 7] = 7, 7
    ca[1] += 8 * (ca[1] > 0)  # the second row's sign
    a, b = operand(ca, np.full((2, K // 32), 254)), operand(cb, np.full((140, K // 32), 192))
    got = product("fp32", a, b)
    assert np.all(got[0] == np.inf) and np.all(got[1] == -np.inf)
