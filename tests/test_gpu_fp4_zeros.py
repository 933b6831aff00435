"""What the 4-bit quantiser and the norm write for values that count as zero
(include/fp4_gemm.h): codes 0 or 8 by the value's sign, scales 0."""
import numpy as np
import pytest

from test_gpu_fp4 import gpu_ready, quantize, rows  # noqa: F401
from oracle import feed_forward as ff

pytestmark = pytest.mark.gpu
K = 96


def values():
    rng = np.random.default_rng(3)
    sign = rng.choice([-1.0, 1.0], (4, K))
    v = sign * np.array([[2.0 ** -110], [0.0], [1.0], [2.0 ** -149]])
    v[2, 16:48] *= 2.0 ** -40  # two blocks far below the row's largest: their scale rounds to 0
    return v, sign


def check(codes, byte, scale, sign):
    zero = 8 * (sign < 0)
    for r in (0, 1, 3):
        assert np.array_equal(codes[r], zero[r]) and not byte[r].any() and scale[r] == 0
    assert np.array_equal(codes[2, 16:48], zero[2, 16:48]) and not byte[2, 1:3].any()
    assert np.all(np.abs(ff.code_value(codes[2, :16])) == 6) and scale[2] > 0


def test_codes_of_zeros_have_the_values_signs():
    v, sign = values()
    x = rows(4, K, "fp32", 0, 0, v)
    q, _, sf, sc = quantize(x, K, "nv")
    check(ff.unpack_codes(q.cpu().numpy(), K), ff.unpack_scales(sf.cpu().numpy(), 4, K // 16),
          sc.cpu().numpy(), sign)


def test_the_norm_writes_the_same():
    import torch
    import dense_fp32_matrix_03_gb300 as lib
    v, sign = values()
    x = rows(4, K, "fp32", 0, 0, v)
    q = torch.empty(4, K // 2, dtype=torch.uint8, device="cuda")
    sf = torch.empty(lib.sgemm_fp4_scales_size("nv", 4, K), dtype=torch.uint8, device="cuda")
    sc = torch.empty(4, device="cuda")
    lib.check(lib.sgemm_rms_norm_fp4("fp32", "nv", 4, K, 1e-5, x.ptr, x.ld, None, 0, None, None, 0,
                                     q, K, sf, sc))
    check(ff.unpack_codes(q.cpu().numpy(), K), ff.unpack_scales(sf.cpu().numpy(), 4, K // 16),
          sc.cpu().numpy(), sign)
