"""The row quantiser of the gated activation (include/int8_gemm.h) at the ends
of fp32's range."""
import numpy as np
import pytest

from test_gpu_experts import Rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu_ready():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import dense_fp32_matrix_03_gb300 as lib
    lib.load()
    torch.cuda.init()


@pytest.mark.parametrize("type_", ["bf16", "fp32"])
def test_quantize_gated_rows_past_the_range(type_):
    """Finite gates and values whose product is past fp32: scale NaN, codes 0,
    in that row alone; gates far below zero leave zeros, not NaN."""
    import torch
    import dense_fp32_matrix_03_gb300 as lib
    K = 40
    v = np.ones((4, 2 * K))
    v[1, 3], v[1, K + 3] = 1e30, 1e30
    v[2, 5], v[2, K + 5] = -1e30, 1e4
    v[3, :K] = -200.0
    x = Rows(4, 2 * K, type_, values=v)
    q = torch.full((4, K), 77, dtype=torch.int8, device="cuda")
    s = torch.full((4,), -1.0, device="cuda")
    assert lib.sgemm_i8_quantize_rows(type_, "swiglu", 4, K, x.ptr, x.ld, q, K, s) == lib.SGEMM_OK
    assert torch.isnan(s).tolist() == [False, True, False, False]
    assert not q[1].any() and s[3] == 0 and not q[3].any()
    assert bool((q[0] == 127).all()) and q[2, 5] == 0 and bool((q[2] == 127).sum() == K - 1)
