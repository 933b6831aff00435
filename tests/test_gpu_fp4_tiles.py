"""GPU parity of the 4-bit products (include/fp4_gemm.h) over many tiles a CTA
pair, against the oracle, element by element; bounds as in test_gpu_fp4.py."""
import numpy as np
import pytest

from oracle import feed_forward as ff
from test_gpu_fp4 import Operand, bound, forced, gpu_ready, product  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("type_", ["fp32", "bf16"])
@pytest.mark.parametrize("format_", ["nv", "mx"])
@pytest.mark.parametrize("forced", ["wide"], indirect=True)  # noqa: F811
@pytest.mark.parametrize("M,N,K", [(15400, 785, 96), (12800, 1041, 64), (20000, 767, 32)])
def test_token_scales_stay_with_their_tile(forced, format_, type_, M, N, K):  # noqa: F811
    """A pair's tiles follow each other with token scales some 2^20 apart, and
    the last channels of a tile leave lanes without work: a scale of the next
    tile, read a tile too early, would show in every value."""
    import torch
    rng = np.random.default_rng(M)
    a, b = Operand(M, K, format_, rng, wide=False), Operand(N, K, format_, rng, wide=False)
    size = np.exp2(rng.integers(-10, 11, -(-M // 256))).astype(np.float32)
    a.sc = (a.sc * np.repeat(size, 256)[:M]).astype(np.float32)
    a.scale = torch.from_numpy(a.sc).cuda()
    got = product(type_, a, b)
    ref, mag = ff.product4(a.values, a.sc, b.values, b.sc)
    assert np.all(np.abs(got - ref) <= bound(type_, K, ref, mag))
