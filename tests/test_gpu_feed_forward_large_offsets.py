"""Rows, results and experts more than 2^31 elements apart: offsets of the norm,
its gradient, the 4-bit quantiser and products and the few-token expert layer
that pass 32 bits.  Only the rows in use are written; the bounds are those of the
operators' own tests."""
import numpy as np
import pytest

from oracle import feed_forward as ff
from test_gpu_experts import E24, SUB, U
from test_gpu_fp4 import Operand, bound

pytestmark = pytest.mark.gpu
FAR = 2 ** 30 + 64  # elements between rows: the third row is past 2^31
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def gpu_ready():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import dense_fp32_matrix_03_gb300 as lib
    lib.load()
    torch.cuda.init()


class Far:
    """R rows of n elements, FAR apart."""

    def __init__(self, R, n, dtype, values=None):
        import torch
        self.buf = torch.empty((R - 1) * FAR + n, dtype=dtype, device="cuda")
        self.rows = [self.buf[i * FAR:i * FAR + n] for i in range(R)]
        if values is not None:
            for row, v in zip(self.rows, values):
                row.copy_(torch.from_numpy(v).to(dtype))

    def np(self):
        return np.stack([r.double().cpu().numpy() for r in self.rows])


def test_norm_and_gradient():
    import torch
    import dense_fp32_matrix_03_gb300 as lib
    M, H = 3, 264
    rng = np.random.default_rng(1)
    bf = torch.bfloat16
    x = Far(M, H, bf, rng.standard_normal((M, H)))
    y = Far(M, H, bf)
    lib.check(lib.sgemm_rms_norm("bf16", M, H, EPS, x.buf, FAR, None, 0, None, None, 0, y.buf, FAR))
    ref, _ = ff.rms_norm(x.np(), np.ones(H), EPS)
    assert np.all(np.abs(y.np() - ref) <= (U["bf16"] + 24 * E24) * np.abs(ref))
    dx = Far(M, H, bf)
    dw = torch.empty(H, device="cuda")
    size = lib.sgemm_rms_norm_grad_workspace_size(M, H)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    lib.check(lib.sgemm_rms_norm_grad("bf16", M, H, EPS, x.buf, FAR, None, y.buf, FAR, None, 0,
                                      dx.buf, FAR, dw, ws, size))
    gx, gw, mx, mw = ff.rms_norm_grad(x.np(), np.ones(H), y.np(), np.zeros((M, H)), EPS)
    assert np.all(np.abs(dx.np() - gx) <= U["bf16"] * np.abs(gx) + 48 * E24 * mx)
    assert np.all(np.abs(dw.double().cpu().numpy() - gw) <= 80 * E24 * mw)
    del y, dx
    q = torch.empty((M, 288), dtype=torch.int8, device="cuda")
    sc = torch.empty(M, device="cuda")
    lib.check(lib.sgemm_rms_norm_i8("bf16", M, H, EPS, x.buf, FAR, None, 0, None, None, 0, q, 288, sc))
    codes, _ = ff.quantize8(x.np().astype(np.float32))
    assert np.array_equal(q[:, :H].cpu().numpy(), codes)
    sf = torch.empty(lib.sgemm_fp4_scales_size("nv", M, H), dtype=torch.uint8, device="cuda")
    q4 = torch.empty((M, 144), dtype=torch.uint8, device="cuda")
    lib.check(lib.sgemm_fp4_quantize_rows("bf16", "none", "nv", M, H, x.buf, FAR, q4, 288, sf, sc))
    codes, byte, row = ff.quantize4(x.np().astype(np.float32), "nv")
    assert np.array_equal(ff.unpack_codes(q4.cpu().numpy(), H), codes)
    assert np.array_equal(sc.cpu().numpy(), row)


@pytest.mark.parametrize("kernel,M", [("few", 3), ("slim", 3), ("narrow", 3), ("wide", 3)])
def test_products(kernel, M):
    """Codes a gigabyte apart and results past 2^31 elements."""
    import torch
    import dense_fp32_matrix_03_gb300 as lib
    rng = np.random.default_rng(2)
    N, K = 6, 300
    a, b = Operand(M, K, "nv", rng, wide=False), Operand(N, K, "nv", rng, wide=False)
    ld = 2 ** 31 - 64  # the longest leading dimension, in codes
    buf = torch.empty((N - 1) * (ld // 2) + b.codes.shape[1], dtype=torch.uint8, device="cuda")
    for i in range(N):
        buf[i * (ld // 2):i * (ld // 2) + b.codes.shape[1]] = b.codes[i]
    c = Far(M, N, torch.bfloat16)
    try:
        lib.check(lib.sgemm_fp4_tune_force(kernel))
        lib.check(lib.sgemm_fp4("bf16", "nv", M, N, K, a.codes, a.ld, a.sf, a.scale, buf, ld, b.sf,
                                b.scale, c.buf, FAR))
        assert lib.sgemm_fp4_last_kernel() == lib.FP4_KERNELS[kernel]
    finally:
        lib.sgemm_fp4_tune_force("auto")
    lib.check(lib.sgemm_poll_error())
    ref, mag = ff.product4(a.values, a.sc, b.values, b.sc)
    assert np.all(np.abs(c.np() - ref) <= bound("bf16", K, ref, mag))


def test_experts_layer():
    import torch
    import dense_fp32_matrix_03_gb300 as lib
    rng = np.random.default_rng(3)
    T, k, E, H, F = 4, 2, 3, 96, 48
    w1 = rng.integers(-127, 128, (E, 2 * F, H)).astype(np.int8)
    w2 = rng.integers(-127, 128, (E, H, F)).astype(np.int8)
    W1, W2 = Far(E, 2 * F * H, torch.int8), Far(E, H * F, torch.int8)
    for e in range(E):
        W1.rows[e].copy_(torch.from_numpy(w1[e].reshape(-1)))
        W2.rows[e].copy_(torch.from_numpy(w2[e].reshape(-1)))
    s1 = ((0.5 + rng.random((E, 2 * F))) / 700).astype(np.float32)
    s2 = ((0.5 + rng.random((E, H))) / 500).astype(np.float32)
    x = Far(T, H, torch.float16, rng.standard_normal((T, H)))
    out = Far(T, H, torch.float16)
    ids = np.array([[2, 0], [1, 2], [2, 2], [0, 1]], np.int32)
    size = lib.sgemm_experts_layer_workspace_size(T, k, H, F)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    dev = lambda v: torch.from_numpy(v).cuda()  # noqa: E731
    lib.check(lib.sgemm_experts_layer("fp16", "i8", T, k, E, H, F, x.buf, FAR, dev(ids), None, W1.buf,
                                      H, FAR, dev(s1), W2.buf, F, FAR, dev(s2), out.buf, FAR, ws,
                                      size))
    lib.check(lib.sgemm_poll_error())
    ref, err = ff.experts_layer(x.np(), ids, None, w1.astype(np.float64), s1.astype(np.float64),
                                w2.astype(np.float64), s2.astype(np.float64), U["fp16"])
    assert np.all(np.abs(out.np() - ref) <= err + (U["fp16"] + 2.0 ** -23) * np.abs(ref) + SUB)
