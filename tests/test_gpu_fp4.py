"""GPU parity of the 4-bit quantiser and products (include/fp4_gemm.h) against
the oracle (oracle/feed_forward.py), element by element, through the C ABI.

Bounds: the quantiser's codes, block scales and row scales are compared bit for
bit (the definition says every fp32 operation); of the gated activation, whose
exp is rounded as CUDA's is, codes are the nearest value of x times the written
scales' inverse, to 2^-18 of it (silu within 8 e of its value, products and
divisions some more).  Products: u |ref| for the result's rounding, 3 e |ref|
for the scales, and for the sums 0.6 K e + 16 e of the sum of magnitudes: of 64
values of k at a time each product is cut, at worst, two bits below fp32's last
place of the largest number added (64 * 2^-26) and the sum at it (2^-23)."""
import numpy as np
import pytest

from oracle import feed_forward as ff
from test_gpu_experts import E24, SUB, TYPES, U, Rows, tdtype
from test_gpu_norm import check_4_bits

pytestmark = pytest.mark.gpu
FORMATS = ["mx", "nv"]


@pytest.fixture(scope="module", autouse=True)
def gpu_ready():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import dense_fp32_matrix_03_gb300 as lib
    lib.load()
    torch.cuda.init()


def quantize(x, K, format_, act="none", pad=32):
    import torch
    import dense_fp32_matrix_03_gb300 as lib
    M = x.R
    ld = (K + 31) // 32 * 32 + pad
    q = torch.full((M, ld // 2), 0x5A, dtype=torch.uint8, device="cuda")
    sf = torch.full((lib.sgemm_fp4_scales_size(format_, M, K),), 0xA5, dtype=torch.uint8,
                    device="cuda")
    sc = torch.full((M,), -1.0, device="cuda")
    assert lib.sgemm_fp4_quantize_rows(x.type_, act, format_, M, K, x.ptr, x.ld, q, ld, sf,
                                       sc) == lib.SGEMM_OK
    return q, ld, sf, sc


def rows(M, H, type_, pad, offset, values):
    r = Rows(M, H, type_, pad, offset, values)
    r.type_ = type_
    return r


SHAPES = [(1, 1, 0, 0), (2, 7, 0, 1), (3, 16, 0, 0), (5, 31, 0, 0), (4, 33, 0, 0), (9, 100, 4, 4),
          (200, 96, 0, 0), (333, 257, 0, 0), (1, 4096, 0, 0), (7, 1002, 2, 2), (129, 64, 8, 8),
          (2, 8200, 0, 0), (2, 20011, 0, 3), (1000, 130, 0, 0)]


@pytest.mark.parametrize("format_", FORMATS)
@pytest.mark.parametrize("type_", TYPES)
@pytest.mark.parametrize("M,K,pad,offset", SHAPES)
def test_quantiser(type_, format_, M, K, pad, offset):
    rng = np.random.default_rng(K)
    v = rng.standard_normal((M, K)) * np.exp2(rng.integers(-8, 9, (M, 1)))
    v[rng.random((M, K)) < 0.1] = 0
    if M > 1:
        v[1] = 0
    if M > 4:
        v[2, 0], v[3, K - 1] = np.nan, -np.inf
        v[4] = np.exp2(rng.integers(-14, 10, K)) * rng.choice([-1, 1.5, 1.25, 1.75], K)  # ties
    x = rows(M, K, type_, pad, offset, v)
    q, _, sf, sc = quantize(x, K, format_)
    codes, byte, row = ff.quantize4(x.view.float().cpu().numpy(), format_)
    check_4_bits(q, sf, codes, byte)
    assert np.array_equal(sc.cpu().numpy(), row, equal_nan=True)


@pytest.mark.parametrize("format_", FORMATS)
@pytest.mark.parametrize("type_", ["bf16", "fp32"])
def test_quantiser_at_the_ends_of_the_range(type_, format_):
    """The largest numbers, subnormals, a row next to the limit of zero."""
    K = 70
    rng = np.random.default_rng(1)
    v = rng.choice([-1.0, 1, 1.5], (7, K))
    size = np.array([2.0 ** 127, 2.0 ** -126, 2.0 ** -133, 2.0 ** -100, 2.0 ** -101, 1, 2.0 ** -149])
    v = v * size[:, None]
    v[5, 1:] *= np.exp2(-rng.integers(0, 60, K - 1))  # blocks far below the row's largest
    x = rows(7, K, type_, 0, 0, v)
    q, _, sf, sc = quantize(x, K, format_)
    codes, byte, row = ff.quantize4(x.view.float().cpu().numpy(), format_)
    check_4_bits(q, sf, codes, byte)
    assert np.array_equal(sc.cpu().numpy(), row)


@pytest.mark.parametrize("format_", FORMATS)
@pytest.mark.parametrize("type_", TYPES)
@pytest.mark.parametrize("M,K,pad,offset", [(3, 16, 0, 0), (5, 31, 0, 1), (200, 96, 8, 8),
                                            (9, 1002, 0, 0), (2, 8200, 0, 0), (64, 2048, 0, 0)])
def test_quantiser_of_the_gated_activation(type_, format_, M, K, pad, offset):
    rng = np.random.default_rng(K)
    v = rng.standard_normal((M, 2 * K)) * np.exp2(rng.integers(-3, 4, (M, 1)))
    if M > 4:
        v[1] = 0
        v[2, K + 3] = np.nan
        v[3, 5] = np.inf
        v[4, :K] = -200.0  # silu underflows
    x = rows(M, 2 * K, type_, pad, offset, v)
    q, _, sf, sc = quantize(x, K, format_, "swiglu")
    xv = x.np()
    with np.errstate(over="ignore", invalid="ignore"):
        g = xv[:, :K]
        want = g / (1 + np.exp(-g)) * xv[:, K:]
    ok = np.isfinite(want).all(1)
    got_row = sc.double().cpu().numpy()
    assert np.array_equal(np.isnan(got_row), ~ok)
    codes = ff.unpack_codes(q.cpu().numpy(), K)
    byte = ff.unpack_scales(sf.cpu().numpy(), M, -(-K // ff.BLOCK[format_]))
    assert not codes[~ok].any() and not byte[~ok].any()
    want, codes, byte, got_row = want[ok], codes[ok], byte[ok], got_row[ok]
    top = np.abs(want).max(1)
    n = ff.BLOCK[format_]
    blocks = np.zeros((want.shape[0], byte.shape[1] * n))
    blocks[:, :K] = np.abs(want)
    blocks = blocks.reshape(want.shape[0], -1, n).max(2)
    s = ff.scale_value(byte, format_)
    if format_ == "nv":
        row = np.where(top >= 2.0 ** -100, top / 2688, 0)
        assert np.all(np.abs(got_row - row) <= 2.0 ** -18 * row + 1e-38)
        ideal = np.where(row > 0, 1.0, 0)[:, None] * blocks * 448 / np.where(top > 0, top, 1)[:, None]
        step = np.exp2(np.floor(np.log2(np.maximum(ideal, 2.0 ** -6))) - 3)
        assert np.all(np.abs(s - ideal) <= step / 2 + 2.0 ** -18 * ideal)
    else:
        assert np.all(got_row == 1)
        big = blocks > 1e-30
        assert np.all((blocks / s)[big] >= 4 * (1 - 2.0 ** -18))
        assert np.all((blocks / s)[big] <= 8 * (1 + 2.0 ** -18))
    unit = np.repeat(s, n, axis=1)[:, :K] * got_row[:, None]
    on = unit > 0
    u = np.where(on, want / np.where(on, unit, 1), 0)
    a = np.abs(u)
    half = np.where(a <= 2, 0.25, np.where(a <= 4, 0.5, 1.0))
    off = np.abs(np.minimum(a, 6.0) - np.abs(ff.code_value(codes)))
    assert np.all(off <= half + 2.0 ** -18 * a + 1e-30)
    # (a value that underflows has no sign to speak of)
    signed = (np.abs(ff.code_value(codes)) > 0)
    assert np.all(np.sign(ff.code_value(codes))[signed] == np.sign(u)[signed])
    assert not codes[~on].any() or np.all(np.abs(ff.code_value(codes))[~on] == 0)


class Operand:
    """Rows in 4 bits with random codes and scales, packed for the library; what
    lies behind rows, blocks and values is garbage where the layout allows it."""

    def __init__(self, M, K, format_, rng, pad=0, row_scale=True, wide=True):
        import torch
        self.M, self.K, self.format_ = M, K, format_
        self.ld = max((K + 31) // 32 * 32 + pad, 32)
        codes = rng.integers(0, 16, (M, K)).astype(np.uint8)
        blocks = -(-K // ff.BLOCK[format_])
        if format_ == "nv":
            lo, hi = (0, 127) if wide else (48, 64)
        else:
            lo, hi = (100, 140) if wide else (120, 130)
        byte = rng.integers(lo, hi, (M, blocks)).astype(np.uint8)
        packed = ff.pack_codes(codes, self.ld)
        used = -(-K // 2)
        packed[:, used:] = rng.integers(0, 256, (M, self.ld // 2 - used))
        self.codes = torch.from_numpy(packed).cuda()
        fill = 0x7F if format_ == "nv" else 0xFF  # NaN behind the last row
        self.sf = torch.from_numpy(ff.pack_scales(byte, fill)).cuda()
        sc = ((0.5 + rng.random(M)) / 16).astype(np.float32)
        self.scale = torch.from_numpy(sc).cuda() if row_scale else None
        self.sc = sc if row_scale else np.ones(M, np.float32)
        self.values = ff.values4(codes, byte, format_)


def product(type_, a, b, ldc=None, offset=0, check=None):
    """C of the library, and the part around it untouched."""
    import torch
    import dense_fp32_matrix_03_gb300 as lib
    M, N, K = a.M, b.M, a.K
    ldc = ldc or N
    c = torch.full((offset + M * ldc + 8,), float("nan"), dtype=tdtype(type_), device="cuda")
    ptr = c.data_ptr() + offset * c.element_size()
    assert lib.sgemm_fp4(type_, a.format_, M, N, K, a.codes, a.ld, a.sf, a.scale, b.codes, b.ld,
                         b.sf, b.scale, ptr, ldc) == lib.SGEMM_OK
    assert lib.sgemm_poll_error() == lib.SGEMM_OK
    body = c[offset:offset + M * ldc].view(M, ldc)
    assert bool(torch.isnan(c[:offset].float()).all())
    assert bool(torch.isnan(c[offset + M * ldc:].float()).all())
    assert bool(torch.isnan(body[:, N:].float()).all())
    return body[:, :N].double().cpu().numpy()


def bound(type_, K, ref, mag):
    return (U[type_] + 3 * E24) * np.abs(ref) + (0.6 * K + 16) * E24 * mag + SUB


# M, N, K: one token to more than a tile of any kernel, odd and ragged sizes,
# k of one value, of less and more than a block, a scale tile and a stage
SIZES = [(1, 1, 1), (1, 9, 15), (2, 64, 16), (3, 130, 33), (4, 100, 64), (5, 257, 100),
         (8, 128, 128), (9, 300, 129), (16, 96, 255), (17, 200, 256), (31, 129, 257),
         (33, 640, 512), (64, 384, 300), (65, 1000, 777), (100, 136, 1024), (128, 128, 384),
         (129, 260, 640), (200, 777, 96), (256, 512, 1000), (300, 250, 2049), (513, 390, 320),
         (1000, 1500, 777)]


@pytest.mark.parametrize("format_", FORMATS)
@pytest.mark.parametrize("type_", TYPES)
@pytest.mark.parametrize("M,N,K", SIZES)
def test_product(type_, format_, M, N, K):
    rng = np.random.default_rng(M + N + K)
    wide = type_ != "fp16"  # (its range)
    a = Operand(M, K, format_, rng, pad=32 * (K % 3), wide=wide)
    b = Operand(N, K, format_, rng, pad=64 * (N % 2), wide=wide)
    if type_ == "fp16":
        a.scale *= 2.0 ** -8
        a.sc = a.sc * np.float32(2.0 ** -8)
    got = product(type_, a, b, ldc=N + (M % 3), offset=(M % 2))
    ref, mag = ff.product4(a.values, a.sc, b.values, b.sc)
    assert np.isfinite(ref).all()
    assert np.all(np.abs(got - ref) <= bound(type_, K, ref, mag))


@pytest.mark.parametrize("format_", FORMATS)
@pytest.mark.parametrize("M", [1, 5, 40, 300])
def test_product_without_row_scales(format_, M):
    rng = np.random.default_rng(M)
    for sa, sb in ((False, False), (True, False), (False, True)):
        a = Operand(M, 200, format_, rng, row_scale=sa, wide=False)
        b = Operand(72, 200, format_, rng, row_scale=sb, wide=False)
        ref, mag = ff.product4(a.values, a.sc, b.values, b.sc)
        assert np.all(np.abs(product("fp32", a, b) - ref) <= bound("fp32", 200, ref, mag))


@pytest.mark.parametrize("M", [1, 3, 16, 70, 260])
@pytest.mark.parametrize("format_", FORMATS)
def test_product_of_whole_numbers_is_exact(format_, M):
    """Codes of whole numbers, scales of one: sums below 2^24 are exact."""
    import torch
    rng = np.random.default_rng(M)
    N, K = 150, 600
    one = 0x38 if format_ == "nv" else 127
    ops = []
    for r in (M, N):
        o = Operand(r, K, format_, rng, row_scale=False)
        codes = rng.choice([0, 2, 4, 5, 6, 7, 10, 12, 13, 14, 15], (r, K)).astype(np.uint8)
        byte = np.full((r, -(-K // ff.BLOCK[format_])), one, np.uint8)
        o.codes = torch.from_numpy(ff.pack_codes(codes, o.ld)).cuda()
        o.sf = torch.from_numpy(ff.pack_scales(byte)).cuda()
        o.values = ff.values4(codes, byte, format_)
        ops.append(o)
    assert np.array_equal(product("fp32", *ops), ops[0].values @ ops[1].values.T)


@pytest.mark.parametrize("forced", ["few", "slim", "narrow", "wide"], indirect=True)
@pytest.mark.parametrize("lo", [62, 180])
def test_products_of_very_small_and_very_large_scales(forced, lo):
    """Block scales of some 2^-64 (2^54) in both operands: sums near fp32's ends
    keep their last places (half a unit in the last place of 2^-149 besides)."""
    import torch
    rng = np.random.default_rng(lo)
    K = 640
    ops = []
    for r in (4, 140):
        o = Operand(r, K, "mx", rng, row_scale=False)
        codes = rng.integers(0, 16, (r, K)).astype(np.uint8)
        byte = rng.integers(lo, lo + 4, (r, K // 32)).astype(np.uint8)
        o.codes = torch.from_numpy(ff.pack_codes(codes, o.ld)).cuda()
        o.sf = torch.from_numpy(ff.pack_scales(byte)).cuda()
        o.values = ff.values4(codes, byte, "mx")
        ops.append(o)
    ref, mag = ff.product4(ops[0].values, ops[0].sc, ops[1].values, ops[1].sc)
    assert np.abs(ref).max() < 3e38
    got = product("fp32", *ops)
    assert np.all(np.abs(got - ref) <= bound("fp32", K, ref, mag) - SUB + K * 2.0 ** -149)


@pytest.mark.parametrize("M", [1, 6, 50, 300])
def test_scales_that_are_no_number(M):
    """A NaN scale of a token or a channel reaches its row or column alone, a
    NaN block scale too."""
    import torch
    rng = np.random.default_rng(M)
    N, K = 140, 320
    for format_ in FORMATS:
        a, b = Operand(M, K, format_, rng, wide=False), Operand(N, K, format_, rng, wide=False)
        a.scale[M - 1] = float("nan")
        b.scale[7] = float("inf")
        byte = ff.unpack_scales(b.sf.cpu().numpy(), N, -(-K // ff.BLOCK[format_])).copy()
        byte[11, 3] = 0x7F if format_ == "nv" else 0xFF
        b.sf = torch.from_numpy(ff.pack_scales(byte)).cuda()
        got = product("fp32", a, b)
        spoilt = np.zeros((M, N), bool)
        spoilt[M - 1], spoilt[:, 11] = True, True
        assert np.isnan(got[spoilt]).all()
        assert not np.isfinite(got[:, 7]).any()
        spoilt[:, 7] = True
        ref, mag = ff.product4(a.values, a.sc, b.values, b.sc)
        ok = ~spoilt
        assert np.all((np.abs(got - ref) <= bound("fp32", K, ref, mag))[ok])


def test_product_of_no_values_is_zero():
    import torch
    import dense_fp32_matrix_03_gb300 as lib
    c = torch.full((5, 9), 3.0, device="cuda")
    assert lib.sgemm_fp4("fp32", "nv", 5, 9, 0, None, 32, None, None, None, 32, None, None, c,
                         9) == lib.SGEMM_OK
    assert not c.cpu().numpy().any()


@pytest.mark.parametrize("format_", FORMATS)
@pytest.mark.parametrize("M", [3, 200])
def test_quantised_then_multiplied_on_streams_and_in_a_graph(format_, M):
    """A layer as a program calls it: the quantiser, then the product, twice on
    different streams at once and replayed from a graph; the same bits each
    time."""
    import torch
    import dense_fp32_matrix_03_gb300 as lib
    rng = np.random.default_rng(M)
    N, K = 640, 512
    b = Operand(N, K, format_, rng, wide=False)
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")

    def buffers():
        return (torch.zeros(M, K // 2, dtype=torch.uint8, device="cuda"),
                torch.zeros(lib.sgemm_fp4_scales_size(format_, M, K), dtype=torch.uint8,
                            device="cuda"),
                torch.zeros(M, device="cuda"), torch.zeros(M, N, dtype=torch.bfloat16, device="cuda"))

    def layer(bufs, stream=None):
        q, sf, sc, y = bufs
        lib.check(lib.sgemm_fp4_quantize_rows("bf16", "none", format_, M, K, x, K, q, K, sf, sc,
                                              stream))
        lib.check(lib.sgemm_fp4("bf16", format_, M, N, K, q, K, sf, sc, b.codes, b.ld, b.sf,
                                b.scale, y, N, stream))

    captured, eager = buffers(), [(buffers(), torch.cuda.Stream()) for _ in range(2)]
    layer(captured)  # (attributes are set outside the capture)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer(captured)
        layer(captured)
    for seed in (1, 2):
        x.copy_(torch.from_numpy(np.random.default_rng(seed).standard_normal((M, K))))
        torch.cuda.synchronize()
        graph.replay()
        for bufs, stream in eager:
            layer(bufs, stream)
        torch.cuda.synchronize()
        assert lib.sgemm_poll_error() == lib.SGEMM_OK
        codes, byte, row = ff.quantize4(x.float().cpu().numpy(), format_)
        ref, mag = ff.product4(ff.values4(codes, byte, format_), row, b.values, b.sc)
        got = captured[3].double().cpu().numpy()
        assert np.all(np.abs(got - ref) <= bound("bf16", K, ref, mag))
        for bufs, _ in eager:
            assert torch.equal(bufs[3], captured[3])


@pytest.fixture
def forced(request):
    """Every product of the test on one kernel."""
    import dense_fp32_matrix_03_gb300 as lib
    lib.check(lib.sgemm_fp4_tune_force(request.param))
    yield request.param
    lib.check(lib.sgemm_fp4_tune_force("auto"))


# tiles of 128 and 256, one short of them and one past them; k of less than a
# stage (256), of several times the ring; many tiles a cluster (both
# accumulators, their shared columns, several rounds)
KERNEL_SIZES = [(1, 128, 256), (16, 130, 64), (32, 1000, 3000), (3, 60000, 300), (64, 200, 2600), (33, 127, 700), (127, 129, 512), (128, 256, 1280),
                (129, 255, 257), (255, 257, 1536), (256, 256, 2048), (257, 513, 768),
                (700, 640, 4096), (2100, 1900, 300), (3000, 4100, 128), (64, 30000, 100),
                (6000, 300, 520)]


@pytest.mark.parametrize("type_", ["bf16", "fp32"])
@pytest.mark.parametrize("format_", FORMATS)
@pytest.mark.parametrize("forced", ["slim", "narrow", "wide"], indirect=True)
@pytest.mark.parametrize("M,N,K", KERNEL_SIZES)
def test_every_kernel(forced, type_, format_, M, N, K):
    import dense_fp32_matrix_03_gb300 as lib
    rng = np.random.default_rng(M + N + K)
    a, b = Operand(M, K, format_, rng, wide=False), Operand(N, K, format_, rng, wide=False)
    got = product(type_, a, b)
    if forced != "slim" or M <= 32:  # (it takes no more)
        assert lib.sgemm_fp4_last_kernel() == lib.FP4_KERNELS[forced]
    ref, mag = ff.product4(a.values, a.sc, b.values, b.sc)
    assert np.all(np.abs(got - ref) <= bound(type_, K, ref, mag))


@pytest.mark.parametrize("type_", TYPES)
@pytest.mark.parametrize("format_", FORMATS)
@pytest.mark.parametrize("forced", ["few"], indirect=True)
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 33, 1023), (2, 128, 1024), (3, 129, 1025),
                                   (4, 250, 4096), (1, 1000, 5000), (2, 4, 9001), (4, 97, 31),
                                   (3, 640, 2048), (1, 130, 64)])
def test_few_tokens(forced, type_, format_, M, N, K):
    import dense_fp32_matrix_03_gb300 as lib
    rng = np.random.default_rng(M + N + K)
    a, b = Operand(M, K, format_, rng, wide=False), Operand(N, K, format_, rng, wide=False)
    got = product(type_, a, b, ldc=N + 3)
    assert lib.sgemm_fp4_last_kernel() == lib.SGEMM_FP4_KERNEL_FEW
    ref, mag = ff.product4(a.values, a.sc, b.values, b.sc)
    assert np.all(np.abs(got - ref) <= bound(type_, K, ref, mag))


@pytest.mark.parametrize("forced", ["slim", "narrow"], indirect=True)
@pytest.mark.parametrize("M,N,K", [(16, 128, 4096), (30, 300, 5000), (16, 256, 8192),
                                   (7, 130, 4352), (32, 1000, 9001), (3, 4000, 6145)])
def test_clusters_that_share_k(forced, M, N, K):
    import dense_fp32_matrix_03_gb300 as lib
    rng = np.random.default_rng(K)
    for format_ in FORMATS:
        a, b = Operand(M, K, format_, rng, wide=False), Operand(N, K, format_, rng, wide=False)
        got = product("fp32", a, b, ldc=N + 1)
        assert lib.sgemm_fp4_last_split_count() > 1
        ref, mag = ff.product4(a.values, a.sc, b.values, b.sc)
        assert np.all(np.abs(got - ref) <= bound("fp32", K, ref, mag))


def test_hooks_refuse_what_they_do_not_know():
    import dense_fp32_matrix_03_gb300 as lib
    assert lib.sgemm_fp4_tune_force(-1) == lib.SGEMM_ERR_INVALID_ARG
    assert lib.sgemm_fp4_tune_force(5) == lib.SGEMM_ERR_INVALID_ARG
