"""GPU parity of the 8-bit integer products (include/int8_gemm.h) against the
fp64 oracle (oracle/expert_layer.py), element by element, through the C ABI.

Bound, derived from the arithmetic: u = half a unit in the last place of the
result type (bf16 2^-8, fp16 2^-11, fp32 2^-24); the sum is an integer, exact
in fp32 up to 2^24, then scaled twice and rounded: (u + 3 * 2^-24) |ref|.
Where sum|a||b| can pass 2^24 the tensor cores may lose 2^-23 of the running
sum with each 16 values of k: + K/16 * 2^-23 * sum|a||b| sa sb."""
import numpy as np
import pytest

from oracle import expert_layer as ex

pytestmark = pytest.mark.gpu

U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
TYPES = ["bf16", "fp16", "fp32"]


@pytest.fixture(scope="module", autouse=True)
def gpu_ready():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import dense_fp32_matrix_03_gb300 as lib
    lib.load()
    torch.cuda.init()


def tdtype(type_):
    import torch
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[type_]


def codes(shape, ld, rng, offset=0, extreme=False):
    """(device buffer, address, host values): 8-bit rows with pitch ld, the
    pad bytes set to 99."""
    import torch
    v = rng.integers(-128, 128, shape).astype(np.int8)
    if extreme:
        v = np.where(rng.random(shape) < 0.97, 127, v).astype(np.int8)
    buf = np.full(offset + int(np.prod(shape[:-1])) * ld + 1, 99, np.int8)
    buf[offset:-1].reshape(*shape[:-1], ld)[..., :shape[-1]] = v
    d = torch.from_numpy(buf).cuda()
    return d, d.data_ptr() + offset, v


def scales(shape, rng, K):
    return ((0.5 + rng.random(shape)) / np.sqrt(5500.0 * np.sqrt(max(K, 1)))).astype(np.float32)


def tolerance(type_, K, ref, mag, raw):
    return (U[type_] + 3 * 2.0 ** -24) * np.abs(ref) + \
        np.where(raw > 2.0 ** 24, K / 16 * 2.0 ** -23 * mag, 0) + 2.0 ** -24


def pitch(K, how):
    return {"tight": max(K, 1), "pad16": max((K + 15) // 16 * 16, 16), "plus4": K + (-K) % 4 + 4}[how]


def run_dense(type_, M, N, K, how="pad16", ldc_pad=0, offset=0, seed=0, extreme=False, c_off=0):
    import torch
    import dense_fp32_matrix_03_gb300 as lib
    rng = np.random.default_rng(seed + M + N + K)
    ld = pitch(K, how)
    da, pa, a = codes((M, K), ld, rng, offset, extreme)
    db, pb, b = codes((N, K), ld, rng, offset, extreme)
    sa, sb = scales(M, rng, K), scales(N, rng, K)
    ldc = N + ldc_pad
    c = torch.full((c_off + M * ldc,), 7.0, dtype=tdtype(type_), device="cuda")
    assert lib.sgemm_i8(type_, M, N, K, pa, ld, torch.from_numpy(sa).cuda(), pb, ld,
                        torch.from_numpy(sb).cuda(), c.data_ptr() + c_off * c.element_size(),
                        ldc) == lib.SGEMM_OK
    assert lib.sgemm_poll_error() == lib.SGEMM_OK
    got = c.double().cpu().numpy()
    assert (got[:c_off] == 7).all()
    got = got[c_off:].reshape(M, ldc)
    assert (got[:, N:] == 7).all(), "columns past N were written"
    got = got[:, :N]
    ref, mag, raw = ex.product(a, sa, b, sb)
    err = np.abs(got - ref)
    assert np.all(err <= tolerance(type_, K, ref, mag, raw)), float(np.max(err / (mag + 1e-30)))


@pytest.mark.parametrize("type_", TYPES)
@pytest.mark.parametrize("M,N,K", [
    (1, 1, 1), (1, 4096, 4096), (2, 100, 15), (3, 128, 16), (8, 256, 17), (15, 7, 64), (16, 64, 127),
    (17, 129, 128), (32, 4092, 777), (33, 1500, 129), (37, 4092, 4092), (63, 200, 1024),
    (64, 512, 2048), (65, 257, 256), (128, 384, 640), (129, 1000, 500), (200, 640, 1100),
    (255, 256, 96), (90, 2121, 448), (700, 2121, 448), (333, 1026, 64), (256, 256, 512), (257, 300, 1000), (513, 2050, 300), (1000, 1500, 777),
    (17, 1500, 2100), (33, 777, 2049), (40, 1000, 4100), (64, 1024, 4097), (1000, 33, 4099),
    (300, 512, 2048), (40, 256, 2048), (300, 900, 5000)])
def test_dense_shapes(type_, M, N, K):
    run_dense(type_, M, N, K)


@pytest.mark.parametrize("M,N,K", [(70000, 1, 16), (1100000, 3, 32), (3, 70000, 16), (600, 40000, 48)])
def test_dense_lopsided(M, N, K):
    """Many tokens for few channels and the other way: grids near and past
    their limits."""
    run_dense("fp32", M, N, K)


@pytest.mark.parametrize("how", ["tight", "plus4"])
@pytest.mark.parametrize("M,N,K", [(1, 100, 333), (70, 130, 65), (130, 300, 777), (5, 64, 4)])
def test_dense_rows_off_16_bytes(how, M, N, K):
    run_dense("fp32", M, N, K, how)


@pytest.mark.parametrize("offset", [1, 4, 8])
def test_dense_bases_off_16_bytes(offset):
    run_dense("bf16", 70, 130, 256, offset=offset)


@pytest.mark.parametrize("type_", TYPES)
@pytest.mark.parametrize("ldc_pad,c_off", [(1, 0), (8, 0), (0, 1), (3, 2)])
def test_dense_result_pitches(type_, ldc_pad, c_off):
    run_dense(type_, 75, 264, 200, ldc_pad=ldc_pad, c_off=c_off)
    run_dense(type_, 300, 520, 140, ldc_pad=ldc_pad, c_off=c_off)
    run_dense(type_, 2100, 2050, 70, ldc_pad=ldc_pad, c_off=c_off)


@pytest.mark.parametrize("M,N,K", [(16, 128, 1024), (40, 200, 1040), (300, 256, 9000), (5, 128, 16384)])
def test_dense_extreme_codes(M, N, K):
    """Mostly 127 times 127: exact up to K = 1024, and the longest sums."""
    run_dense("fp32", M, N, K, extreme=True)


def test_dense_long_k():
    run_dense("fp32", 40, 70, 131071)


def test_dense_all_minimum():
    """-128 * -128 * 1024 = 2^24, the last exact sum."""
    import torch
    import dense_fp32_matrix_03_gb300 as lib
    for M in (4, 300):
        a = torch.full((M, 1024), -128, dtype=torch.int8, device="cuda")
        b = torch.full((256, 1024), -128, dtype=torch.int8, device="cuda")
        one = torch.ones(max(M, 256), device="cuda")
        c = torch.zeros(M, 256, device="cuda")
        assert lib.sgemm_i8("fp32", M, 256, 1024, a, 1024, one, b, 1024, one, c, 256) == 0
        assert bool((c == 2.0 ** 24).all())


@pytest.mark.parametrize("M,N", [(3, 5), (300, 300)])
def test_dense_no_k(M, N):
    import torch
    import dense_fp32_matrix_03_gb300 as lib
    one = torch.ones(max(M, N), device="cuda")
    c = torch.full((M, N), 7.0, device="cuda")
    assert lib.sgemm_i8("fp32", M, N, 0, None, 1, one, None, 1, one, c, N) == lib.SGEMM_OK
    assert not bool(c.any())


def test_scale_nan_makes_its_row_nan():
    import torch
    import dense_fp32_matrix_03_gb300 as lib
    for M in (5, 300):
        N, K = 130, 64
        a = torch.zeros(M, K, dtype=torch.int8, device="cuda")
        b = torch.ones(N, K, dtype=torch.int8, device="cuda")
        sa, sb = torch.ones(M, device="cuda"), torch.ones(N, device="cuda")
        sa[2] = float("nan")
        c = torch.zeros(M, N, device="cuda")
        assert lib.sgemm_i8("fp32", M, N, K, a, K, sa, b, K, sb, c, N) == lib.SGEMM_OK
        assert bool(torch.isnan(c[2]).all())
        c[2] = 0
        assert not bool(c.any())


def run_experts(type_, counts, N, K, tail=0, how="pad16", offsets=None, seed=1):
    import torch
    import dense_fp32_matrix_03_gb300 as lib
    rng = np.random.default_rng(seed + N + K)
    E, M = len(counts), sum(counts) + tail
    ld = pitch(K, how)
    da, pa, a = codes((M, K), ld, rng)
    db, pb, b = codes((E, N, K), ld, rng)
    sa, sb = scales(M, rng, K), scales((E, N), rng, K)
    sa[M - tail:] = np.nan  # rows past the last expert: never read
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    c = torch.full((M, N), 7.0, dtype=tdtype(type_), device="cuda")
    assert lib.sgemm_i8_experts(type_, M, N, K, E, torch.from_numpy(off).cuda(), pa, ld,
                                torch.from_numpy(sa).cuda(), pb, ld, N * ld,
                                torch.from_numpy(sb).cuda(), c, N) == lib.SGEMM_OK
    assert lib.sgemm_poll_error() == lib.SGEMM_OK
    got = c.double().cpu().numpy()
    assert (got[M - tail:] == 7).all(), "rows past the last expert were written"
    live = slice(0, M - tail)
    ref, mag, raw = (x[live] for x in ex.product_experts(off, a, np.nan_to_num(sa), b, sb, N))
    err = np.abs(got[live] - ref)
    assert np.all(err <= tolerance(type_, K, ref, mag, raw)), float(np.max(err / (mag + 1e-30)))


@pytest.mark.parametrize("type_", TYPES)
@pytest.mark.parametrize("counts,N,K,tail", [
    ([1], 64, 64, 0), ([0, 3, 0, 0, 5], 130, 200, 2), ([2] * 32, 256, 256, 0),
    ([1, 0, 130, 17, 64, 0, 65, 3], 300, 333, 5), ([300, 0, 1, 257, 256], 512, 700, 0),
    ([0, 0, 0], 128, 128, 4), ([1000, 2], 384, 128, 1), ([5] * 100, 70, 96, 3)])
def test_experts(type_, counts, N, K, tail):
    run_experts(type_, counts, N, K, tail)


@pytest.mark.parametrize("how", ["tight", "plus4"])
def test_experts_off_16_bytes(how):
    run_experts("fp32", [3, 0, 90, 20], 130, 77, 2, how)


def test_experts_most():
    counts = [int(x) for x in np.random.default_rng(2).integers(0, 4, 1024)]
    run_experts("bf16", counts, 40, 48, 1)


def test_experts_offsets_are_kept_inside():
    """Offsets outside the M rows are cut to them."""
    import torch
    import dense_fp32_matrix_03_gb300 as lib
    M, N, K, E = 40, 64, 64, 3
    a = torch.ones(M, K, dtype=torch.int8, device="cuda")
    b = torch.ones(E, N, K, dtype=torch.int8, device="cuda") * \
        torch.arange(1, 4, dtype=torch.int8, device="cuda")[:, None, None]
    one = torch.ones(E * N, device="cuda")
    c = torch.full((M, N), 7.0, device="cuda")
    off = torch.tensor([-5, 10, 30, 1000], dtype=torch.int32, device="cuda")
    assert lib.sgemm_i8_experts("fp32", M, N, K, E, off, a, K, one, b, K, N * K, one, c, N) == 0
    assert bool((c[:10] == 64).all() and (c[10:30] == 128).all() and (c[30:] == 192).all())


def test_weights_beyond_32_bit_offsets():
    """Experts' weights of more than 2^31 bytes; results checked in the last."""
    import torch
    import dense_fp32_matrix_03_gb300 as lib
    E, N, K = 70, 8192, 4096
    b = torch.zeros(E, N, K, dtype=torch.int8, device="cuda")
    gen = torch.Generator(device="cuda")
    gen.manual_seed(4)
    b[-1] = torch.randint(-128, 128, (N, K), device="cuda", dtype=torch.int8, generator=gen)
    for M in (9, 300):
        a = torch.randint(-128, 128, (M, K), device="cuda", dtype=torch.int8, generator=gen)
        off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        off[-1] = M
        one = torch.ones(E * N, device="cuda")
        c = torch.zeros(M, N, device="cuda")
        assert lib.sgemm_i8_experts("fp32", M, N, K, E, off, a, K, one, b, K, N * K, one, c, N) == 0
        ref = a.double() @ b[-1].double().t()
        mag = a.double().abs() @ b[-1].double().abs().t()
        assert bool(((c - ref).abs() <= 2.0 ** -24 * ref.abs() + K / 16 * 2.0 ** -23 * mag).all())


def test_two_streams_and_a_graph():
    """Calls on two streams at once, and a captured call replayed on new
    inputs, give what a plain call gives."""
    import torch
    import dense_fp32_matrix_03_gb300 as lib
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    for M, N, K in ((5, 512, 2048), (300, 1024, 512)):
        rnd = lambda *s: torch.randint(-128, 128, s, device="cuda", dtype=torch.int8, generator=gen)
        a, b = rnd(M, K), rnd(N, K)
        sa, sb = torch.rand(M, device="cuda", generator=gen), torch.rand(N, device="cuda", generator=gen)
        want = torch.zeros(M, N, device="cuda")
        call = lambda c, s=None: lib.check(
            lib.sgemm_i8("fp32", M, N, K, a, K, sa, b, K, sb, c, N, s))
        call(want)
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(2)]
        outs = [torch.zeros(M, N, device="cuda") for _ in streams]
        torch.cuda.synchronize()
        for _ in range(3):
            for s, c in zip(streams, outs):
                call(c, s)
        torch.cuda.synchronize()
        assert all(torch.equal(c, want) for c in outs)
        c = torch.zeros(M, N, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(c)
        a.copy_(rnd(M, K))
        call(want)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(c, want)


@pytest.mark.parametrize("M", [1, 3, 7, 40, 300])
def test_operands_written_just_before(M):
    """A product right behind the kernels that write its operands: its early
    start (set-up and requests into L2 overlap their end) must not see older
    values."""
    import torch
    import dense_fp32_matrix_03_gb300 as lib
    N, K, rounds = 512, 1024, 12
    gen = torch.Generator(device="cuda")
    gen.manual_seed(6)
    xs = torch.randn(rounds, M, K, device="cuda", generator=gen)
    ws = torch.randn(rounds, N, K, device="cuda", generator=gen)
    q = torch.zeros(M, K, dtype=torch.int8, device="cuda")
    wq = torch.zeros(N, K, dtype=torch.int8, device="cuda")
    s, sw = torch.zeros(M, device="cuda"), torch.zeros(N, device="cuda")
    c = torch.zeros(rounds, M, N, device="cuda")

    def call(i):
        lib.check(lib.sgemm_i8_quantize_rows("fp32", "none", N, K, ws[i], K, wq, K, sw))
        lib.check(lib.sgemm_i8_quantize_rows("fp32", "none", M, K, xs[i], K, q, K, s))
        lib.check(lib.sgemm_i8("fp32", M, N, K, q, K, s, wq, K, sw, c[i], N))

    for i in range(rounds):  # each alone
        call(i)
        torch.cuda.synchronize()
    want = c.clone()
    for _ in range(5):
        c.zero_()
        for i in range(rounds):
            call(i)
        torch.cuda.synchronize()
        assert torch.equal(c, want)


def test_experts_chain_written_just_before():
    """Sort, dispatch and product in one chain, over and over into the same
    buffers, as a decoding loop runs them."""
    import torch
    import dense_fp32_matrix_03_gb300 as lib
    T, k, E, N, K, rounds = 24, 3, 8, 256, 512, 20
    gen = torch.Generator(device="cuda")
    gen.manual_seed(7)
    ids = torch.randint(-1, E, (rounds, T, k), device="cuda", dtype=torch.int32, generator=gen)
    xs = torch.randn(rounds, T, K, device="cuda", generator=gen)
    w = torch.randint(-127, 128, (E, N, K), device="cuda", dtype=torch.int8, generator=gen)
    sw = torch.rand(E, N, device="cuda", generator=gen)
    S = T * k
    i32 = dict(dtype=torch.int32, device="cuda")
    off, slots, pos = torch.empty(E + 1, **i32), torch.empty(S, **i32), torch.empty(S, **i32)
    q, s = torch.zeros(S, K, dtype=torch.int8, device="cuda"), torch.zeros(S, device="cuda")
    y, out = torch.zeros(S, N, device="cuda"), torch.zeros(rounds, T, N, device="cuda")
    wt = torch.rand(T, k, device="cuda", generator=gen)

    def call(i):
        lib.check(lib.sgemm_experts_sort(T, k, E, ids[i], off, slots, pos))
        lib.check(lib.sgemm_experts_dispatch_i8("fp32", T, k, E, K, xs[i], K, pos, off, q, K, s))
        lib.check(lib.sgemm_i8_experts("fp32", S, N, K, E, off, q, K, s, w, K, N * K, sw, y, N))
        lib.check(lib.sgemm_experts_combine("fp32", T, k, E, N, y, N, pos, off, wt, out[i], N))

    for i in range(rounds):
        call(i)
        torch.cuda.synchronize()
    want = out.clone()
    for _ in range(5):
        out.zero_()
        for i in range(rounds):
            call(i)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
