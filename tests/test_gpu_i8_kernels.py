"""Every kernel that runs an 8-bit product (include/int8_gemm.h), each made to
run (sgemm_i8_tune_force) and seen to have run (sgemm_i8_last_kernel), against
the fp64 oracle element by element: the rule that chooses among them may move
with sizes, so no test here leaves the choice to it but the ones about it.

Bound: u = half a unit in the last place of the result type (bf16 2^-8, fp16
2^-11, fp32 2^-24); the integer sum is exact in fp32 while sum|a||b| <= 2^24,
then scaled twice and rounded: (u + 3 * 2^-24) |ref|.  Beyond 2^24 the sums of
FEW, NARROW and WIDE may lose 5 * 2^-23 of the largest partial sum with each 16
values of k: the 16 products are cut two bits below fp32's last place of the
largest number in the addition (16 * 2^-25), the new sum at that place (2^-23).
DOTS and ANY_LAYOUT add 32-bit integers and round once (2^-24)."""
import numpy as np
import pytest

from oracle import expert_layer as ex
from test_gpu_i8 import U, codes, pitch, scales, tdtype

pytestmark = pytest.mark.gpu

TYPES = ["bf16", "fp16", "fp32"]
TILED = ["few", "narrow", "wide"]
INTEGER = ["dots", "any_layout"]


@pytest.fixture(scope="module", autouse=True)
def gpu_ready():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import dense_fp32_matrix_03_gb300 as lib
    lib.load()
    torch.cuda.init()
    yield
    lib.sgemm_i8_tune_force("auto")


@pytest.fixture
def forced():
    import dense_fp32_matrix_03_gb300 as lib

    def force(kernel):
        assert lib.sgemm_i8_tune_force(kernel) == lib.SGEMM_OK
    yield force
    lib.sgemm_i8_tune_force("auto")


def ran(kernel):
    import dense_fp32_matrix_03_gb300 as lib
    assert lib.sgemm_poll_error() == lib.SGEMM_OK
    assert lib.sgemm_i8_last_kernel() == lib.I8_KERNELS[kernel]


def tolerance(kernel, type_, K, ref, mag, raw):
    lost = 1 * 2.0 ** -24 if kernel in INTEGER else 5 * K / 16 * 2.0 ** -23
    return (U[type_] + 3 * 2.0 ** -24) * np.abs(ref) + np.where(raw > 2.0 ** 24, lost * mag, 0) + \
        2.0 ** -24


def dense(kernel, type_, M, N, K, ldc_pad=0, c_off=0, values=None, seed=0):
    import torch
    import dense_fp32_matrix_03_gb300 as lib
    rng = np.random.default_rng(seed + M + N + K)
    ld = pitch(K, "pad16")
    da, pa, a = codes((M, K), ld, rng)
    db, pb, b = codes((N, K), ld, rng)
    if values is not None:  # constant operands
        a[:], b[:] = values
        for d, x, n in ((da, a, M), (db, b, N)):
            d[:-1].view(n, ld)[:, :K] = torch.from_numpy(x).cuda()
    sa, sb = scales(M, rng, K), scales(N, rng, K)
    ldc = N + ldc_pad
    c = torch.full((c_off + M * ldc,), 7.0, dtype=tdtype(type_), device="cuda")
    assert lib.sgemm_i8(type_, M, N, K, pa, ld, torch.from_numpy(sa).cuda(), pb, ld,
                        torch.from_numpy(sb).cuda(), c.data_ptr() + c_off * c.element_size(),
                        ldc) == lib.SGEMM_OK
    ran(kernel)
    got = c.double().cpu().numpy()
    assert (got[:c_off] == 7).all()
    got = got[c_off:].reshape(M, ldc)
    assert (got[:, N:] == 7).all(), "columns past N were written"
    ref, mag, raw = ex.product(a, sa, b, sb)
    err = np.abs(got[:, :N] - ref)
    assert np.all(err <= tolerance(kernel, type_, K, ref, mag, raw)), \
        float(np.max(err / (mag + 1e-30)))


# one slot of k to 33, so that every ring wraps; full and ragged tiles; every
# form of the few-token kernel
@pytest.mark.parametrize("type_", TYPES)
@pytest.mark.parametrize("M,N,K", [
    (1, 64, 16), (5, 300, 1000), (7, 300, 2100), (12, 300, 2100), (16, 31, 333), (33, 257, 2100),
    (60, 300, 4200), (64, 130, 129), (129, 384, 640), (257, 300, 4200), (300, 520, 777),
    (513, 1030, 300)])
@pytest.mark.parametrize("kernel", TILED + ["any_layout"])
def test_shapes(forced, kernel, type_, M, N, K):
    forced(kernel)
    dense(kernel, type_, M, N, K)


@pytest.mark.parametrize("type_", TYPES)
@pytest.mark.parametrize("M,N,K", [(1, 300, 5000), (2, 257, 333), (3, 130, 2100), (4, 31, 16)])
def test_shapes_of_the_integer_dots(forced, type_, M, N, K):
    forced("dots")
    dense("dots", type_, M, N, K)


@pytest.mark.parametrize("type_", TYPES)
@pytest.mark.parametrize("M,N,K", [(2500, 2500, 1000), (2337, 2563, 130)])
@pytest.mark.parametrize("kernel", ["narrow", "wide"])
def test_several_tiles_a_cta(forced, kernel, type_, M, N, K):
    """More tiles than multiprocessors (pairs of them), several slots each: the
    rings and accumulators go on from one tile to the next."""
    import torch
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    edge = 128 if kernel == "narrow" else 256
    assert -(-M // edge) * -(-N // edge) > sms / (edge // 128)
    forced(kernel)
    dense(kernel, type_, M, N, K)


@pytest.mark.parametrize("K,split", [(300, 1), (640, 2), (1100, 4), (2100, 8), (9000, 8)])
@pytest.mark.parametrize("type_,pad", [("bf16", 0), ("fp16", 3), ("fp32", 0), ("fp32", 1)])
def test_shared_k(forced, type_, pad, K, split):
    """Clusters of every size share a tile's k."""
    import dense_fp32_matrix_03_gb300 as lib
    forced("narrow")
    for M in (3, 40, 128):
        dense("narrow", type_, M, 130, K, ldc_pad=pad)
        assert lib.sgemm_i8_last_split_count() == split


# rows of results on 16, 8 and fewer bytes, inside a larger matrix
@pytest.mark.parametrize("type_", TYPES)
@pytest.mark.parametrize("ldc_pad,c_off", [(0, 0), (8, 0), (4, 4), (1, 0), (0, 1), (3, 2)])
@pytest.mark.parametrize("kernel", TILED)
def test_result_pitches(forced, kernel, type_, ldc_pad, c_off):
    forced(kernel)
    for M, N, K in ((75, 264, 200), (300, 520, 140), (290, 519, 400)):
        dense(kernel, type_, M, N, K, ldc_pad=ldc_pad, c_off=c_off)


@pytest.mark.parametrize("kernel", TILED)
@pytest.mark.parametrize("values", [(127, 127), (127, -97), (101, 119), (-128, -128)])
@pytest.mark.parametrize("K", [1024, 9000, 16384])
def test_long_sums_of_one_sign(forced, kernel, values, K):
    """Partial sums that grow all the way; 127 * 97 = 31 modulo 32 loses most
    where products are cut."""
    forced(kernel)
    dense(kernel, "fp32", 64, 256, K, values=values)


@pytest.mark.parametrize("kernel", TILED + ["any_layout"])
@pytest.mark.parametrize("values", [None, (127, 97)])
def test_longest_sums(forced, kernel, values):
    forced(kernel)
    dense(kernel, "fp32", 40, 70, 131071, values=values)


@pytest.mark.parametrize("kernel", TILED + INTEGER)
def test_the_last_exact_sum(forced, kernel):
    """-128 * -128 * 1024 = 2^24, and 2^24 - 129 beside it, to the bit."""
    import torch
    import dense_fp32_matrix_03_gb300 as lib
    M = 4 if kernel == "dots" else 300
    a = torch.full((M, 1040), -128, dtype=torch.int8, device="cuda")
    a[:, 1024:] = 0
    b = torch.full((256, 1040), -128, dtype=torch.int8, device="cuda")
    a[1, 0], a[1, 1024], b[:, 1024] = -127, 1, -1
    one = torch.ones(max(M, 256), device="cuda")
    c = torch.zeros(M, 256, device="cuda")
    forced(kernel)
    assert lib.sgemm_i8("fp32", M, 256, 1040, a, 1040, one, b, 1040, one, c, 256) == 0
    ran(kernel)
    assert bool((c[0] == 2.0 ** 24).all() and (c[2:] == 2.0 ** 24).all())
    assert bool((c[1] == 2.0 ** 24 - 129).all())


@pytest.mark.parametrize("type_", TYPES)
@pytest.mark.parametrize("kernel", TILED + INTEGER)
def test_nan_and_infinite_scales_stay_in_their_row_and_column(forced, kernel, type_):
    import torch
    import dense_fp32_matrix_03_gb300 as lib
    M, N, K = (4 if kernel == "dots" else 300), 300, 400
    a = torch.ones(M, K, dtype=torch.int8, device="cuda")
    b = torch.ones(N, K, dtype=torch.int8, device="cuda")
    sa, sb = torch.ones(M, device="cuda"), torch.ones(N, device="cuda")
    sa[2], sb[-1], sb[17] = float("nan"), float("nan"), float("inf")
    c = torch.zeros(M, N, dtype=tdtype(type_), device="cuda")
    forced(kernel)
    assert lib.sgemm_i8(type_, M, N, K, a, K, sa, b, K, sb, c, N) == lib.SGEMM_OK
    ran(kernel)
    c = c.float()
    assert bool(torch.isnan(c[2]).all() and torch.isnan(c[:, -1]).all())
    keep = [i for i in range(M) if i != 2]
    assert bool(torch.isinf(c[keep, 17]).all())
    cols = [j for j in range(N - 1) if j != 17]
    assert bool((c[keep][:, cols] == 400).all())


def experts(kernel, type_, counts, N, K, tail=0, ldc_pad=0, seed=1):
    import torch
    import dense_fp32_matrix_03_gb300 as lib
    rng = np.random.default_rng(seed + N + K)
    E, M = len(counts), sum(counts) + tail
    ld = pitch(K, "pad16")
    da, pa, a = codes((M, K), ld, rng)
    db, pb, b = codes((E, N, K), ld, rng)
    sa, sb = scales(M, rng, K), scales((E, N), rng, K)
    sa[M - tail:] = np.nan
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    ldc = N + ldc_pad
    c = torch.full((M, ldc), 7.0, dtype=tdtype(type_), device="cuda")
    assert lib.sgemm_i8_experts(type_, M, N, K, E, torch.from_numpy(off).cuda(), pa, ld,
                                torch.from_numpy(sa).cuda(), pb, ld, N * ld,
                                torch.from_numpy(sb).cuda(), c, ldc) == lib.SGEMM_OK
    ran(kernel)
    got = c.double().cpu().numpy()
    assert (got[M - tail:] == 7).all(), "rows past the last expert were written"
    assert (got[:, N:] == 7).all(), "columns past N were written"
    live = slice(0, M - tail)
    ref, mag, raw = (x[live] for x in ex.product_experts(off, a, np.nan_to_num(sa), b, sb, N))
    err = np.abs(got[live, :N] - ref)
    assert np.all(err <= tolerance(kernel, type_, K, ref, mag, raw)), \
        float(np.max(err / (mag + 1e-30)))


# empty experts, single rows, tiles that end inside an expert, rows past the last
@pytest.mark.parametrize("type_", TYPES)
@pytest.mark.parametrize("counts,N,K,tail,pad", [
    ([1], 64, 64, 0, 0), ([0, 3, 0, 0, 5], 130, 200, 2, 1), ([1, 0, 130, 17, 64, 0, 65, 3], 300, 333, 5, 4),
    ([300, 0, 1, 257, 256, 0], 512, 700, 3, 0), ([0, 0, 0], 128, 128, 4, 0),
    ([1000, 2, 0, 31], 385, 2100, 1, 0), ([5] * 100, 70, 96, 3, 2), ([700, 90, 513], 1100, 500, 9, 0)])
@pytest.mark.parametrize("kernel", TILED + ["any_layout"])
def test_experts(forced, kernel, type_, counts, N, K, tail, pad):
    forced(kernel)
    experts(kernel, type_, counts, N, K, tail, pad)


@pytest.mark.parametrize("kernel", TILED)
def test_one_expert_has_every_row(forced, kernel):
    forced(kernel)
    experts(kernel, "bf16", [0] * 40 + [1000] + [0] * 23, 200, 300, 24)


@pytest.mark.parametrize("kernel", TILED + ["any_layout"])
def test_rows_past_the_last_expert_reach_nothing(forced, kernel):
    """Bit for bit the same results whatever codes and scales stand there."""
    import torch
    import dense_fp32_matrix_03_gb300 as lib
    N, K, tail = 200, 300, 60
    gen = torch.Generator(device="cuda")
    gen.manual_seed(10)
    rnd = lambda *s: torch.randint(-128, 128, s, device="cuda", dtype=torch.int8, generator=gen)
    for counts in ([1], [33, 65], [256, 0, 129]):
        E, M = len(counts), sum(counts) + tail
        off = torch.tensor([0, *np.cumsum(counts)], dtype=torch.int32, device="cuda")
        a, b, ld = rnd(M, 304), rnd(E, N, 304), 304
        sa, sb = torch.rand(M, device="cuda", generator=gen), torch.ones(E, N, device="cuda")
        forced(kernel)
        results = []
        for code, scale in ((-128, float("nan")), (127, float("inf")), (0, 1.0)):
            a[M - tail:], sa[M - tail:] = code, scale
            c = torch.full((M, N), 7.0, device="cuda")
            assert lib.sgemm_i8_experts("fp32", M, N, K, E, off, a, ld, sa, b, ld, N * ld, sb, c,
                                        N) == lib.SGEMM_OK
            ran(kernel)
            assert bool((c[M - tail:] == 7).all())
            results.append(c)
        assert torch.equal(results[0], results[1]) and torch.equal(results[0], results[2])


@pytest.mark.parametrize("K", [64, 1104])
@pytest.mark.parametrize("kernel,tm", [("few", 8), ("narrow", 128), ("wide", 256),
                                       ("any_layout", 64)])
def test_offsets_that_descend(forced, kernel, tm, K):
    """Experts 0, 2, 4 and 6 have all rows, the others none.  Every kernel works
    off as many tiles as ascending offsets can need, in the experts' order, and
    leaves out the rest: a row holds one of these experts' whole results."""
    import torch
    import dense_fp32_matrix_03_gb300 as lib
    E, M, N = 8, 1024, 128
    a = torch.ones(M, K, dtype=torch.int8, device="cuda")
    b = torch.arange(1, E + 1, dtype=torch.int8, device="cuda")[:, None, None].repeat(1, N, K)
    one = torch.ones(max(M, E * N), device="cuda")
    pad = 4096
    c = torch.full((M * N + 2 * pad,), 7.0, device="cuda")
    off = torch.tensor([0, M] * (E // 2) + [0], dtype=torch.int32, device="cuda")
    forced(kernel)
    assert lib.sgemm_i8_experts("fp32", M, N, K, E, off, a, K, one, b, K, N * K, one,
                                c.data_ptr() + pad * 4, N) == lib.SGEMM_OK
    ran(kernel)
    assert bool((c[:pad] == 7).all() and (c[pad + M * N:] == 7).all())
    worked = [e for i, e in enumerate(range(0, E, 2)) if i * (M // tm) < M // tm + E]
    allowed = torch.tensor([K * (e + 1.0) for e in worked], device="cuda")
    rows = c[pad:pad + M * N].view(M, N)
    assert bool((rows[:, :, None] == allowed).any(2).all())


@pytest.mark.parametrize("kernel", TILED)
def test_weights_beyond_32_bit_offsets(forced, kernel):
    """Experts' weights of more than 2^31 bytes; results checked in the last."""
    import torch
    import dense_fp32_matrix_03_gb300 as lib
    E, N, K, M = 70, 8192, 4096, 300
    b = torch.zeros(E, N, K, dtype=torch.int8, device="cuda")
    gen = torch.Generator(device="cuda")
    gen.manual_seed(4)
    rnd = lambda *s: torch.randint(-128, 128, s, device="cuda", dtype=torch.int8, generator=gen)
    b[-1] = rnd(N, K)
    a = rnd(M, K)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[-1] = M
    one = torch.ones(E * N, device="cuda")
    c = torch.zeros(M, N, device="cuda")
    forced(kernel)
    assert lib.sgemm_i8_experts("fp32", M, N, K, E, off, a, K, one, b, K, N * K, one, c, N) == 0
    ran(kernel)
    ref = a.double() @ b[-1].double().t()
    mag = a.double().abs() @ b[-1].double().abs().t()
    assert bool(((c - ref).abs() <= 2.0 ** -24 * ref.abs() + 5 * K / 16 * 2.0 ** -23 * mag).all())


@pytest.mark.parametrize("kernel,M", [("dots", 3), ("few", 40), ("few", 300), ("narrow", 40),
                                      ("narrow", 300), ("wide", 40), ("wide", 300),
                                      ("any_layout", 40)])
def test_operands_written_just_before(forced, kernel, M):
    """Bit for bit what the call gives alone, right behind the kernels that
    write both operands, over and over into the same buffers."""
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
    forced(kernel)

    def call(i):
        lib.check(lib.sgemm_i8_quantize_rows("fp32", "none", N, K, ws[i], K, wq, K, sw))
        lib.check(lib.sgemm_i8_quantize_rows("fp32", "none", M, K, xs[i], K, q, K, s))
        lib.check(lib.sgemm_i8("fp32", M, N, K, q, K, s, wq, K, sw, c[i], N))

    for i in range(rounds):
        call(i)
        torch.cuda.synchronize()
    ran(kernel)
    want = c.clone()
    assert not torch.equal(want[0], want[1])
    for _ in range(5):
        c.zero_()
        for i in range(rounds):
            call(i)
        torch.cuda.synchronize()
        assert torch.equal(c, want)


@pytest.mark.parametrize("kernel", TILED)
def test_experts_chain_written_just_before(forced, kernel):
    """Sort, dispatch in 8 bits, product, combine, each written just before
    the next reads it."""
    import torch
    import dense_fp32_matrix_03_gb300 as lib
    T, k, E, N, K, rounds = 200, 3, 8, 256, 512, 10
    gen = torch.Generator(device="cuda")
    gen.manual_seed(7)
    ids = torch.randint(-1, E, (rounds, T, k), device="cuda", dtype=torch.int32, generator=gen)
    xs = torch.randn(rounds, T, K, device="cuda", generator=gen)
    w = torch.randint(-127, 128, (E, N, K), device="cuda", dtype=torch.int8, generator=gen)
    sw = torch.rand(E, N, device="cuda", generator=gen)
    S = T * k
    i32 = dict(dtype=torch.int32, device="cuda")
    now = torch.empty(T, k, **i32)
    off, slots, pos = torch.empty(E + 1, **i32), torch.empty(S, **i32), torch.empty(S, **i32)
    q, s = torch.zeros(S, K, dtype=torch.int8, device="cuda"), torch.zeros(S, device="cuda")
    y, out = torch.zeros(S, N, device="cuda"), torch.zeros(rounds, T, N, device="cuda")
    wt = torch.rand(T, k, device="cuda", generator=gen)
    forced(kernel)

    def call(i):
        now.copy_(ids[i])
        lib.check(lib.sgemm_experts_sort(T, k, E, now, off, slots, pos))
        lib.check(lib.sgemm_experts_dispatch_i8("fp32", T, k, E, K, xs[i], K, pos, off, q, K, s))
        lib.check(lib.sgemm_i8_experts("fp32", S, N, K, E, off, q, K, s, w, K, N * K, sw, y, N))
        lib.check(lib.sgemm_experts_combine("fp32", T, k, E, N, y, N, pos, off, wt, out[i], N))

    for i in range(rounds):
        call(i)
        torch.cuda.synchronize()
    ran(kernel)
    want = out.clone()
    for _ in range(5):
        out.zero_()
        for i in range(rounds):
            call(i)
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_a_kernel_that_cannot_take_a_call_leaves_it_to_the_rule(forced):
    forced("dots")
    dense("few", "bf16", 5, 64, 64)
    forced("wide")
    import torch
    import dense_fp32_matrix_03_gb300 as lib
    a = torch.ones(4, 33, dtype=torch.int8, device="cuda")  # rows off 16 bytes
    one, c = torch.ones(4, device="cuda"), torch.zeros(4, 4, device="cuda")
    assert lib.sgemm_i8("fp32", 4, 4, 33, a, 33, one, a, 33, one, c, 4) == lib.SGEMM_OK
    ran("any_layout")
    assert bool((c == 33).all())


# the rule, at sizes well inside each kernel's range; results at sampled rows
@pytest.mark.parametrize("type_", TYPES)
@pytest.mark.parametrize("M,N,K,want", [
    (1, 4096, 4096, "dots"), (4, 2048, 1024, "dots"), (16, 4096, 4096, "few"),
    (64, 1024, 4096, "few"), (256, 4096, 4096, "narrow"), (1000, 1500, 777, "narrow"),
    (8192, 8192, 4096, "wide"), (4096, 4096, 1000, "wide")])
def test_rule_dense(type_, M, N, K, want):
    import torch
    import dense_fp32_matrix_03_gb300 as lib
    gen = torch.Generator(device="cuda")
    gen.manual_seed(8)
    ld = pitch(K, "pad16")
    rnd = lambda r: torch.randint(-128, 128, (r, ld), device="cuda", dtype=torch.int8, generator=gen)
    a, b = rnd(M), rnd(N)
    sa, sb = (torch.rand(r, device="cuda", generator=gen) / 1000 for r in (M, N))
    c = torch.full((M, N), 7.0, dtype=tdtype(type_), device="cuda")
    assert lib.sgemm_i8(type_, M, N, K, a, ld, sa, b, ld, sb, c, N) == lib.SGEMM_OK
    ran(want)
    at = torch.unique(torch.randint(0, M, (64,), device="cuda", generator=gen))
    x, w = a[at, :K].double(), b[:, :K].double()
    s = sa[at].double()[:, None] * sb.double()[None, :]
    raw = (x.abs() @ w.abs().t()).cpu().numpy()
    ref, mag = ((x @ w.t()) * s).cpu().numpy(), raw * s.cpu().numpy()
    err = np.abs(c[at].double().cpu().numpy() - ref)
    assert np.all(err <= tolerance(want, type_, K, ref, mag, raw))


@pytest.mark.parametrize("rows,K,want", [(8, 2048, "few"), (60, 256, "narrow"),
                                         (1024, 2048, "wide")])
def test_rule_experts(rows, K, want):
    import torch
    import dense_fp32_matrix_03_gb300 as lib
    E, N = 32, 4096
    gen = torch.Generator(device="cuda")
    gen.manual_seed(9)
    M = E * rows
    rnd = lambda *s: torch.randint(-128, 128, s, device="cuda", dtype=torch.int8, generator=gen)
    a, b = rnd(M, K), rnd(E, N, K)
    sa, sb = torch.rand(M, device="cuda", generator=gen), torch.rand(E, N, device="cuda", generator=gen)
    cuts = torch.sort(torch.randint(0, M + 1, (E - 1,), device="cuda", generator=gen))[0]
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[1:E], off[E] = cuts.int(), M
    c = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda")
    assert lib.sgemm_i8_experts("bf16", M, N, K, E, off, a, K, sa, b, K, N * K, sb, c, N) == 0
    ran(want)
    first = off.tolist()
    for e in range(E):
        rows_e = [r for r in (first[e], (first[e] + first[e + 1]) // 2, first[e + 1] - 1)
                  if first[e] <= r < first[e + 1]]
        if not rows_e:
            continue
        x, w = a[rows_e].double(), b[e].double()
        s = sa[rows_e].double()[:, None] * sb[e].double()[None, :]
        ref, raw = ((x @ w.t()) * s).cpu().numpy(), (x.abs() @ w.abs().t()).cpu().numpy()
        err = np.abs(c[rows_e].double().cpu().numpy() - ref)
        assert np.all(err <= tolerance(want, "bf16", K, ref, raw * s.cpu().numpy(), raw)), e
