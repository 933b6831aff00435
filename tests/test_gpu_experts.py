"""GPU parity of the expert layer's row operators (include/expert_layer.h) and
of the row quantiser (include/int8_gemm.h) against the fp64 oracle
(oracle/expert_layer.py), element by element, through the C ABI.

Bounds, derived from the arithmetic: u = half a unit in the last place of the
row type (bf16 2^-8, fp16 2^-11, fp32 2^-24), e = 2^-24 per fp32 operation.
  dispatch   a copy: bit for bit
  combine    u |ref| + (k + 1) e sum|w r|          (k fma, one rounding)
  drows      (u + e) |ref|
  dw         (H / 32 + 16) e sum|r g|              (at least 32 partial sums)
  codes      |q - x 127 / a| <= 1/2 + 127 * 2^-23  (two fp32 operations)
plus the smallest fp16 subnormal where results can underflow."""
import numpy as np
import pytest

from oracle import expert_layer as ex

pytestmark = pytest.mark.gpu

U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
E24 = 2.0 ** -24
SUB = 2.0 ** -24
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


class Rows:
    """A device matrix of R x H values with a padded pitch and an offset
    base; pad holds NaN, so that a read of it shows and a write does too."""

    def __init__(self, R, H, type_, pad=0, offset=0, values=None):
        import torch
        self.R, self.H, self.ld = R, H, max(H + pad, 1)
        self.buf = torch.full((offset + max(R * self.ld, 1),), float("nan"),
                              dtype=tdtype(type_), device="cuda")
        self.off = offset
        self.view = self.buf[offset:offset + R * self.ld].view(R, self.ld)[:, :H]
        if values is not None:
            self.view.copy_(torch.from_numpy(values).to(tdtype(type_)))

    @property
    def ptr(self):
        return self.buf.data_ptr() + self.off * self.buf.element_size()

    def np(self):
        return self.view.double().cpu().numpy()

    def pad_untouched(self):
        import torch
        whole = self.buf[self.off:self.off + self.R * self.ld].view(self.R, self.ld)
        return bool(torch.isnan(whole[:, self.H:].float()).all()) and \
            bool(torch.isnan(self.buf[:self.off].float()).all())


def ints(n, fill=-7):
    import torch
    return torch.full((max(n, 1),), fill, dtype=torch.int32, device="cuda")


def run_sort(ids, E):
    import torch
    import dense_fp32_matrix_03_gb300 as lib
    T, k = ids.shape
    d = torch.from_numpy(ids.astype(np.int32)).cuda()
    offsets, slots, positions = ints(E + 1), ints(T * k), ints(T * k)
    assert lib.sgemm_experts_sort(T, k, E, d, offsets, slots, positions) == lib.SGEMM_OK
    return offsets, slots, positions


def make_ids(T, k, E, rng, drop=0.25, skew=True):
    if skew:
        p = rng.random(E) ** 3 + 1e-3
        ids = rng.choice(E, size=(T, k), p=p / p.sum())
    else:
        ids = rng.integers(0, E, (T, k))
    gone = rng.random((T, k)) < drop
    return np.where(gone, rng.choice([-1, E, E + 5, -2 ** 31, 2 ** 31 - 1], (T, k)), ids)


@pytest.mark.parametrize("T,k,E,drop", [
    (1, 1, 1, 0.0), (1, 1, 1, 1.0), (3, 5, 2, 0.3), (33, 1, 7, 0.0), (8, 4, 32, 0.0),
    (31, 64, 1024, 0.2), (1365, 3, 60, 0.1), (1366, 3, 60, 0.1), (4097, 1, 1, 0.5),
    (2500, 2, 1023, 0.0), (20000, 8, 64, 0.05), (70001, 3, 128, 0.3), (5000, 1, 16, 1.0)])
def test_sort(T, k, E, drop):
    rng = np.random.default_rng(T + k)
    ids = make_ids(T, k, E, rng, drop)
    got = [x.cpu().numpy() for x in run_sort(ids, E)]
    for g, want in zip(got, ex.sort(ids, E)):
        assert np.array_equal(g, want)


def test_sort_of_nothing():
    import dense_fp32_matrix_03_gb300 as lib
    offsets = ints(6)
    assert lib.sgemm_experts_sort(0, 4, 5, None, offsets, None, None) == lib.SGEMM_OK
    assert not offsets.cpu().numpy().any()


# T, k, E, H, pad, offset: rows on 16-byte boundaries and off them, shorter
# than a warp's vectors and longer than a block's, more choices than move at once
SHAPES = [(1, 1, 1, 1, 0, 0), (5, 2, 3, 7, 0, 0), (16, 4, 32, 2048, 0, 0), (3, 8, 8, 64, 0, 0),
          (9, 3, 4, 333, 0, 1), (17, 9, 12, 96, 8, 8), (130, 2, 5, 1500, 4, 4), (6, 17, 20, 40, 0, 2),
          (4, 3, 2, 9000, 24, 0), (2, 64, 100, 10, 1, 0), (40, 5, 6, 2825, 0, 0), (12, 2, 3, 641, 3, 5),
          (7, 2, 4, 17, 0, 3), (300, 4, 6, 1123, 0, 0)]


@pytest.mark.parametrize("type_", TYPES)
@pytest.mark.parametrize("T,k,E,H,pad,offset", SHAPES)
def test_rows_there_and_back(type_, T, k, E, H, pad, offset):
    import torch
    import dense_fp32_matrix_03_gb300 as lib
    rng = np.random.default_rng(H)
    ids = make_ids(T, k, E, rng)
    if T > 2:
        ids[1] = -1  # a token without a choice
    offsets, _, positions = run_sort(ids, E)
    ro, _, rp = ex.sort(ids, E)
    total = int(ro[-1])
    R = T * k
    x = Rows(T, H, type_, pad, offset, rng.standard_normal((T, H)))
    g = Rows(T, H, type_, pad, 0, rng.standard_normal((T, H)))
    rv = rng.standard_normal((R, H))
    rv[total:] = np.nan  # never read
    if R > total:
        rv[total:, ::2] = np.inf
    rows = Rows(R, H, type_, pad, offset, rv)
    w = rng.random((T, k)).astype(np.float32)
    w.reshape(-1)[rp >= total] = np.nan  # never used
    dw_ = torch.from_numpy(w).cuda()
    u = U[type_]

    out = Rows(R, H, type_, pad, offset)
    assert lib.sgemm_experts_dispatch(type_, T, k, E, H, x.ptr, x.ld, positions, offsets, out.ptr,
                                      out.ld) == lib.SGEMM_OK
    assert np.array_equal(out.np(), ex.dispatch(x.np(), rp, total, k))
    assert out.pad_untouched()

    for weights in (dw_, None):
        out = Rows(T, H, type_, pad, offset)
        assert lib.sgemm_experts_combine(type_, T, k, E, H, rows.ptr, rows.ld, positions, offsets,
                                         weights, out.ptr, out.ld) == lib.SGEMM_OK
        ref, mag = ex.combine(rows.np(), rp, total, None if weights is None else w, T, k)
        assert np.all(np.abs(out.np() - ref) <= u * np.abs(ref) + (k + 1) * E24 * mag + SUB)
        assert out.pad_untouched()
    if T > 2:
        assert not out.np()[1].any()

    out = Rows(T, H, type_, pad, offset)
    assert lib.sgemm_experts_dispatch_grad(type_, T, k, E, H, rows.ptr, rows.ld, positions,
                                           offsets, out.ptr, out.ld) == lib.SGEMM_OK
    ref, mag = ex.dispatch_grad(rows.np(), rp, total, T, k)
    assert np.all(np.abs(out.np() - ref) <= u * np.abs(ref) + (k + 1) * E24 * mag + SUB)

    ref, dwref, mag = ex.combine_grad(g.np(), rows.np(), rp, total, w, k)
    for want_dw in (True, False):
        out = Rows(R, H, type_, pad, offset)
        dw = torch.full((T, k), float("nan"), device="cuda")
        assert lib.sgemm_experts_combine_grad(
            type_, T, k, E, H, g.ptr, g.ld, rows.ptr if want_dw else None, rows.ld, positions,
            offsets, dw_, out.ptr, out.ld, dw if want_dw else None) == lib.SGEMM_OK
        assert np.all(np.abs(out.np() - ref) <= (u + E24) * np.abs(ref) + SUB)
        assert out.pad_untouched()
        if want_dw:
            assert np.all(np.abs(dw.double().cpu().numpy() - dwref) <= (H / 32 + 16) * E24 * mag)
    # weights NULL: every drow is its token's row
    out = Rows(R, H, type_, pad, offset)
    assert lib.sgemm_experts_combine_grad(type_, T, k, E, H, g.ptr, g.ld, None, 1, positions,
                                          offsets, None, out.ptr, out.ld, None) == lib.SGEMM_OK
    assert np.array_equal(out.np(), ex.dispatch(g.np(), rp, total, k))


@pytest.mark.parametrize("type_", TYPES)
def test_gradient_is_the_difference_quotient(type_):
    """combine is linear in rows and in weights: for a step d of either,
    <g, combine(x + d) - combine(x)> = <gradient, d>, up to the roundings of
    the three calls (values are small integers, so in fp32 they are exact)."""
    import torch
    import dense_fp32_matrix_03_gb300 as lib
    T, k, E, H = 6, 3, 4, 32
    rng = np.random.default_rng(9)
    ids = make_ids(T, k, E, rng)
    offsets, _, positions = run_sort(ids, E)
    val = lambda *s: rng.integers(-3, 4, s).astype(np.float64)
    rows, step = val(T * k, H), val(T * k, H)
    g, w, wstep = val(T, H), val(T, k).astype(np.float32), val(T, k).astype(np.float32)

    def combined(rows, w):
        r, out = Rows(T * k, H, type_, values=rows), Rows(T, H, type_)
        assert lib.sgemm_experts_combine(type_, T, k, E, H, r.ptr, H, positions, offsets,
                                         torch.from_numpy(w).cuda(), out.ptr, H) == lib.SGEMM_OK
        return out.np()

    G, r, dr = Rows(T, H, type_, values=g), Rows(T * k, H, type_, values=rows), Rows(T * k, H, type_)
    dw = torch.zeros(T, k, device="cuda")
    assert lib.sgemm_experts_combine_grad(type_, T, k, E, H, G.ptr, H, r.ptr, H, positions,
                                          offsets, torch.from_numpy(w).cuda(), dr.ptr, H,
                                          dw) == lib.SGEMM_OK
    base = combined(rows, w)
    # |out| <= 3 * 3 * 6 = 54: integers up to 256 are exact in every type
    assert np.sum(g * (combined(rows + step, w) - base)) == np.sum(dr.np() * step)
    assert np.sum(g * (combined(rows, w + wstep) - base)) == \
        np.sum(dw.double().cpu().numpy() * wstep)


@pytest.mark.parametrize("T,k,E,H", [(5, 2, 3, 0), (0, 2, 3, 8)])
def test_empty_rows(T, k, E, H):
    import torch
    import dense_fp32_matrix_03_gb300 as lib
    ids = np.zeros((T, k), np.int64)
    offsets, _, positions = run_sort(ids, E) if T else (ints(E + 1, 0), None, ints(1))
    dw = torch.full((max(T, 1), k), 3.0, device="cuda")
    sc = torch.full((max(T * k, 1),), 3.0, device="cuda")
    ld = max(H, 1)
    assert lib.sgemm_experts_dispatch("bf16", T, k, E, H, None, ld, positions, offsets, None,
                                      ld) == lib.SGEMM_OK
    assert lib.sgemm_experts_combine("bf16", T, k, E, H, None, ld, positions, offsets, None, None,
                                     ld) == lib.SGEMM_OK
    assert lib.sgemm_experts_combine_grad("bf16", T, k, E, H, None, ld, None, ld, positions,
                                          offsets, None, None, ld, dw) == lib.SGEMM_OK
    assert lib.sgemm_experts_dispatch_i8("bf16", T, k, E, H, None, ld, positions, offsets, None,
                                         ld, sc) == lib.SGEMM_OK
    want = 0.0 if T else 3.0
    assert bool((dw == want).all()) and bool((sc == want).all())


def check_codes(q, s, x, slack=127 * 2.0 ** -23, scale_err=2.0 ** -23):
    y, sref = ex.quantize(x)
    bad = np.isnan(sref)
    assert np.array_equal(np.isnan(s), bad)
    assert np.all(np.abs(s[~bad] - sref[~bad]) <= scale_err * sref[~bad])
    assert np.all(np.abs(q[~bad] - y[~bad]) <= 0.5 + slack)
    assert not q[bad].any()


@pytest.mark.parametrize("type_", TYPES)
@pytest.mark.parametrize("M,K,pad,offset,qpad", [
    (1, 1, 0, 0, 0), (3, 7, 0, 0, 0), (70, 64, 0, 0, 0), (5, 333, 1, 1, 3), (9, 1500, 4, 0, 4),
    (2, 4096, 0, 8, 0), (37, 4092, 0, 0, 4), (3, 20000, 0, 0, 0), (300, 40, 0, 2, 9),
    (2, 4095, 0, 0, 1), (40, 2002, 0, 0, 14), (6, 2001, 2, 1, 15), (5, 5, 0, 0, 3)])
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_quantize_rows(type_, M, K, pad, offset, qpad, act):
    import torch
    import dense_fp32_matrix_03_gb300 as lib
    rng = np.random.default_rng(K)
    width = 2 * K if act == "swiglu" else K
    v = rng.standard_normal((M, width)) * np.exp(rng.standard_normal((M, 1)))
    special = M > 4
    if special:
        v[1] = 0
        v[2, K // 2] = np.inf
        v[3, width - 1] = np.nan
        v[4] *= 1e-3
    x = Rows(M, width, type_, pad, offset, v)
    q = torch.full((M, K + qpad), 77, dtype=torch.int8, device="cuda")
    s = torch.full((M,), -1.0, device="cuda")
    assert lib.sgemm_i8_quantize_rows(type_, act, M, K, x.ptr, x.ld, q, K + qpad, s) == \
        lib.SGEMM_OK
    got, scale = q[:, :K].cpu().numpy().astype(np.float64), s.double().cpu().numpy()
    assert bool((q[:, K:] == 77).all())
    if act == "none":
        check_codes(got, scale, x.np())
    else:
        # silu in fp32: exp within 2 units, a sum, a quotient and a product:
        # each value and the row's maximum within 8 * 2^-23 of exact
        with np.errstate(invalid="ignore"):
            h = ex.gated(x.np())
        check_codes(got, scale, h, slack=127 * 18 * 2.0 ** -23, scale_err=10 * 2.0 ** -23)


def test_quantize_extremes():
    """Rows at the ends of fp32's range."""
    import torch
    import dense_fp32_matrix_03_gb300 as lib
    x = np.array([[3e38, -1e38, 0, 1], [2.0 ** -100, 2.0 ** -101, 0, 0],
                  [2.0 ** -101, -(2.0 ** -120), 0, 0], [1e-45, 0, 0, 0], [-5, 5, 2.5, -0.0]])
    X = torch.from_numpy(x.astype(np.float32)).cuda()
    q = torch.zeros(5, 4, dtype=torch.int8, device="cuda")
    s = torch.zeros(5, device="cuda")
    assert lib.sgemm_i8_quantize_rows("fp32", "none", 5, 4, X, 4, q, 4, s) == lib.SGEMM_OK
    check_codes(q.cpu().numpy().astype(np.float64), s.double().cpu().numpy(), X.double().cpu().numpy())
    assert q[4].tolist() == [-127, 127, 64, 0]  # 63.5 to even


@pytest.mark.parametrize("type_", TYPES)
@pytest.mark.parametrize("T,k,E,H,pad,offset", SHAPES)
def test_dispatch_i8(type_, T, k, E, H, pad, offset):
    """The codes and scales sgemm_i8_quantize_rows gives, in expert order."""
    import torch
    import dense_fp32_matrix_03_gb300 as lib
    rng = np.random.default_rng(H + 1)
    ids = make_ids(T, k, E, rng)
    offsets, _, positions = run_sort(ids, E)
    ro, _, rp = ex.sort(ids, E)
    total = int(ro[-1])
    v = rng.standard_normal((T, H))
    if T > 4:
        v[3, 0] = np.nan
    x = Rows(T, H, type_, pad, offset, v)
    ld = (H + 15) // 16 * 16
    q1 = torch.zeros(T, ld, dtype=torch.int8, device="cuda")
    s1 = torch.zeros(T, device="cuda")
    assert lib.sgemm_i8_quantize_rows(type_, "none", T, H, x.ptr, x.ld, q1, ld, s1) == lib.SGEMM_OK
    q = torch.full((T * k, ld), 77, dtype=torch.int8, device="cuda")
    s = torch.full((T * k,), -1.0, device="cuda")
    assert lib.sgemm_experts_dispatch_i8(type_, T, k, E, H, x.ptr, x.ld, positions, offsets, q, ld,
                                         s) == lib.SGEMM_OK
    q1, s1, q, s = (z.double().cpu().numpy() for z in (q1, s1, q, s))
    assert (q[:, H:] == 77).all()
    assert np.array_equal(q[:, :H], ex.dispatch(q1[:, :H], rp, total, k))
    want = ex.dispatch(s1[:, None], rp, total, k)[:, 0]
    assert np.array_equal(s, want, equal_nan=True)


def test_corrupt_positions_stay_inside():
    """Positions outside 0 .. T*k-1 are ignored, not followed."""
    import torch
    import dense_fp32_matrix_03_gb300 as lib
    T, k, E, H = 4, 2, 2, 16
    positions = torch.tensor([0, 1, 2, -5, 99, 2 ** 31 - 1, 6, 7], dtype=torch.int32, device="cuda")
    offsets = torch.tensor([0, 4, 1000], dtype=torch.int32, device="cuda")
    x = torch.arange(T * H, device="cuda", dtype=torch.float32).view(T, H)
    rows = torch.full((T * k, H), -1.0, device="cuda")
    assert lib.sgemm_experts_dispatch("fp32", T, k, E, H, x, H, positions, offsets, rows, H) == 0
    assert bool((rows[0] == x[0]).all() and (rows[1] == x[0]).all() and (rows[2] == x[1]).all())
    assert bool((rows[3:6] == -1).all() and (rows[6] == x[3]).all())
    out = torch.zeros(T, H, device="cuda")
    assert lib.sgemm_experts_combine("fp32", T, k, E, H, rows, H, positions, offsets, None, out,
                                     H) == 0
    assert bool((out[2] == 0).all() and (out[1] == x[1]).all())


def test_rows_beyond_32_bit_offsets():
    """70000 rows of 32768 bf16 values: element offsets pass 2^31."""
    import torch
    import dense_fp32_matrix_03_gb300 as lib
    T, k, E, H = 35000, 2, 16, 32768
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    ids = torch.randint(0, E, (T, k), device="cuda", dtype=torch.int32, generator=gen)
    offsets, slots, positions = ints(E + 1), ints(T * k), ints(T * k)
    assert lib.sgemm_experts_sort(T, k, E, ids, offsets, slots, positions) == lib.SGEMM_OK
    x = torch.randint(-8, 9, (T, H), device="cuda", dtype=torch.int8, generator=gen).bfloat16()
    rows = torch.empty(T * k, H, dtype=torch.bfloat16, device="cuda")
    assert lib.sgemm_experts_dispatch("bf16", T, k, E, H, x, H, positions, offsets, rows, H) == 0
    out = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    assert lib.sgemm_experts_combine("bf16", T, k, E, H, rows, H, positions, offsets, None, out,
                                     H) == 0
    assert torch.equal(out, 2 * x)  # integers up to 16: exact
    at = torch.tensor([0, 1, T * k // 2, T * k - 1], device="cuda")
    assert torch.equal(rows[at], x[slots[at].long() // k])


def test_longest_row():
    """One row of 2^31 - 1 values, moved one by one: a column index a stride
    past the end does not fit 31 bits."""
    import torch
    import dense_fp32_matrix_03_gb300 as lib
    H = 2 ** 31 - 1
    x = torch.zeros(H, dtype=torch.bfloat16, device="cuda")
    ends = torch.arange(1, 100001, device="cuda") % 255
    x[:100000], x[-100000:] = ends, ends
    offsets = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    positions = torch.zeros(1, dtype=torch.int32, device="cuda")
    row, out = torch.empty_like(x), torch.empty_like(x)
    assert lib.sgemm_experts_dispatch("bf16", 1, 1, 1, H, x, H, positions, offsets, row, H) == 0
    assert torch.equal(row, x)
    assert lib.sgemm_experts_combine("bf16", 1, 1, 1, H, row, H, positions, offsets, None, out,
                                     H) == 0
    assert torch.equal(out, x)


def test_side_stream_repeats_bit_for_bit():
    import torch
    import dense_fp32_matrix_03_gb300 as lib
    T, k, E, H = 777, 3, 10, 1500
    rng = np.random.default_rng(11)
    ids = torch.from_numpy(make_ids(T, k, E, rng).astype(np.int32)).cuda()
    x = torch.randn(T, H, device="cuda")
    rows = torch.randn(T * k, H, device="cuda")
    w = torch.rand(T, k, device="cuda")
    torch.cuda.synchronize()
    results = []
    for _ in range(2):
        st = torch.cuda.Stream()
        offsets, slots, positions = ints(E + 1), ints(T * k), ints(T * k)
        drows, dw, out = torch.empty_like(rows), torch.empty_like(w), torch.empty_like(x)
        st.wait_stream(torch.cuda.current_stream())
        lib.check(lib.sgemm_experts_sort(T, k, E, ids, offsets, slots, positions, st))
        lib.check(lib.sgemm_experts_combine(
            "fp32", T, k, E, H, rows, H, positions, offsets, w, out, H, st))
        lib.check(lib.sgemm_experts_combine_grad(
            "fp32", T, k, E, H, x, H, rows, H, positions, offsets, w, drows, H, dw, st))
        st.synchronize()
        results.append([t.clone() for t in (offsets, slots, positions, drows, dw, out)])
    assert all(torch.equal(a, b) for a, b in zip(*results))
