"""GPU parity of the norm and its gradient (include/rms_norm.h) against the
oracle (oracle/feed_forward.py), element by element, through the C ABI.

Bounds, derived from the arithmetic: u = half a unit in the last place of the
row type, e = 2^-24 per fp32 operation; at least 32 threads share a row, so its
sums are H / 32 additions deep, plus ten to join them.
  sum        bit for bit (one fp32 addition, one rounding)
  y          (u + (H / 64 + 16) e) |ref|: the square root halves the sum's error
  codes      bit for bit: neither sums nor square roots reach them
  scale      (H / 64 + 16) e |ref|
  dx         u |ref| + (H / 32 + 32) e (|dsum| + rho |w dy| + rho^3 |s| mean|w dy s|)
  dweight    (M / 128 + H / 64 + 64) e sum|dy s rho|: rows are spread over 300
             partial sums or more, 32 threads join them
plus the smallest subnormal of fp16 where results can underflow."""
import numpy as np
import pytest

from oracle import feed_forward as ff
from test_gpu_experts import E24, SUB, TYPES, U, Rows, tdtype

pytestmark = pytest.mark.gpu
EPS = 1e-5
F32 = np.float32


@pytest.fixture(scope="module", autouse=True)
def gpu_ready():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import dense_fp32_matrix_03_gb300 as lib
    lib.load()
    torch.cuda.init()


def vec(values, type_):
    import torch
    return torch.from_numpy(values).to(tdtype(type_)).cuda()


def draw(rng, *shape):
    """Values of both signs, rows of different sizes."""
    x = rng.standard_normal(shape)
    return x * np.exp2(rng.integers(-6, 7, shape[:1]))[:, None] if len(shape) > 1 else x


# M, H, pad, offset: one value to rows longer than the registers (8192 values
# of 16 bits in 16-byte vectors, 4096 of 32), on 16-byte boundaries and off
# them, few rows and many
SHAPES = [(1, 1, 0, 0), (3, 2, 0, 1), (2, 7, 0, 0), (5, 31, 0, 0), (4, 64, 0, 0), (9, 100, 4, 4),
          (200, 96, 0, 0), (333, 257, 0, 0), (1, 4096, 0, 0), (160, 1500, 0, 0), (7, 1002, 2, 2),
          (3, 8192, 8, 8), (2, 8200, 0, 0), (2, 20011, 0, 3), (170, 4100, 0, 0), (1000, 33, 1, 1)]


def problem(M, H, type_, pad, offset, seed, zero_row=True):
    rng = np.random.default_rng(seed)
    xv, rv = draw(rng, M, H), draw(rng, M, H)
    if zero_row and M > 1:
        xv[1], rv[1] = 0, 0
    x, r = Rows(M, H, type_, pad, offset, xv), Rows(M, H, type_, pad, offset, rv)
    w = vec(1 + 0.3 * rng.standard_normal(H), type_)
    return rng, x, r, w


def kept(x, r, type_):
    """The sum as the row type keeps it, by torch on the CPU."""
    import torch
    s = x.view.cpu().float()
    if r is not None:
        s = (s + r.view.cpu().float()).to(tdtype(type_)).float()
    return s.numpy()


@pytest.mark.parametrize("type_", TYPES)
@pytest.mark.parametrize("M,H,pad,offset", SHAPES)
def test_norm(type_, M, H, pad, offset):
    import dense_fp32_matrix_03_gb300 as lib
    _, x, r, w = problem(M, H, type_, pad, offset, H)
    u = U[type_]
    for res, weight, keep in ((r, w, True), (None, w, False), (r, None, False), (None, None, True)):
        s = kept(x, res, type_)
        wv = np.ones(H) if weight is None else w.double().cpu().numpy()
        ref, _ = ff.rms_norm(s.astype(np.float64), wv, EPS)
        y, total = Rows(M, H, type_, pad, offset), Rows(M, H, type_, pad, offset)
        assert lib.sgemm_rms_norm(type_, M, H, EPS, x.ptr, x.ld, res and res.ptr, res and res.ld or 0,
                                  weight, total.ptr if keep else None, total.ld if keep else 0,
                                  y.ptr, y.ld) == lib.SGEMM_OK
        assert np.all(np.abs(y.np() - ref) <= (u + (H / 64 + 16) * E24) * np.abs(ref) + SUB)
        assert y.pad_untouched()
        if keep:
            assert np.array_equal(total.np(), s) and total.pad_untouched()


@pytest.mark.parametrize("type_", TYPES)
@pytest.mark.parametrize("M,H,pad,offset", SHAPES)
def test_norm_in_8_bits(type_, M, H, pad, offset):
    import torch
    import dense_fp32_matrix_03_gb300 as lib
    _, x, r, w = problem(M, H, type_, pad, offset, H + 1)
    s = kept(x, r, type_)
    v = s * w.float().cpu().numpy()
    codes, scale = ff.quantize8(v)
    _, rho = ff.rms_norm(s.astype(np.float64), np.ones(H), EPS)
    for ldq, shift in ((H + pad, 0), ((H + 15) // 16 * 16, 16), (H + 3, 5)):
        q = torch.full((M * ldq + shift + 16,), 99, dtype=torch.int8, device="cuda")
        sc = torch.full((M,), -1.0, device="cuda")
        total = Rows(M, H, type_, pad, offset)
        assert lib.sgemm_rms_norm_i8(type_, M, H, EPS, x.ptr, x.ld, r.ptr, r.ld, w, total.ptr,
                                     total.ld, q.data_ptr() + shift, ldq, sc) == lib.SGEMM_OK
        got = q[shift:shift + M * ldq].view(M, ldq).cpu().numpy()
        assert np.array_equal(got[:, :H], codes)
        assert np.all(got[:, H:] == 99) and bool((q[:shift] == 99).all())
        want = scale * rho
        assert np.all(np.abs(sc.cpu().numpy() - want) <= (H / 64 + 16) * E24 * np.abs(want))
        assert np.array_equal(total.np(), s)


@pytest.mark.parametrize("format_", ["mx", "nv"])
@pytest.mark.parametrize("type_", TYPES)
@pytest.mark.parametrize("M,H,pad,offset", SHAPES)
def test_norm_in_4_bits(type_, format_, M, H, pad, offset):
    import torch
    import dense_fp32_matrix_03_gb300 as lib
    _, x, r, w = problem(M, H, type_, pad, offset, H + 2)
    s = kept(x, r, type_)
    codes, byte, row = ff.quantize4(s * w.float().cpu().numpy(), format_)
    _, rho = ff.rms_norm(s.astype(np.float64), np.ones(H), EPS)
    ld = (H + 31) // 32 * 32 + 32
    q = torch.full((M, ld // 2), 0x5A, dtype=torch.uint8, device="cuda")
    sf = torch.full((lib.sgemm_fp4_scales_size(format_, M, H),), 0xA5, dtype=torch.uint8,
                    device="cuda")
    sc = torch.full((M,), -1.0, device="cuda")
    total = Rows(M, H, type_, pad, offset)
    assert lib.sgemm_rms_norm_fp4(type_, format_, M, H, EPS, x.ptr, x.ld, r.ptr, r.ld, w,
                                  total.ptr, total.ld, q, ld, sf, sc) == lib.SGEMM_OK
    check_4_bits(q, sf, codes, byte)
    want = row * rho
    assert np.all(np.abs(sc.cpu().numpy() - want) <= (H / 64 + 16) * E24 * np.abs(want))
    assert np.array_equal(total.np(), s)


def check_4_bits(q, sf, codes, byte):
    """Codes and block scales bit for bit, the zeros behind them, and nothing
    else written (q was full of 0x5A, sf of 0xA5)."""
    M, K = codes.shape
    q, sf = q.cpu().numpy(), sf.cpu().numpy()
    full = -(-K // 8) * 4  # bytes written
    got = ff.unpack_codes(q, 2 * q.shape[1])
    assert np.array_equal(got[:, :K], codes)
    assert not got[:, K:2 * full].any() and np.all(q[:, full:] == 0x5A)
    blocks = byte.shape[1]
    assert np.array_equal(sf, ff.pack_scales(byte, 0xA5)), (blocks,)


@pytest.mark.parametrize("type_", TYPES)
@pytest.mark.parametrize("M,H,pad,offset", SHAPES + [(5000, 40, 0, 0)])
def test_gradient(type_, M, H, pad, offset):
    import torch
    import dense_fp32_matrix_03_gb300 as lib
    rng, s, dy, w = problem(M, H, type_, pad, offset, H + 3, zero_row=False)
    if M > 1:
        s.view[1] = 0  # rho = 1 / sqrt(eps)
    ds = Rows(M, H, type_, pad, offset, draw(rng, M, H))
    size = lib.sgemm_rms_norm_grad_workspace_size(M, H)
    ws = torch.full((size // 4,), float("nan"), device="cuda")
    for weight, stream, want_dw in ((w, ds, True), (None, ds, True), (w, None, True),
                                    (w, ds, False)):
        wv = np.ones(H) if weight is None else w.double().cpu().numpy()
        dv = ds.np() if stream is not None else np.zeros((M, H))
        ref, dwref, mag, dwmag = ff.rms_norm_grad(s.np(), wv, dy.np(), dv, EPS)
        dx = Rows(M, H, type_, pad, offset)
        dw = torch.full((H,), float("nan"), device="cuda")
        args = (type_, M, H, EPS, s.ptr, s.ld, weight, dy.ptr, dy.ld, stream and stream.ptr,
                stream and stream.ld or 0, dx.ptr, dx.ld)
        assert lib.sgemm_rms_norm_grad(*args, dw if want_dw else None, ws if want_dw else None,
                                       size if want_dw else 0) == lib.SGEMM_OK
        bound = U[type_] * np.abs(ref) + (H / 32 + 32) * E24 * mag + SUB
        near = np.abs(dx.np() - ref) <= bound
        if type_ == "fp16":
            # a result beyond 65504 and half a step rounds to an infinity: the row of
            # zeros has rho = 316, times w dy of up to some 64 * 4 * 2
            over = np.abs(ref) + bound >= 65520
            near |= over & np.isinf(dx.np()) & (np.sign(dx.np()) == np.sign(ref))
        assert np.all(near)
        assert dx.pad_untouched()
        if want_dw:
            got = dw.double().cpu().numpy()
            assert np.all(np.abs(got - dwref) <= (M / 128 + H / 64 + 64) * E24 * dwmag)
            # the same bits again, whatever the workspace holds
            ws.fill_(1e30)
            again = torch.empty_like(dw)
            assert lib.sgemm_rms_norm_grad(*args, again, ws, size) == lib.SGEMM_OK
            assert torch.equal(again, dw)


def test_gradient_is_the_difference_quotient():
    """<dy, y(s + d) - y(s - d)> / 2 = <gradient, d> up to d^3 and roundings, fp32:
    y's error (H / 64 + 17) e |y| per value against differences of some 2^-7."""
    import torch
    import dense_fp32_matrix_03_gb300 as lib
    M, H = 4, 48
    rng = np.random.default_rng(11)
    s, dy, d = (rng.standard_normal((M, H)).astype(F32) for _ in range(3))
    w = vec((1 + 0.3 * rng.standard_normal(H)).astype(F32), "fp32")
    d *= F32(2.0 ** -7)

    def y(rows):
        out = torch.empty(M, H, device="cuda")
        assert lib.sgemm_rms_norm("fp32", M, H, EPS, torch.from_numpy(rows).cuda(), H, None, 0, w,
                                  None, 0, out, H) == lib.SGEMM_OK
        return out.double().cpu().numpy()

    dx, dw = torch.empty(M, H, device="cuda"), torch.empty(H, device="cuda")
    size = lib.sgemm_rms_norm_grad_workspace_size(M, H)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    assert lib.sgemm_rms_norm_grad("fp32", M, H, EPS, torch.from_numpy(s).cuda(), H, w,
                                   torch.from_numpy(dy).cuda(), H, None, 0, dx, H, dw, ws,
                                   size) == lib.SGEMM_OK
    up, down = (s + d).astype(F32), (s - d).astype(F32)
    step = (up.astype(np.float64) - down) / 2
    got = (dx.double().cpu().numpy() * step).sum()
    diff = ((y(up) - y(down)) / 2 * dy).sum()
    # the third derivative's share: |d|^3 of some 2^-21 times a small constant a value
    bound = M * H * (2.0 ** -21 * 10 + 18 * E24 * 10)
    assert abs(got - diff) <= bound and abs(diff) > 10 * bound


@pytest.mark.parametrize("type_", TYPES)
@pytest.mark.parametrize("H", [96, 9001])
def test_in_place(type_, H):
    """sum over res or x, y over x, dx over dy or dsum: the same bits as apart."""
    import torch
    import dense_fp32_matrix_03_gb300 as lib
    M = 5
    rng, x, r, w = problem(M, H, type_, 0, 0, 3)
    s, y = Rows(M, H, type_), Rows(M, H, type_)
    norm = lambda a, b, sum_, out: lib.check(lib.sgemm_rms_norm(  # noqa: E731
        type_, M, H, EPS, a, H, b, H, w, sum_, H if sum_ is not None else 0, out, H))
    norm(x.view, r.view, s.view, y.view)
    x2, r2 = x.view.clone(), r.view.clone()
    norm(x2, r2, r2, x2)
    assert torch.equal(r2, s.view) and torch.equal(x2, y.view)
    x2, r2 = x.view.clone(), r.view.clone()
    norm(x2, r2, x2, r2)
    assert torch.equal(x2, s.view) and torch.equal(r2, y.view)
    x2 = x.view.clone()
    norm(x2, r.view, None, x2)
    assert torch.equal(x2, y.view)
    dy, ds = Rows(M, H, type_, values=draw(rng, M, H)), Rows(M, H, type_, values=draw(rng, M, H))
    size = lib.sgemm_rms_norm_grad_workspace_size(M, H)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    results = []
    for over in (None, "dy", "ds"):
        g, d = dy.view.clone(), ds.view.clone()
        dx = {"dy": g, "ds": d}.get(over, torch.empty_like(g))
        dw = torch.empty(H, device="cuda")
        lib.check(lib.sgemm_rms_norm_grad(type_, M, H, EPS, s.view, H, w, g, H, d, H, dx, H, dw, ws,
                                          size))
        results.append((dx.clone(), dw))
    for dx, dw in results[1:]:
        assert torch.equal(dx, results[0][0]) and torch.equal(dw, results[0][1])


@pytest.mark.parametrize("type_", TYPES)
def test_rows_that_hold_no_number(type_):
    """A row with an infinity or NaN spoils itself alone; its codes are zeros and
    its scale NaN."""
    import torch
    import dense_fp32_matrix_03_gb300 as lib
    M, H = 6, 80
    _, x, _, w = problem(M, H, type_, 0, 0, 5, zero_row=False)
    x.view[1, 3] = float("inf")
    x.view[2, 79] = float("nan")
    x.view[4, 0] = -float("inf")
    bad = np.array([0, 1, 1, 0, 1, 0], bool)
    y = Rows(M, H, type_)
    lib.check(lib.sgemm_rms_norm(type_, M, H, EPS, x.ptr, H, None, 0, w, None, 0, y.ptr, H))
    got = y.np()
    assert np.isfinite(got[~bad]).all()
    for i, j in ((1, 3), (2, 79), (4, 0)):
        assert np.isnan(got[i, j])
    q = torch.full((M, H), 9, dtype=torch.int8, device="cuda")
    sc = torch.empty(M, device="cuda")
    lib.check(lib.sgemm_rms_norm_i8(type_, M, H, EPS, x.ptr, H, None, 0, w, None, 0, q, H, sc))
    assert np.array_equal(np.isnan(sc.cpu().numpy()), bad)
    assert not q.cpu().numpy()[bad].any() and q.cpu().numpy()[~bad].any(1).all()
    for format_ in ("mx", "nv"):
        q = torch.full((M, 48), 9, dtype=torch.uint8, device="cuda")
        sf = torch.full((lib.sgemm_fp4_scales_size(format_, M, H),), 9, dtype=torch.uint8,
                        device="cuda")
        lib.check(lib.sgemm_rms_norm_fp4(type_, format_, M, H, EPS, x.ptr, H, None, 0, w, None, 0,
                                         q, 96, sf, sc))
        assert np.array_equal(np.isnan(sc.cpu().numpy()), bad)
        assert not q.cpu().numpy()[bad][:, :40].any()
        assert not ff.unpack_scales(sf.cpu().numpy(), M, -(-H // ff.BLOCK[format_]))[bad].any()


def test_squares_past_the_range():
    """A row whose sum of squares leaves fp32's range has rho 0: zeros, and the
    gradient of the stream alone.  (fp16 cannot hold such values.)"""
    import torch
    import dense_fp32_matrix_03_gb300 as lib
    M, H = 2, 64
    x = torch.full((M, H), 2.0 ** 70, device="cuda")
    x[1] = 1.0
    y, sc = torch.empty_like(x), torch.empty(M, device="cuda")
    q = torch.empty(M, H, dtype=torch.int8, device="cuda")
    lib.check(lib.sgemm_rms_norm("fp32", M, H, EPS, x, H, None, 0, None, None, 0, y, H))
    lib.check(lib.sgemm_rms_norm_i8("fp32", M, H, EPS, x, H, None, 0, None, None, 0, q, H, sc))
    assert not y[0].cpu().numpy().any() and sc[0].item() == 0
    assert np.allclose(y[1].cpu().numpy(), 1, atol=1e-4) and sc[1].item() > 0
    ds = torch.randn(M, H, device="cuda")
    dx = torch.empty_like(x)
    lib.check(lib.sgemm_rms_norm_grad("fp32", M, H, EPS, x, H, None, ds, H, ds, H, dx, H, None,
                                      None, 0))
    assert torch.isfinite(dx[1]).all()


def test_rows_without_values():
    import torch
    import dense_fp32_matrix_03_gb300 as lib
    sc = torch.full((3,), 7.0, device="cuda")
    assert lib.sgemm_rms_norm_i8("bf16", 3, 0, EPS, None, 1, None, 0, None, None, 0, None, 1,
                                 sc) == lib.SGEMM_OK
    assert not sc.cpu().numpy().any()
    for format_ in ("mx", "nv"):
        sc.fill_(7.0)
        assert lib.sgemm_rms_norm_fp4("bf16", format_, 3, 0, EPS, None, 1, None, 0, None, None, 0,
                                      None, 32, None, sc) == lib.SGEMM_OK
        assert not sc.cpu().numpy().any()
    dw = torch.full((40,), 7.0, device="cuda")
    assert lib.sgemm_rms_norm_grad("bf16", 0, 40, EPS, None, 40, None, None, 40, None, 0, None, 40,
                                   dw, None, 0) == lib.SGEMM_OK
    assert not dw.cpu().numpy().any()


def test_captured_and_on_another_stream():
    """The forward and backward calls captured once and replayed on new inputs,
    beside an eager call on another stream."""
    import torch
    import dense_fp32_matrix_03_gb300 as lib
    M, H = 300, 512
    rng = np.random.default_rng(2)
    x, r, dy, s, y, dx = (torch.zeros(M, H, dtype=torch.bfloat16, device="cuda") for _ in range(6))
    w = vec(1 + 0.3 * rng.standard_normal(H), "bf16")
    dw = torch.empty(H, device="cuda")
    size = lib.sgemm_rms_norm_grad_workspace_size(M, H)
    ws, ws2 = (torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(2))

    def both(x, s, y, dx, dw, ws, stream=None):
        lib.check(lib.sgemm_rms_norm("bf16", M, H, EPS, x, H, r, H, w, s, H, y, H, stream))
        lib.check(lib.sgemm_rms_norm_grad("bf16", M, H, EPS, s, H, w, dy, H, None, 0, dx, H, dw, ws,
                                          size, stream))

    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(x, s, y, dx, dw, ws)
    for seed in (1, 2):
        gen = np.random.default_rng(seed)
        for t in (x, r, dy):
            t.copy_(torch.from_numpy(gen.standard_normal((M, H))))
        eager = [torch.empty_like(t) for t in (s, y, dx, dw)]
        torch.cuda.synchronize()
        graph.replay()
        both(x, *eager, ws2, stream=side)
        torch.cuda.synchronize()
        for a, b in zip((s, y, dx, dw), eager):
            assert torch.equal(a, b)
        ref, _ = ff.rms_norm(s.double().cpu().numpy(), w.double().cpu().numpy(), EPS)
        assert np.all(np.abs(y.double().cpu().numpy() - ref) <= 1.01 * U["bf16"] * np.abs(ref))
