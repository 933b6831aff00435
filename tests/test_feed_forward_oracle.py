"""Pins of the oracle of the norm, the 4-bit format and the few-token expert
layer (oracle/feed_forward.py), on the CPU: the norm against its invariants and
its gradient against central differences, the 4-bit values against the format's
tables and torch's e4m3, the layout against a one-to-one map, the quantiser
against the nearest value over the whole grid, the layer against its parts."""
import numpy as np
import pytest

from oracle import feed_forward as ff


def test_norm_has_unit_rms_and_its_gradient_is_the_difference_quotient():
    rng = np.random.default_rng(0)
    M, H, eps = 3, 17, 1e-5
    s, w, dy, ds = (rng.standard_normal((M, H)) for _ in range(4))
    w = w[0]
    y, rho = ff.rms_norm(s, np.ones(H), eps)
    assert np.allclose((y * y).mean(1) + eps * rho ** 2, 1)
    dx, dw, _, _ = ff.rms_norm_grad(s, w, dy, ds, eps)

    def loss(s_, w_):
        return (ff.rms_norm(s_, w_, eps)[0] * dy).sum() + (s_ * ds).sum()

    h = 1e-6
    for i in range(M):
        for j in range(H):
            d = np.zeros((M, H))
            d[i, j] = h
            assert abs((loss(s + d, w) - loss(s - d, w)) / (2 * h) - dx[i, j]) < 1e-7
    for j in range(H):
        d = np.zeros(H)
        d[j] = h
        assert abs((loss(s, w + d) - loss(s, w - d)) / (2 * h) - dw[j]) < 1e-7


def test_e4m3_is_torchs():
    torch = pytest.importorskip("torch")
    b = np.arange(127, dtype=np.uint8)
    v = torch.from_numpy(b).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ff.e4m3_value(b), v) and np.array_equal(ff.e4m3_byte(v), b)
    x = np.concatenate([np.linspace(0, 448, 9001), np.exp2(np.linspace(-14, 8.8, 9001))])
    x = x.astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ff.round_e4m3(x), want)


def test_codes_are_the_nearest_values():
    u = np.linspace(-7, 7, 5601)
    c = ff.round_code(u)
    near = np.abs(u[:, None] - np.concatenate([ff.LEVELS, -ff.LEVELS])[None, :]).min(1)
    assert np.allclose(np.abs(u - ff.code_value(c)), near)
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    assert list(ff.round_code(ties)) == [0, 2, 2, 4, 4, 6, 6]
    assert list(ff.round_code(-ties)) == [8, 10, 10, 12, 12, 14, 14]
    assert list(ff.round_code(np.array([100.0, -0.0, 6.0]))) == [7, 8, 7]


@pytest.mark.parametrize("rows,blocks", [(1, 1), (130, 9), (256, 4), (31, 7)])
def test_layout_is_one_to_one(rows, blocks):
    r, j = np.meshgrid(np.arange(-(-rows // 128) * 128), np.arange(-(-blocks // 4) * 4),
                       indexing="ij")
    at = ff.scale_offset(r, j, blocks).reshape(-1)
    assert np.array_equal(np.sort(at), np.arange(at.size))
    b = np.random.default_rng(1).integers(0, 256, (rows, blocks)).astype(np.uint8)
    assert np.array_equal(ff.unpack_scales(ff.pack_scales(b, 0xFF), rows, blocks), b)
    c = np.random.default_rng(2).integers(0, 16, (rows, 2 * blocks + 1)).astype(np.uint8)
    assert np.array_equal(ff.unpack_codes(ff.pack_codes(c, 2 * blocks + 32), c.shape[1]), c)


@pytest.mark.parametrize("format_", ["mx", "nv"])
@pytest.mark.parametrize("K", [1, 16, 40, 200])
def test_quantiser_stays_within_half_a_step(format_, K):
    rng = np.random.default_rng(K)
    v = (rng.standard_normal((20, K)) * np.exp2(rng.integers(-20, 20, (20, 1)))).astype(np.float32)
    v[3] = 0
    v[4, 0] = np.nan
    codes, byte, row = ff.quantize4(v, format_)
    got = ff.values4(codes, byte, format_) * row[:, None]
    assert np.isnan(row[4]) and not codes[4].any() and not byte[4].any()
    assert not codes[3].any()
    s = np.repeat(ff.scale_value(byte, format_), ff.BLOCK[format_], axis=1)[:, :K]
    ok = np.arange(20) != 4
    a = np.abs(v[ok])
    unit = s[ok] * row[ok, None]
    # codes are a sixteenth apart from the largest on (mx: up to 8 units, cut at 6);
    # e4m3 scales may be 1/16 too small
    gap = np.where(a <= 2 * unit, 0.25, np.where(a <= 4 * unit, 0.5, 1.0)) * unit
    over = np.maximum(a - 6 * unit, 0)
    assert np.all(np.abs(got[ok] - v[ok]) <= np.maximum(gap, over) * (1 + 1e-5) + 1e-30)
    if format_ == "mx":
        assert np.all(a < 8 * unit + 1e-37)
    else:
        assert np.all(over <= 6 * unit / 15 + 1e-30)


def test_product_is_exact_on_small_integers():
    a = np.array([[1.0, -2, 3]])
    b = np.array([[4.0, 0.5, 1], [0, 0, 6]])
    c, mag = ff.product4(a, np.array([2.0]), b, np.array([1.0, 0.5]))
    assert np.array_equal(c, [[12.0, 18.0]]) and np.array_equal(mag, [[16.0, 18.0]])


def test_layer_is_its_parts():
    rng = np.random.default_rng(5)
    T, k, E, H, F = 3, 2, 4, 6, 5
    x, W1 = rng.standard_normal((T, H)), rng.standard_normal((E, 2 * F, H))
    W2 = rng.standard_normal((E, H, F))
    w = rng.random((T, k))
    ids = np.array([[0, 3], [2, 2], [-1, 9]])
    out, err = ff.experts_layer(x, ids, w, W1, None, W2, None, 2.0 ** -8)

    def expert(e, t):
        g, u = W1[e, :F] @ x[t], W1[e, F:] @ x[t]
        return W2[e] @ (g / (1 + np.exp(-g)) * u)

    assert np.allclose(out[0], w[0, 0] * expert(0, 0) + w[0, 1] * expert(3, 0))
    assert np.allclose(out[1], (w[1, 0] + w[1, 1]) * expert(2, 1))
    assert not out[2].any() and not err[2].any() and np.all(err[:2] > 0)
