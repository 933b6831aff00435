"""Pins of the expert layer's fp64 oracle (oracle/expert_layer.py), on the CPU:
the sort against sorted() and its inverse, dispatch and combine as matrix
products with a selection matrix, both gradients against central differences
(the maps are linear in rows and in weights, so differences are exact up to
rounding), the quantiser against its definition's inequalities, the product
against exact integers."""
import numpy as np
import pytest

from oracle import expert_layer as ex


def problem(T, k, E, H, seed, drop=0.3):
    rng = np.random.default_rng(seed)
    ids = np.stack([rng.permutation(max(E, k))[:k] for _ in range(T)])
    ids = np.where(rng.random((T, k)) < drop, -1, ids)
    offsets, slots, positions = ex.sort(ids, E)
    return rng, ids, offsets, slots, positions


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (7, 3, 5), (40, 2, 3), (12, 4, 9)])
def test_sort_is_stable_and_inverse(T, k, E):
    _, ids, offsets, slots, positions = problem(T, k, E, 1, T)
    flat = ids.reshape(-1)
    key = np.where((flat >= 0) & (flat < E), flat, E)
    assert list(slots) == sorted(range(T * k), key=lambda s: (key[s], s))
    assert np.array_equal(positions[slots], np.arange(T * k))
    for e in range(E):
        assert offsets[e + 1] - offsets[e] == np.sum(key == e)


def selection(ids, E, positions, total, T, k):
    S = np.zeros((T * k, T))
    for t in range(T):
        for j in range(k):
            if positions[t * k + j] < total:
                S[positions[t * k + j], t] = 1
    return S


def test_dispatch_and_combine_are_selection_products():
    T, k, E, H = 9, 3, 4, 6
    rng, ids, offsets, _, positions = problem(T, k, E, H, 3)
    S = selection(ids, E, positions, offsets[-1], T, k)
    x, rows = rng.standard_normal((T, H)), rng.standard_normal((T * k, H))
    w = rng.random((T, k))
    wpos = np.zeros(T * k)
    wpos[positions] = w.reshape(-1)
    assert np.allclose(ex.dispatch(x, positions, offsets[-1], k), S @ x)
    assert np.allclose(ex.combine(rows, positions, offsets[-1], w, T, k)[0],
                       S.T @ (wpos[:, None] * rows))
    assert np.allclose(ex.dispatch_grad(rows, positions, offsets[-1], T, k)[0], S.T @ rows)


def test_gradients_against_differences():
    T, k, E, H = 5, 2, 3, 4
    rng, ids, offsets, _, positions = problem(T, k, E, H, 4)
    total = offsets[-1]
    rows, w, g = rng.standard_normal((T * k, H)), rng.random((T, k)), rng.standard_normal((T, H))
    drows, dw, _ = ex.combine_grad(g, rows, positions, total, w, k)

    def loss(rows, w):
        return np.sum(g * ex.combine(rows, positions, total, w, T, k)[0])

    h = 1e-3
    for arr, grad, which in ((rows, drows, 0), (w, dw, 1)):
        num = np.zeros_like(arr)
        for i in np.ndindex(arr.shape):
            up, dn = arr.copy(), arr.copy()
            up[i] += h
            dn[i] -= h
            args = ((up, w), (dn, w)) if which == 0 else ((rows, up), (rows, dn))
            num[i] = (loss(*args[0]) - loss(*args[1])) / (2 * h)
        assert np.max(np.abs(num - grad)) < 1e-9
    x, gr = rng.standard_normal((T, H)), rng.standard_normal((T * k, H))
    dx, _ = ex.dispatch_grad(gr, positions, total, T, k)
    num = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        up, dn = x.copy(), x.copy()
        up[i] += h
        dn[i] -= h
        num[i] = np.sum(gr * (ex.dispatch(up, positions, total, k)
                              - ex.dispatch(dn, positions, total, k))) / (2 * h)
    assert np.max(np.abs(num - dx)) < 1e-9


def test_quantize_definition():
    rng = np.random.default_rng(5)
    x = rng.standard_normal((6, 11))
    x[2] = 0
    x[3] = 2.0 ** -101
    x[4, 3] = np.inf
    x[5, 0] = np.nan
    y, s = ex.quantize(x)
    q = np.rint(y)
    for r in (0, 1):
        assert np.max(np.abs(q[r])) == 127
        assert np.max(np.abs(q[r] * s[r] - x[r])) <= s[r] / 2 * (1 + 1e-12)
    assert s[2] == s[3] == 0 and not q[2:].any()
    assert np.isnan(s[4]) and np.isnan(s[5])


def test_product_is_the_integer_product():
    rng = np.random.default_rng(6)
    a = rng.integers(-128, 128, (5, 33)).astype(np.int8)
    b = rng.integers(-128, 128, (2, 4, 33)).astype(np.int8)
    offsets = [0, 3, 5]
    out, _, raw = ex.product_experts(offsets, a, np.ones(5), b, np.ones((2, 4)), 4)
    for e in range(2):
        lo, hi = offsets[e], offsets[e + 1]
        assert np.array_equal(out[lo:hi], a[lo:hi].astype(np.int64) @ b[e].astype(np.int64).T)
        assert (np.abs(out[lo:hi]) <= raw[lo:hi]).all()


def test_gated_activation():
    x = np.array([[0.0, 1.0, -2.0, 3.0, 5.0, 7.0]])
    want = [0.0, 5.0 / (1 + np.exp(-1.0)), -14.0 / (1 + np.exp(2.0))]
    assert np.allclose(ex.gated(x)[0], want)
