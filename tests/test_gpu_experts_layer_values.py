"""The few-token expert layer (sgemm_experts_layer, include/expert_layer.h) on
values that are not ordinary: small and large hidden values, tokens that hold no
numbers.  The bound is the oracle's; what a hidden value may be off by however
small it is: 2^-36 in fp16 (a rest below 2^-14, kept 2^11 times, to half of 2^-24),
in bf16 2^-100 (its own least number is 2^-133; gates below -88, where exp(-x) is
past fp32, lose some 2^-121 times the up value)."""
import numpy as np
import pytest

from oracle import feed_forward as ff
from test_gpu_experts import SUB, U, Rows
from test_gpu_experts_layer import TYPES, WTYPES, Layer, gpu_ready  # noqa: F401

pytestmark = pytest.mark.gpu
LEAST = {"bf16": 2.0 ** -100, "fp16": 2.0 ** -36}


def layer_of(layer, x, ids, w):
    """(out, reference, bound) of rows x (fp64)."""
    import torch
    import dense_fp32_matrix_03_gb300 as lib
    T = x.shape[0]
    xr, out = Rows(T, layer.H, layer.type_, 0, 0, x), Rows(T, layer.H, layer.type_, 0, 0)
    assert layer((xr.ptr, xr.ld), torch.from_numpy(ids.astype(np.int32)).cuda(),
                 torch.from_numpy(w).cuda(), (out.ptr, out.ld)) == lib.SGEMM_OK
    assert lib.sgemm_poll_error() == lib.SGEMM_OK
    u = U[layer.type_]
    with np.errstate(all="ignore"):
        ref, err = ff.experts_layer(xr.np(), ids, w, layer.v1, layer.s1, layer.v2, layer.s2, u,
                                    LEAST[layer.type_])
    return out.np(), ref, err + (u + 2.0 ** -23) * np.abs(ref) + SUB


def hidden_max(layer, x, e):
    """The largest hidden value of a token through expert e."""
    w = layer.v1[e] if layer.s1 is None else layer.v1[e] * layer.s1[e][:, None]
    g = w @ x
    g, u = g[:layer.F], g[layer.F:]
    with np.errstate(over="ignore"):
        return np.abs(g / (1 + np.exp(-g)) * u).max()


@pytest.mark.parametrize("wtype", WTYPES)
@pytest.mark.parametrize("type_", TYPES)
@pytest.mark.parametrize("T", [3, 16, 40])
def test_small_hidden_values_keep_their_digits(type_, wtype, T):
    """Tokens of 2^-5 to 2^-14 (hidden values some 2^-11 to 2^-29), with down
    weights 2^12 times the ordinary, so that the result shows them."""
    rng = np.random.default_rng(T)
    layer = Layer(type_, wtype, 4, 200, 136, rng)
    if wtype == "i8":
        layer.d2 *= 2.0 ** 12
        layer.s2 = layer.s2 * 2.0 ** 12
    else:
        layer.W2 *= 2.0 ** 12
        layer.v2 = layer.v2 * 2.0 ** 12
    x = rng.standard_normal((T, 200)) * np.exp2(-rng.integers(5, 15, (T, 1)))
    got, ref, bound = layer_of(layer, x, rng.integers(0, 4, (T, 2)),
                               rng.random((T, 2)).astype(np.float32))
    assert np.all(np.abs(got - ref) <= bound)


@pytest.mark.parametrize("wtype", WTYPES)
@pytest.mark.parametrize("type_", TYPES)
@pytest.mark.parametrize("T", [2, 12, 33])
def test_ordinary_values_with_the_closer_bound(type_, wtype, T):
    rng = np.random.default_rng(T)
    layer = Layer(type_, wtype, 5, 264, 200, rng)
    got, ref, bound = layer_of(layer, rng.standard_normal((T, 264)), rng.integers(0, 5, (T, 3)),
                               rng.random((T, 3)).astype(np.float32))
    assert np.all(np.abs(got - ref) <= bound)


@pytest.mark.parametrize("wtype", WTYPES)
@pytest.mark.parametrize("type_", TYPES)
@pytest.mark.parametrize("T", [4, 20])
def test_large_hidden_values(type_, wtype, T):
    """Tokens whose hidden values grow past fp16's range: bf16 carries them, fp16
    up to 65504; beyond, that token's row is no number, and it alone."""
    rng = np.random.default_rng(T)
    layer = Layer(type_, wtype, 3, 128, 96, rng)
    x = rng.standard_normal((T, 128)) * np.exp2(np.linspace(3, 9, T))[:, None]
    ids = rng.integers(0, 3, (T, 1))
    w = ((0.5 + rng.random((T, 1))) / 64).astype(np.float32)
    got, ref, bound = layer_of(layer, x, ids, w)
    most = np.array([hidden_max(layer, x[t], ids[t, 0]) for t in range(T)])
    past = most > 65000 if type_ == "fp16" else np.zeros(T, bool)
    assert type_ == "bf16" or (past.any() and not past.all())
    assert np.all((np.abs(got - ref) <= bound)[~past])
    assert not np.isfinite(got[most > 66000]).any() or type_ == "bf16"


@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("wtype", WTYPES)
@pytest.mark.parametrize("type_", TYPES)
@pytest.mark.parametrize("T,H,F", [(2, 64, 48), (9, 333, 77), (40, 128, 64)])
def test_a_token_that_is_no_number_spoils_its_own_row_alone(type_, wtype, value, T, H, F):
    rng = np.random.default_rng(T)
    layer = Layer(type_, wtype, 3, H, F, rng)
    x = rng.standard_normal((T, H))
    x[1, H - 1] = value
    got, ref, bound = layer_of(layer, x, rng.integers(0, 3, (T, 2)),
                               rng.random((T, 2)).astype(np.float32))
    clean = np.arange(T) != 1
    assert np.all((np.abs(got - ref) <= bound)[clean])
    assert not np.isfinite(got[1]).any()
