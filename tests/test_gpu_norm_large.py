"""The norm's gradient where the forward call's rho is 0 (include/rms_norm.h): rows
whose squares leave fp32's range, and whose products with dy may, too.  Such a row
passes dsum on and adds nothing to the weight's gradient; a row that holds an
infinity or NaN spoils itself and the columns that it reaches."""
import numpy as np
import pytest

from oracle import feed_forward as ff
from test_gpu_experts import E24, U, tdtype
from test_gpu_norm import EPS, gpu_ready  # noqa: F401

pytestmark = pytest.mark.gpu


def grad(type_, s, w, dy, ds):
    import torch
    import dense_fp32_matrix_03_gb300 as lib
    M, H = s.shape
    t = [torch.from_numpy(a).to(tdtype(type_)).cuda() for a in (s, w, dy, ds)]
    dx, dw = torch.empty_like(t[0]), torch.full((H,), 7.0, device="cuda")
    size = lib.sgemm_rms_norm_grad_workspace_size(M, H)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    lib.check(lib.sgemm_rms_norm_grad(type_, M, H, EPS, t[0], H, t[1], t[2], H, t[3], H, dx, H, dw,
                                      ws, size))
    return [a.double().cpu().numpy() for a in (*t, dx, dw)]


@pytest.mark.parametrize("size", [2.0 ** 70, 1.5 * 2.0 ** 126])
@pytest.mark.parametrize("type_", ["bf16", "fp32"])
@pytest.mark.parametrize("H", [64, 1000, 9001])
def test_rows_past_the_range_pass_the_streams_gradient_on(type_, H, size):
    M = 9
    rng = np.random.default_rng(H)
    s, dy, ds = (rng.standard_normal((M, H)) for _ in range(3))
    big = np.array([0, 1, 0, 0, 1, 0, 0, 0, 1], bool)
    s[big] = size * rng.choice([-1, 1], (3, H))
    dy[big] *= 8
    s, w, dy, ds, dx, dw = grad(type_, s, 1 + 0.3 * rng.standard_normal(H), dy, ds)
    assert np.array_equal(dx[big], ds[big])
    rest = ~big
    ref, dwref, mag, dwmag = ff.rms_norm_grad(s[rest], w, dy[rest], ds[rest], EPS)
    assert np.all(np.abs(dx[rest] - ref) <= U[type_] * np.abs(ref) + (H / 32 + 32) * E24 * mag)
    assert np.all(np.abs(dw - dwref) <= (H / 64 + 64) * E24 * dwmag)


@pytest.mark.parametrize("value", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("type_", ["bf16", "fp16", "fp32"])
def test_rows_that_hold_no_number_show_in_the_gradient(type_, value):
    M, H = 5, 200
    rng = np.random.default_rng(1)
    s, dy, ds = (rng.standard_normal((M, H)) for _ in range(3))
    s[2, 33] = value
    s, w, dy, ds, dx, dw = grad(type_, s, np.ones(H), dy, ds)
    assert np.isnan(dx[2, 33]) and np.isnan(dw[33])
    other = np.arange(M) != 2
    assert np.isfinite(dx[other]).all()
