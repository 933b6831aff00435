"""GPU parity of the whole expert layer for a few tokens
(sgemm_experts_layer, include/expert_layer.h) against the oracle
(oracle/feed_forward.py), element by element, through the C ABI.  The bound is
the oracle's (h kept in two parts of the row type, fp32 sums) plus out's own rounding."""
import numpy as np
import pytest

from oracle import feed_forward as ff
from test_gpu_experts import SUB, U, Rows, tdtype

pytestmark = pytest.mark.gpu
TYPES = ["bf16", "fp16"]
WTYPES = ["i8", "same"]


@pytest.fixture(scope="module", autouse=True)
def gpu_ready():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import dense_fp32_matrix_03_gb300 as lib
    lib.load()
    torch.cuda.init()


def up(n, step):
    return -(-n // step) * step


class Layer:
    """Experts' weights on the device, rows padded with values that would show,
    and what they stand for."""

    def __init__(self, type_, wtype, E, H, F, rng, pad=0):
        import torch
        self.type_, self.wtype, self.E, self.H, self.F = type_, wtype, E, H, F
        step = 16 if wtype == "i8" else 8
        self.ld1, self.ld2 = up(H, step) + pad * step, up(F, step) + pad * step
        self.s1 = self.s2 = None
        made = []
        for n, K, ld in ((2 * F, H, self.ld1), (H, F, self.ld2)):
            if wtype == "i8":
                w = torch.full((E, n, ld), 127, dtype=torch.int8, device="cuda")
                v = rng.integers(-128, 128, (E, n, K)).astype(np.int8)
                w[:, :, :K] = torch.from_numpy(v).cuda()
                s = ((0.5 + rng.random((E, n))) / (74 * max(K, 1) ** 0.5)).astype(np.float32)
                made.append((w, v.astype(np.float64), torch.from_numpy(s).cuda(), s.astype(np.float64)))
            else:
                w = torch.full((E, n, ld), float("nan"), dtype=tdtype(type_), device="cuda")
                v = rng.standard_normal((E, n, K)) / max(K, 1) ** 0.5
                w[:, :, :K] = torch.from_numpy(v).to(tdtype(type_)).cuda()
                made.append((w, w[:, :, :K].double().cpu().numpy(), None, None))
        (self.W1, self.v1, self.d1, self.s1), (self.W2, self.v2, self.d2, self.s2) = made

    def __call__(self, x, ids, weights, out, ws=None, stream=None):
        import torch
        import dense_fp32_matrix_03_gb300 as lib
        T, k = ids.shape
        size = lib.sgemm_experts_layer_workspace_size(T, k, self.H, self.F)
        if ws is None:
            ws = torch.full((max(size, 1),), 0xFF, dtype=torch.uint8, device="cuda")  # NaN
        return lib.sgemm_experts_layer(
            self.type_, self.wtype, T, k, self.E, self.H, self.F, x[0], x[1], ids, weights, self.W1,
            self.ld1, 2 * self.F * self.ld1, self.d1, self.W2, self.ld2, self.H * self.ld2, self.d2,
            out[0], out[1], ws, size, stream)

    def reference(self, x, ids, weights):
        return ff.experts_layer(x, ids, weights, self.v1, self.s1, self.v2, self.s2, U[self.type_])


def run(layer, T, k, rng, drop=0.2, pad=0, offset=0, weighted=True, ids=None):
    import torch
    import dense_fp32_matrix_03_gb300 as lib
    H, E, type_ = layer.H, layer.E, layer.type_
    if ids is None:
        ids = rng.integers(0, E, (T, k))
        gone = rng.random((T, k)) < drop
        ids = np.where(gone, rng.choice([-1, E, -2 ** 31, 2 ** 31 - 1], (T, k)), ids)
        if T > 2:
            ids[1] = -1
    x = Rows(T, H, type_, pad, offset, rng.standard_normal((T, H)))
    out = Rows(T, H, type_, pad, offset)
    w = rng.random((T, k)).astype(np.float32) if weighted else None
    if weighted:
        w[(ids < 0) | (ids >= E)] = np.nan  # never used
    d_ids = torch.from_numpy(ids.astype(np.int32)).cuda()
    d_w = torch.from_numpy(w).cuda() if weighted else None
    assert layer((x.ptr, x.ld), d_ids, d_w, (out.ptr, out.ld)) == lib.SGEMM_OK
    assert lib.sgemm_poll_error() == lib.SGEMM_OK
    ref, err = layer.reference(x.np(), ids, w)
    got = out.np()
    assert np.all(np.abs(got - ref) <= err + (U[type_] + 2.0 ** -23) * np.abs(ref) + SUB)
    assert out.pad_untouched()
    if T > 2:
        none = ~((ids >= 0) & (ids < E)).any(1)
        assert not got[none].any()


# T, k, E, H, F, pad, offset
SIZES = [(1, 1, 1, 16, 16, 0, 0), (1, 4, 8, 256, 128, 0, 0), (2, 2, 3, 8, 3, 0, 0),
         (3, 2, 4, 1, 1, 0, 0), (5, 3, 6, 100, 90, 1, 1), (8, 4, 32, 512, 256, 0, 8),
         (9, 2, 4, 333, 77, 0, 0), (16, 4, 5, 264, 272, 2, 4), (17, 1, 1, 192, 130, 0, 0),
         (33, 3, 2, 160, 48, 0, 0), (64, 8, 60, 96, 64, 0, 0), (64, 1, 1024, 64, 40, 0, 0),
         (8, 64, 7, 128, 33, 0, 0), (1, 64, 100, 64, 64, 0, 0), (12, 4, 16, 1025, 515, 0, 0),
         (1, 2, 4, 2048, 1024, 0, 0)]


@pytest.mark.parametrize("wtype", WTYPES)
@pytest.mark.parametrize("type_", TYPES)
@pytest.mark.parametrize("T,k,E,H,F,pad,offset", SIZES)
def test_layer(type_, wtype, T, k, E, H, F, pad, offset):
    rng = np.random.default_rng(H + F)
    run(Layer(type_, wtype, E, H, F, rng, pad=pad % 2), T, k, rng, pad=pad, offset=offset)


@pytest.mark.parametrize("wtype", WTYPES)
def test_layer_without_weights_and_with_all_rows_on_one_expert(wtype):
    rng = np.random.default_rng(1)
    layer = Layer("bf16", wtype, 6, 200, 120, rng)
    run(layer, 7, 3, rng, weighted=False)
    run(layer, 64, 1, rng, ids=np.full((64, 1), 4))
    run(layer, 5, 4, rng, ids=np.full((5, 4), 2))          # one expert, four times a token
    run(layer, 4, 2, rng, ids=np.full((4, 2), -1))         # nobody
    run(layer, 1, 6, rng, ids=np.array([[5, 4, 3, 2, 1, 0]]))


@pytest.mark.parametrize("wtype", WTYPES)
def test_weights_of_experts_nobody_chose_are_not_read(wtype):
    import torch
    rng = np.random.default_rng(2)
    layer = Layer("fp16", wtype, 5, 64, 48, rng)
    if wtype == "same":
        layer.W1[3] = float("nan")
        layer.W2[3] = float("inf")
    else:
        layer.d1[3] = float("nan")
        layer.d2[3] = float("nan")
    run(layer, 6, 2, rng, ids=rng.choice([0, 1, 2, 4], (6, 2)))
    torch.cuda.synchronize()


def test_layer_without_hidden_values_is_zero():
    import torch
    import dense_fp32_matrix_03_gb300 as lib
    x, out = (torch.full((3, 40), 2.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ids = torch.zeros(3, 2, dtype=torch.int32, device="cuda")
    assert lib.sgemm_experts_layer("bf16", "same", 3, 2, 4, 40, 0, x, 40, ids, None, None, 40, 0,
                                   None, None, 8, 40 * 8, None, out, 40, None, 0) == lib.SGEMM_OK
    assert not out.float().cpu().numpy().any()


@pytest.mark.parametrize("wtype", WTYPES)
@pytest.mark.parametrize("T", [1, 12])
def test_layer_in_a_graph_and_on_streams(wtype, T):
    """Chains of dependent calls (each layer's output is the next one's input),
    captured and replayed with new choices, beside eager calls on another stream
    with a workspace of their own: the same bits."""
    import torch
    import dense_fp32_matrix_03_gb300 as lib
    rng = np.random.default_rng(T)
    k, E, H, F = 2, 6, 256, 192
    layer = Layer("bf16", wtype, E, H, F, rng)
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    ids = torch.zeros(T, k, dtype=torch.int32, device="cuda")
    w = torch.zeros(T, k, device="cuda")
    size = lib.sgemm_experts_layer_workspace_size(T, k, H, F)

    def buffers():
        return ([torch.zeros_like(x) for _ in range(4)],
                torch.zeros(size, dtype=torch.uint8, device="cuda"))

    def chain(bufs, stream=None):
        outs, ws = bufs
        src = x
        for o in outs:
            lib.check(layer((src, H), ids, w, (o, H), ws, stream))
            src = o

    captured, eager, side = buffers(), buffers(), torch.cuda.Stream()
    chain(captured)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain(captured)
    for seed in (1, 2, 3):
        gen = np.random.default_rng(seed)
        x.copy_(torch.from_numpy(gen.standard_normal((T, H))))
        ids.copy_(torch.from_numpy(gen.integers(-1, E, (T, k)).astype(np.int32)))
        w.copy_(torch.from_numpy(gen.random((T, k)).astype(np.float32)))
        torch.cuda.synchronize()
        graph.replay()
        chain(eager, side)
        torch.cuda.synchronize()
        src = x
        for a, b in zip(captured[0], eager[0]):
            assert torch.equal(a, b)
            ref, err = layer.reference(src.double().cpu().numpy(), ids.cpu().numpy(),
                                       w.cpu().numpy())
            assert np.all(np.abs(a.double().cpu().numpy() - ref) <=
                          err + (U["bf16"] + 2.0 ** -23) * np.abs(ref) + SUB)
            src = a
