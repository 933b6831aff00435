"""An expert layer on this library's entry points, served and trained.

    python examples/expert_layer.py [--tokens T] [--steps N]

Serving: the experts' weights are quantised to 8 bits once; every call routes
its tokens to k of E experts, sorts them, quantises the rows in expert order,
runs each expert's gate/up and down products in 8 bits and brings the rows
back, weighted.  The same calls serve a batch of prompts and a decoding step
of a few tokens.

Training: the same routing around 16-bit products of each expert, and the way
back: the gradient of the tokens, of the routing weights and of the experts'
weights.

Everything runs on the current stream; torch supplies memory, the router and,
for the check at the end, fp32 reference results.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_fp32_matrix_03_gb300 as lib  # noqa: E402


def pad16(n):
    return (n + 15) // 16 * 16


class ExpertWeights8:
    """E matrices (N x K) in 8-bit integers, rows padded to 16 bytes, with a
    scale for each row."""

    def __init__(self, w):
        self.E, self.N, self.K = w.shape
        self.ld = pad16(self.K)
        self.q = torch.zeros(self.E, self.N, self.ld, dtype=torch.int8, device=w.device)
        self.scale = torch.empty(self.E, self.N, device=w.device)
        w = w.contiguous()
        lib.check(lib.sgemm_i8_quantize_rows("bf16", "none", self.E * self.N, self.K, w, self.K,
                                             self.q, self.ld, self.scale))


class Routing:
    """A call's choices in expert order."""

    def __init__(self, ids, E):
        self.T, self.k = ids.shape
        self.E, self.S = E, ids.numel()
        i32 = dict(dtype=torch.int32, device=ids.device)
        self.ids = ids.to(torch.int32).contiguous()
        self.offsets = torch.empty(E + 1, **i32)
        self.slots, self.positions = torch.empty(self.S, **i32), torch.empty(self.S, **i32)
        lib.check(lib.sgemm_experts_sort(self.T, self.k, E, self.ids, self.offsets, self.slots,
                                         self.positions))


def serve(x, ids, weights, gate_up, down):
    """out[t] = sum_j weights[t, j] * down_e(silu(gate_e x) * up_e x), e = ids[t, j]."""
    T, H = x.shape
    r = Routing(ids, gate_up.E)
    dev, S, E, F = x.device, r.S, r.E, down.K
    q = torch.empty(S, gate_up.ld, dtype=torch.int8, device=dev)
    s = torch.empty(S, device=dev)
    lib.check(lib.sgemm_experts_dispatch_i8("bf16", T, r.k, E, H, x, H, r.positions, r.offsets, q,
                                            gate_up.ld, s))
    h = torch.zeros(S, 2 * F, dtype=torch.bfloat16, device=dev)
    lib.check(lib.sgemm_i8_experts("bf16", S, 2 * F, H, E, r.offsets, q, gate_up.ld, s, gate_up.q,
                                   gate_up.ld, gate_up.N * gate_up.ld, gate_up.scale, h, 2 * F))
    q = torch.empty(S, down.ld, dtype=torch.int8, device=dev)
    lib.check(lib.sgemm_i8_quantize_rows("bf16", "swiglu", S, F, h, 2 * F, q, down.ld, s))
    y = torch.empty(S, H, dtype=torch.bfloat16, device=dev)
    lib.check(lib.sgemm_i8_experts("bf16", S, H, F, E, r.offsets, q, down.ld, s, down.q, down.ld,
                                   down.N * down.ld, down.scale, y, H))
    out = torch.empty(T, H, dtype=torch.bfloat16, device=dev)
    lib.check(lib.sgemm_experts_combine("bf16", T, r.k, E, H, y, H, r.positions, r.offsets,
                                        weights, out, H))
    return out


def matmul16(a, b, trans_a=False, trans_b=False):
    """op(a) @ op(b) in fp32 from bf16 matrices."""
    M, K = (a.shape[1], a.shape[0]) if trans_a else a.shape
    N = b.shape[0] if trans_b else b.shape[1]
    c = torch.empty(M, N, device=a.device)
    lda, ldb = a.stride(0), b.stride(0)
    size = lib.sgemm_half_workspace_size("bf16", M, N, K, trans_a, trans_b, lda, ldb)
    # operands that do not start on 16 bytes are copied there as well
    size += 2 * (M + N) * (K + 64) + 512
    ws = torch.empty(size, dtype=torch.uint8, device=a.device)
    lib.check(lib.sgemm_half_batched("bf16", M, N, K, 1.0, a, lda, b, ldb, 0.0, c, N, trans_a,
                                     trans_b, 0, 0, 0, 1, ws, size))
    return c


def train_step(x, ids, weights, w, dout):
    """One linear expert layer out[t] = sum_j weights[t, j] * w[ids[t, j]] x[t]:
    out, and the gradients dx, dweights, dw for dout."""
    T, H = x.shape
    E, N, _ = w.shape
    r = Routing(ids, E)
    k, S, dev = r.k, r.S, x.device
    args = (r.positions, r.offsets)
    rows = torch.empty(S, H, dtype=torch.bfloat16, device=dev)
    lib.check(lib.sgemm_experts_dispatch("bf16", T, k, E, H, x, H, *args, rows, H))
    first = r.offsets.tolist()  # the products are launched expert by expert
    y = torch.zeros(S, N, dtype=torch.bfloat16, device=dev)
    for e in range(E):
        if first[e + 1] > first[e]:
            y[first[e]:first[e + 1]] = matmul16(rows[first[e]:first[e + 1]], w[e], trans_b=True)
    out = torch.empty(T, N, dtype=torch.bfloat16, device=dev)
    lib.check(lib.sgemm_experts_combine("bf16", T, k, E, N, y, N, *args, weights, out, N))

    dy = torch.empty_like(y)
    dweights = torch.empty(T, k, device=dev)
    lib.check(lib.sgemm_experts_combine_grad("bf16", T, k, E, N, dout, N, y, N, *args, weights,
                                             dy, N, dweights))
    drows = torch.zeros_like(rows)
    dw = torch.zeros(E, N, H, device=dev)
    for e in range(E):
        a, b = first[e], first[e + 1]
        if b > a:
            drows[a:b] = matmul16(dy[a:b], w[e])
            dw[e] = matmul16(dy[a:b], rows[a:b], trans_a=True)
    dx = torch.empty(T, H, dtype=torch.bfloat16, device=dev)
    lib.check(lib.sgemm_experts_dispatch_grad("bf16", T, k, E, H, drows, H, *args, dx, H))
    return out, dx, dweights, dw


def route(x, router, k):
    val, ids = torch.topk(x.float() @ router, k, dim=1)
    return ids, torch.softmax(val, dim=1)


def relative(a, b):
    return float((a.float() - b.float()).norm() / b.float().norm())


def main(tokens=512, steps=4, H=512, F=384, E=16, k=4):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=gen)
    router = rnd(H, E)
    gate_up = (rnd(E, 2 * F, H) / H ** 0.5).bfloat16()
    down = (rnd(E, H, F) / F ** 0.5).bfloat16()
    g8, d8 = ExpertWeights8(gate_up), ExpertWeights8(down)

    def reference(x, ids, weights):
        out = torch.zeros(x.shape, device="cuda")
        for e in range(E):
            for j in range(k):
                t = (ids[:, j] == e).nonzero()[:, 0]
                h = x[t].float() @ gate_up[e].float().t()
                h = torch.nn.functional.silu(h[:, :F]) * h[:, F:]
                out[t] += weights[t, j, None] * (h @ down[e].float().t())
        return out

    errors = {}
    x = rnd(tokens, H).bfloat16()
    ids, weights = route(x, router, k)
    errors["prompt"] = relative(serve(x, ids, weights, g8, d8), reference(x, ids, weights))
    worst = 0.0
    for _ in range(steps):  # decoding: three sequences, a token each
        x = rnd(3, H).bfloat16()
        ids, weights = route(x, router, k)
        worst = max(worst, relative(serve(x, ids, weights, g8, d8), reference(x, ids, weights)))
    errors["decoding"] = worst

    x, dout = rnd(tokens, H).bfloat16(), rnd(tokens, H).bfloat16()
    w = (rnd(E, H, H) / H ** 0.5).bfloat16()
    ids, weights = route(x, router, k)
    ids[0] = -1                      # a token over every expert's capacity
    out, dx, dweights, dw = train_step(x, ids, weights, w, dout)
    xr, wr, cr = (z.float().requires_grad_() for z in (x, w, weights))
    y = torch.einsum("th,enh->ten", xr, wr)
    kept = (ids >= 0)[:, :, None]
    picked = torch.gather(y, 1, ids.clamp(min=0)[:, :, None].expand(-1, -1, H))
    ref = (torch.where(kept, picked, 0.0) * cr[:, :, None]).sum(1)
    ref.backward(dout.float())
    for name, got, want in (("out", out, ref.detach()), ("dx", dx, xr.grad),
                            ("dweights", dweights, cr.grad), ("dw", dw, wr.grad)):
        errors[name] = relative(got, want)
    lib.check(lib.sgemm_poll_error())
    return errors


if __name__ == "__main__":
    p = argparse.ArgumentParser()
    p.add_argument("--tokens", type=int, default=512)
    p.add_argument("--steps", type=int, default=4)
    a = p.parse_args()
    for name, err in main(a.tokens, a.steps).items():
        print(f"{name:9s} relative error {err:.2e}")
