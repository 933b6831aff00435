"""A transformer's feed-forward block on this library's entry points, served in
few bits and trained.

    python examples/feed_forward.py [--tokens T] [--steps N]

Serving, dense: the residual stream is added up, normed and quantised to 4 bits
in one pass, multiplied by gate and up weights kept in 4 bits; the gated
activation is quantised in one pass and multiplied by the down weights.  The same
calls serve a batch of prompts and a decoding step.

Serving, experts: for a decoding step of a few tokens, the norm in the rows' own
type and the whole expert layer, routed and weighted, in two kernels.

Training: the norm and a 16-bit product, and the way back: the gradient of the
residual stream, of the norm's weight and of the product's.

Everything runs on the current stream; torch supplies memory, the router and,
for the checks, fp32 reference results.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_fp32_matrix_03_gb300 as lib  # noqa: E402

EPS = 1e-5


def up(n, step):
    return (n + step - 1) // step * step


class Rows4:
    """M rows of K values in 4 bits: codes, block scales and row scales."""

    def __init__(self, M, K, format_, device):
        self.M, self.K, self.format_ = M, K, format_
        self.ld = up(K, 32)
        self.codes = torch.empty(M, self.ld // 2, dtype=torch.uint8, device=device)
        self.sf = torch.empty(lib.sgemm_fp4_scales_size(format_, M, K), dtype=torch.uint8,
                              device=device)
        self.scale = torch.empty(M, device=device)

    @classmethod
    def of(cls, x, format_, act="none"):
        """x (bf16) quantised; with act "swiglu" its gated activation."""
        r = cls(x.shape[0], x.shape[1] // (2 if act == "swiglu" else 1), format_, x.device)
        lib.check(lib.sgemm_fp4_quantize_rows("bf16", act, format_, r.M, r.K, x, x.stride(0),
                                              r.codes, r.ld, r.sf, r.scale))
        return r

    def times(self, w):
        """These rows times the transpose of w's, in bf16."""
        y = torch.empty(self.M, w.M, dtype=torch.bfloat16, device=self.codes.device)
        lib.check(lib.sgemm_fp4("bf16", self.format_, self.M, w.M, self.K, self.codes, self.ld,
                                self.sf, self.scale, w.codes, w.ld, w.sf, w.scale, y, w.M))
        return y


def serve_dense(x, res, norm_weight, gate_up, down):
    """(block's output, residual stream): weights in 4 bits."""
    M, H = x.shape
    s = torch.empty_like(x)
    a = Rows4(M, H, gate_up.format_, x.device)
    lib.check(lib.sgemm_rms_norm_fp4("bf16", a.format_, M, H, EPS, x, H, res, H, norm_weight, s, H,
                                     a.codes, a.ld, a.sf, a.scale))
    return Rows4.of(a.times(gate_up), down.format_, "swiglu").times(down), s


class Experts8:
    """E matrices (N x K) in 8-bit integers, rows padded to 16 bytes, with a
    scale for each row."""

    def __init__(self, w):
        self.E, self.N, self.K = w.shape
        self.ld = up(self.K, 16)
        self.q = torch.zeros(self.E, self.N, self.ld, dtype=torch.int8, device=w.device)
        self.scale = torch.empty(self.E, self.N, device=w.device)
        lib.check(lib.sgemm_i8_quantize_rows("bf16", "none", self.E * self.N, self.K,
                                             w.contiguous(), self.K, self.q, self.ld, self.scale))


def serve_experts(x, res, norm_weight, ids, weights, gate_up, down, workspace):
    """(block's output, residual stream) of a few tokens: experts in 8 bits."""
    T, H = x.shape
    s, y, out = (torch.empty_like(x) for _ in range(3))
    lib.check(lib.sgemm_rms_norm("bf16", T, H, EPS, x, H, res, H, norm_weight, s, H, y, H))
    lib.check(lib.sgemm_experts_layer("bf16", "i8", T, ids.shape[1], gate_up.E, H, down.K, y, H,
                                      ids, weights, gate_up.q, gate_up.ld,
                                      gate_up.N * gate_up.ld, gate_up.scale, down.q, down.ld,
                                      down.N * down.ld, down.scale, out, H, workspace,
                                      workspace.numel()))
    return out, s


def matmul16(a, b, trans_a=False, trans_b=False):
    """op(a) @ op(b) in fp32 from bf16 matrices."""
    M, K = (a.shape[1], a.shape[0]) if trans_a else a.shape
    N = b.shape[0] if trans_b else b.shape[1]
    c = torch.empty(M, N, device=a.device)
    size = lib.sgemm_half_workspace_size("bf16", M, N, K, trans_a, trans_b, a.stride(0),
                                         b.stride(0))
    ws = torch.empty(max(size, 1), dtype=torch.uint8, device=a.device)
    lib.check(lib.sgemm_half_batched("bf16", M, N, K, 1.0, a, a.stride(0), b, b.stride(0), 0.0, c,
                                     N, trans_a, trans_b, 0, 0, 0, 1, ws, size))
    return c


def train_step(x, res, norm_weight, w, dout, dstream):
    """out = norm(x + res) w^T and the kept stream; the gradients of x (and res),
    of the norm's weight and of w, for dout and the stream's own gradient."""
    M, H = x.shape
    s, y, dx = (torch.empty_like(x) for _ in range(3))
    lib.check(lib.sgemm_rms_norm("bf16", M, H, EPS, x, H, res, H, norm_weight, s, H, y, H))
    out = matmul16(y, w, trans_b=True)
    dw = matmul16(dout, y, trans_a=True)
    dy = matmul16(dout, w).bfloat16()
    dnorm = torch.empty(H, device=x.device)
    size = lib.sgemm_rms_norm_grad_workspace_size(M, H)
    ws = torch.empty(size, dtype=torch.uint8, device=x.device)
    lib.check(lib.sgemm_rms_norm_grad("bf16", M, H, EPS, s, H, norm_weight, dy, H, dstream, H, dx,
                                      H, dnorm, ws, size))
    return out, s, dx, dnorm, dw


def norm_reference(s, weight):
    return s * torch.rsqrt((s * s).mean(-1, keepdim=True) + EPS) * weight


def relative(a, b):
    return float((a.float() - b.float()).norm() / b.float().norm())


def main(tokens=512, steps=4, H=512, F=768, E=16, k=4):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    norm_weight = (1 + 0.2 * rnd(H)).bfloat16()
    gate_up, down = (rnd(2 * F, H) / H ** 0.5).bfloat16(), (rnd(H, F) / F ** 0.5).bfloat16()
    errors = {}

    def swiglu(h):
        return torch.nn.functional.silu(h[..., :F]) * h[..., F:]

    for format_ in ("nv", "mx"):
        g4, d4 = Rows4.of(gate_up, format_), Rows4.of(down, format_)
        for name, M in (("prompt", tokens), ("decoding", 3)):
            x, res = rnd(M, H).bfloat16(), rnd(M, H).bfloat16()
            out, s = serve_dense(x, res, norm_weight, g4, d4)
            y = norm_reference(s.float(), norm_weight.float())
            ref = swiglu(y @ gate_up.float().t()) @ down.float().t()
            errors[f"{format_} {name}"] = relative(out, ref)

    router = rnd(H, E)
    eg, ed = (rnd(E, 2 * F, H) / H ** 0.5).bfloat16(), (rnd(E, H, F) / F ** 0.5).bfloat16()
    g8, d8 = Experts8(eg), Experts8(ed)
    T = 3
    ws = torch.empty(lib.sgemm_experts_layer_workspace_size(T, k, H, F), dtype=torch.uint8,
                     device="cuda")
    worst = 0.0
    x, res = rnd(T, H).bfloat16(), torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    for _ in range(steps):  # decoding: three sequences, a token each
        val, ids = torch.topk((x + res).float() @ router, k, dim=1)
        weights = torch.softmax(val, dim=1)
        out, s = serve_experts(x, res, norm_weight, ids.to(torch.int32), weights, g8, d8, ws)
        y = norm_reference(s.float(), norm_weight.float()).bfloat16().float()
        ref = torch.zeros(T, H, device="cuda")
        for t in range(T):
            for j in range(k):
                e = ids[t, j]
                ref[t] += weights[t, j] * (ed[e].float() @ swiglu(eg[e].float() @ y[t]))
        worst = max(worst, relative(out, ref))
        x, res = out, s
    errors["experts"] = worst

    w = (rnd(H, H) / H ** 0.5).bfloat16()
    x, res, dout, dstream = (rnd(tokens, H).bfloat16() for _ in range(4))
    out, s, dx, dnorm, dw = train_step(x, res, norm_weight, w, dout, dstream)
    sr, nr, wr = (z.float().requires_grad_() for z in (s, norm_weight, w))
    ref = norm_reference(sr, nr) @ wr.t()
    ((ref * dout.float()).sum() + (sr * dstream.float()).sum()).backward()
    for name, got, want in (("out", out, ref.detach()), ("dx", dx, sr.grad),
                            ("dnorm", dnorm, nr.grad), ("dw", dw, wr.grad)):
        errors[name] = relative(got, want)
    lib.check(lib.sgemm_poll_error())
    return errors


if __name__ == "__main__":
    p = argparse.ArgumentParser()
    p.add_argument("--tokens", type=int, default=512)
    p.add_argument("--steps", type=int, default=4)
    a = p.parse_args()
    for name, err in main(a.tokens, a.steps).items():
        print(f"{name:12s} relative error {err:.2e}")
