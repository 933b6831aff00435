"""Cases, plain forms and exact values of the operators around a feed-forward
block in few bits.

Six operators:

  norm    root-mean-square norm of a residual stream: the sum x + r, kept, and
          the normed row in the rows' own type
  norm8   the same, the normed row in 8-bit integers with one scale, as the
          8-bit products take it
  grad    the norm's way back: the stream's gradient and the weight's
  linear  a linear layer in 4-bit floating point with a scale for each block
          of values: the activations are quantised (as they are, after the
          gated activation, or by the norm itself) and multiplied by weights
          kept in 4 bits.  Format "nv": blocks of 16 with an e4m3 scale and a
          32-bit scale per row; "mx": blocks of 32 with a power of two
  product the product alone, of rows that are in 4 bits already
  layer   a whole expert layer for a few tokens: gate and value products,
          gated activation, product back and weighted sum, weights in 8 bits
          with a scale per channel or in 16 bits

`own` selects what run() calls: False, elementary torch operations in 32 bits;
True, this library's entry points.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
TINY = 2.0 ** -100  # a row whose largest magnitude is below this counts as zero
EPS = 1e-5
BLOCK = {"nv": 16, "mx": 32}
LEVELS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]  # magnitudes of the 4-bit codes


def listed():
    return [
        # one decoding step of eight sequences
        dict(name="norm_step", op="norm", type="bf16", M=8, H=4096),
        # sizes off every vector, 32-bit rows
        dict(name="norm_ragged", op="norm", type="fp32", M=777, H=1500),
        # a decoding batch, then a batch of prompts, before an 8-bit product
        dict(name="norm8_step", op="norm8", type="fp16", M=64, H=4096),
        dict(name="norm8_prompt", op="norm8", type="bf16", M=8192, H=4096),
        # a training micro-batch; a ragged one in 32 bits
        dict(name="grad_train", op="grad", type="bf16", M=8192, H=4096),
        dict(name="grad_ragged", op="grad", type="fp32", M=777, H=1500),
        # one token of one sequence through norm and a square layer
        dict(name="linear_token", op="linear", type="bf16", front="norm", format="nv", M=1,
             N=4096, K=4096),
        # a small decoding batch on the benchmark's odd edge, the layer after the activation
        dict(name="linear_few", op="linear", type="fp16", front="swiglu", format="mx", M=37,
             N=4092, K=4092),
        # a batch of prompts through a wide layer
        dict(name="product_prompt", op="product", type="bf16", format="nv", M=8192, N=8192,
             K=4096),
        # the ragged shape of the fp32 products
        dict(name="product_ragged", op="product", type="fp32", format="mx", M=1000, N=1500,
             K=777),
        # a decoding step of one sequence, 8-bit experts
        dict(name="layer_token", op="layer", type="fp16", weights="i8", T=1, k=4, E=32, H=2048,
             F=2048, drop=0.0),
        # a decoding step of 16 sequences, 16-bit experts
        dict(name="layer_step", op="layer", type="bf16", weights="same", T=16, k=4, E=32, H=2048,
             F=1024, drop=0.0),
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi, step):
    """As _log, every other time rounded to a multiple of `step`."""
    n = _log(rng, lo, hi)
    return n if rng.random() < 0.5 else min(hi, max(step, n // step * step))


def draw(rng):
    op = rng.choice(["norm", "norm8", "grad", "linear", "product", "layer"])
    type_ = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op in ("norm", "norm8", "grad"):
        return dict(op=op, type=type_, M=_log(rng, 1, 8192 if type_ != "fp32" else 4096),
                    H=_size(rng, 64, 4096, 64))
    if op == "layer":
        E = rng.choice([4, 8, 10, 16, 32, 60, 64])
        return dict(op=op, type=rng.choice(["bf16", "fp16"]), weights=rng.choice(["i8", "same"]),
                    T=_log(rng, 1, 32), k=rng.randint(1, 4), E=E, H=_size(rng, 64, 2048, 64),
                    F=_size(rng, 64, 2048, 64), drop=rng.choice([0.0, 0.0, 0.1]))
    case = dict(op=op, type=type_, format=rng.choice(["nv", "mx"]), M=_log(rng, 1, 8192),
                N=_size(rng, 64, 8192, 64), K=_size(rng, 64, 4096, 64))
    if op == "linear":
        # (the activation's codes hang on the last bits of exp: 16-bit results)
        case["front"] = rng.choice(["plain", "norm", "swiglu"])
        if case["front"] == "swiglu" and type_ == "fp32":
            case["type"] = "bf16"
        case["M"] = min(case["M"], 2048)
    return case


def _tokens(shape, gen):
    """Activations: normal values, each token with a size of its own."""
    x = torch.randn(*shape, device="cuda", generator=gen)
    x *= torch.exp(0.5 * torch.randn(shape[0], 1, device="cuda", generator=gen))
    return x


def _up(n, step):
    return (n + step - 1) // step * step


# ------------------------------------------------- the 4-bit format, on torch
#
# Codes: sign and three bits, LEVELS; two to a byte, the even one low; rows of
# a multiple of 16 bytes.  Block scales: tiles of 128 rows by four blocks, 512
# bytes each, tiles of a row block side by side; within a tile the byte of row
# r and block b is at 16 * (r % 32) + 4 * (r // 32) + b.

def _tile_scales(s):
    """(rows, blocks) bytes -> the tiled layout."""
    r, b = s.shape
    full = torch.zeros(_up(r, 128), _up(b, 4), dtype=torch.uint8, device=s.device)
    full[:r, :b] = s
    return full.view(-1, 4, 32, full.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)


def _untile_scales(t, rows, blocks):
    n = _up(blocks, 4)
    v = t.view(-1, n // 4, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, n)
    return v[:rows, :blocks]


def _decode(codes, K, dtype):
    """Packed bytes (rows, ld / 2) -> values (rows, K)."""
    table = torch.tensor(LEVELS + [-v for v in LEVELS], dtype=dtype, device=codes.device)
    both = torch.stack([codes & 15, codes >> 4], dim=2).view(codes.shape[0], -1)[:, :K]
    return table[both.long()] if both.numel() < 1 << 24 else table[both.int()]


def _scale_values(bytes_, format_, dtype):
    if format_ == "nv":
        return bytes_.contiguous().view(torch.float8_e4m3fn).to(dtype)
    return torch.exp2(bytes_.to(dtype) - 127)


def _dequantize(codes, tiled, format_, K, dtype):
    """The values that codes and block scales stand for."""
    blocks = -(-K // BLOCK[format_])
    s = _scale_values(_untile_scales(tiled, codes.shape[0], blocks), format_, dtype)
    s = s.repeat_interleave(BLOCK[format_], dim=1)[:, :K]
    return _decode(codes, K, dtype).mul_(s)


def _packed(rows, K, format_, gen):
    """Rows in 4 bits as weights or activations quantised beforehand have
    them: codes of normal values, block scales that differ by block, row
    scales."""
    ld = _up(K, 32)
    block = BLOCK[format_]
    v = (2.2 * torch.randn(rows, K, device="cuda", generator=gen)).abs_()
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    mag = torch.bucketize(v, edges, out_int32=True).to(torch.uint8)
    del v
    sign = (torch.rand(rows, K, device="cuda", generator=gen) < 0.5).to(torch.uint8) * 8
    full = torch.zeros(rows, ld, dtype=torch.uint8, device="cuda")
    full[:, :K] = mag + sign
    codes = (full[:, 0::2] | (full[:, 1::2] << 4)).contiguous()
    blocks = -(-K // block)
    if format_ == "nv":
        s = 60.0 * torch.exp(0.5 * torch.randn(rows, blocks, device="cuda", generator=gen))
        s = s.clamp_(0.02, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        s = torch.randint(120, 126, (rows, blocks), device="cuda", generator=gen).to(torch.uint8)
    row = (0.5 + torch.rand(rows, device="cuda", generator=gen)) / (60 if format_ == "nv" else 1)
    return dict(codes=codes, ld=ld, sf=_tile_scales(s), scale=row / math.sqrt(K) ** 0.5)


# ------------------------------------------------------------------- inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt, op = TYPES[case["type"]], case["op"]
    st = dict(case=case)

    def empty(*shape, dtype=dt):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    def weight(H):
        return (1 + 0.2 * torch.randn(H, device="cuda", generator=gen)).to(dt)

    if op in ("norm", "norm8", "grad"):
        M, H = case["M"], case["H"]
        st["x"] = _tokens((M, H), gen).to(dt)
        st["w"] = weight(H)
        if op == "grad":  # x is the kept sum
            st["dy"] = _tokens((M, H), gen).to(dt)
            st["ds"] = _tokens((M, H), gen).to(dt)
            st["dx"], st["dw"] = empty(M, H), empty(H, dtype=torch.float32)
            return st
        st["r"] = _tokens((M, H), gen).to(dt)
        st["s"] = empty(M, H)
        if op == "norm":
            st["y"] = empty(M, H)
        else:
            st["q"] = empty(M, _up(H, 16), dtype=torch.int8)
            st["sq"] = empty(M, dtype=torch.float32)
        return st
    if op in ("linear", "product"):
        M, N, K = case["M"], case["N"], case["K"]
        st["b"] = _packed(N, K, case["format"], gen)
        st["y"] = empty(M, N)
        if op == "product":
            st["a"] = _packed(M, K, case["format"], gen)
            return st
        st["x"] = _tokens((M, K * (2 if case["front"] == "swiglu" else 1)), gen).to(dt)
        if case["front"] == "norm":
            st["r"] = _tokens((M, K), gen).to(dt)
            st["w"], st["s"] = weight(K), empty(M, K)
        # what a user's program keeps between calls
        blocks = -(-K // BLOCK[case["format"]])
        st["q"] = torch.zeros(M, _up(K, 32) // 2, dtype=torch.uint8, device="cuda")
        st["sf"] = torch.zeros(_up(M, 128) * _up(blocks, 4), dtype=torch.uint8, device="cuda")
        st["sq"] = empty(M, dtype=torch.float32)
        return st
    T, k, E, H, F = (case[n] for n in ("T", "k", "E", "H", "F"))
    st["x"] = _tokens((T, H), gen).to(dt)
    logits = torch.randn(T, E, device="cuda", generator=gen)
    logits += 0.7 * torch.randn(E, device="cuda", generator=gen)
    val, ids = torch.topk(logits, k, dim=1)
    gone = torch.rand(T, k, device="cuda", generator=gen) < case["drop"]
    st["ids"] = torch.where(gone, -1, ids).to(torch.int32).contiguous()
    st["weights"] = torch.softmax(val, dim=1).contiguous()

    def experts(n, K):
        if case["weights"] == "same":
            ld = _up(K, 8)
            w = torch.zeros(E, n, ld, dtype=dt, device="cuda")
            w[:, :, :K] = (torch.randn(E, n, K, device="cuda", generator=gen) / math.sqrt(K)).to(dt)
            return w, ld, None
        ld = _up(K, 16)
        w = torch.zeros(E, n, ld, dtype=torch.int8, device="cuda")
        for e in range(E):
            w[e, :, :K] = (40 * torch.randn(n, K, device="cuda", generator=gen)).round_() \
                .clamp_(-127, 127).to(torch.int8)
        return w, ld, (0.5 + torch.rand(E, n, device="cuda", generator=gen)) / (40 * math.sqrt(K))

    st["w1"], st["ld1"], st["s1"] = experts(2 * F, H)
    st["w2"], st["ld2"], st["s2"] = experts(H, F)
    st["out"] = empty(T, H)
    return st


# ------------------------------------------------------------- plain forms

def _plain_sum(st, dt):
    """The residual stream's row as it is kept, and 1 / its rms."""
    s = (st["x"].float() + st["r"].float()).to(dt)
    f = s.float()
    return s, f, torch.rsqrt((f * f).mean(1, keepdim=True) + EPS)


def _plain_round4(u):
    """The nearest 4-bit value, ties to the code whose last bit is zero."""
    a = u.abs().clamp(max=6.0)
    small = torch.round(a * 2) / 2
    mid = torch.round(a)
    big = torch.round(a / 2) * 2
    return torch.copysign(torch.where(a < 2, small, torch.where(a < 4, mid, big)), u)


def _plain_quantize4(v, format_):
    """Rows quantised to 4 bits: the values that codes and block scales stand
    for, and the row's scale."""
    M, K = v.shape
    block = BLOCK[format_]
    pad = _up(K, block) - K
    b = torch.nn.functional.pad(v, (0, pad)).view(M, -1, block)
    amax = b.abs().amax(2)
    if format_ == "mx":
        _, e = torch.frexp(amax)  # amax in [2^(e-1), 2^e)
        e = torch.where(amax > 0, e - 3, -127).clamp(-127, 127)
        sf = torch.ldexp(torch.ones_like(amax), e)
        u = torch.ldexp(b, -e[:, :, None])
        return (_plain_round4(u) * sf[:, :, None]).view(M, -1)[:, :K], torch.ones_like(v[:, 0])
    row = amax.amax(1)
    zero = row < TINY
    safe = torch.where(zero, torch.ones_like(row), row)
    sf = (amax * (torch.full_like(row, 448.0) / safe)[:, None]).clamp(max=448.0) \
        .to(torch.float8_e4m3fn).float()
    up = (torch.full_like(row, 2688.0) / safe)[:, None] / sf
    up = torch.where((sf > 0) & ~zero[:, None], up, torch.zeros_like(up))
    val = _plain_round4(b * up[:, :, None]) * sf[:, :, None]
    scale = torch.where(zero, torch.zeros_like(row), row / torch.full_like(row, 2688.0))
    return val.view(M, -1)[:, :K], scale


def _run_plain(st):
    case = st["case"]
    op, dt = case["op"], TYPES[case["type"]]
    if op == "norm":
        s, f, rho = _plain_sum(st, dt)
        return s, (f * rho * st["w"].float()).to(dt)
    if op == "norm8":
        s, f, rho = _plain_sum(st, dt)
        v = f * st["w"].float()
        amax = v.abs().amax(1)
        zero = amax < TINY
        full = torch.full_like(amax, 127.0)
        inv = torch.where(zero, torch.zeros_like(amax), full / amax)
        q = torch.round(v * inv[:, None]).to(torch.int8)
        return s, q, torch.where(zero, torch.zeros_like(amax), amax / full * rho[:, 0])
    if op == "grad":
        s, dy, w = st["x"].float(), st["dy"].float(), st["w"].float()
        rho = torch.rsqrt((s * s).mean(1, keepdim=True) + EPS)
        m = (w * dy * s).mean(1, keepdim=True)
        dx = st["ds"].float() + rho * (w * dy - s * (rho * rho * m))
        return dx.to(dt), (dy * s * rho).sum(0)
    if op in ("linear", "product"):
        K, format_ = case["K"], case["format"]
        s = None
        if op == "product":
            a = _dequantize(st["a"]["codes"], st["a"]["sf"], format_, K, torch.float32)
            sa = st["a"]["scale"]
        elif case["front"] == "norm":
            s, f, rho = _plain_sum(st, dt)
            a, sa = _plain_quantize4(f * st["w"].float(), format_)
            sa = sa * rho[:, 0]
        else:
            v = st["x"].float()
            if case["front"] == "swiglu":
                g = v[:, :K]
                v = g / (1 + torch.exp(-g)) * v[:, K:]
            a, sa = _plain_quantize4(v, format_)
        b = _dequantize(st["b"]["codes"], st["b"]["sf"], format_, K, torch.float32)
        y = ((a @ b.t()) * sa[:, None] * st["b"]["scale"][None, :]).to(dt)
        return y if s is None else (y, s)
    T, k, H, F = (case[n] for n in ("T", "k", "H", "F"))
    x = st["x"].float()
    ids = st["ids"].long()
    out = torch.zeros(T, H, device=x.device)
    for j in range(k):
        e = ids[:, j].clamp(min=0)
        w1, w2 = st["w1"][e, :, :H].float(), st["w2"][e, :, :F].float()
        if st["s1"] is not None:
            w1, w2 = w1 * st["s1"][e][:, :, None], w2 * st["s2"][e][:, :, None]
        gu = torch.bmm(w1, x[:, :, None])[:, :, 0]
        g = gu[:, :F]
        y = torch.bmm(w2, (g / (1 + torch.exp(-g)) * gu[:, F:])[:, :, None])[:, :, 0]
        out += torch.where((ids[:, j] >= 0)[:, None], st["weights"][:, j, None] * y, 0.0)
    return out.to(dt)


# ------------------------------------------------ the library's entry points

def _workspace(st, size):
    """The call's workspace, allocated once and kept as a user's program keeps it."""
    if "ws" not in st:
        st["ws"] = torch.empty(max(1, size), dtype=torch.uint8, device="cuda")
    return st["ws"]


def _run_own(st):
    import dense_fp32_matrix_03_gb300 as lib
    case = st["case"]
    op, type_ = case["op"], case["type"]
    if op == "norm":
        M, H = case["M"], case["H"]
        lib.check(lib.sgemm_rms_norm(type_, M, H, EPS, st["x"], H, st["r"], H, st["w"], st["s"],
                                     H, st["y"], H))
        return st["s"], st["y"]
    if op == "norm8":
        M, H = case["M"], case["H"]
        lib.check(lib.sgemm_rms_norm_i8(type_, M, H, EPS, st["x"], H, st["r"], H, st["w"],
                                        st["s"], H, st["q"], st["q"].shape[1], st["sq"]))
        return st["s"], st["q"][:, :H], st["sq"]
    if op == "grad":
        M, H = case["M"], case["H"]
        ws = _workspace(st, lib.sgemm_rms_norm_grad_workspace_size(M, H))
        lib.check(lib.sgemm_rms_norm_grad(type_, M, H, EPS, st["x"], H, st["w"], st["dy"], H,
                                          st["ds"], H, st["dx"], H, st["dw"], ws, ws.numel()))
        return st["dx"], st["dw"]
    if op in ("linear", "product"):
        M, N, K, format_ = case["M"], case["N"], case["K"], case["format"]
        b = st["b"]
        if op == "product":
            a = st["a"]
            lib.check(lib.sgemm_fp4(type_, format_, M, N, K, a["codes"], a["ld"], a["sf"],
                                    a["scale"], b["codes"], b["ld"], b["sf"], b["scale"],
                                    st["y"], N))
            return st["y"]
        ldq = 2 * st["q"].shape[1]
        if case["front"] == "norm":
            lib.check(lib.sgemm_rms_norm_fp4(type_, format_, M, K, EPS, st["x"], K, st["r"], K,
                                             st["w"], st["s"], K, st["q"], ldq, st["sf"],
                                             st["sq"]))
        else:
            act = "swiglu" if case["front"] == "swiglu" else "none"
            lib.check(lib.sgemm_fp4_quantize_rows(type_, act, format_, M, K, st["x"],
                                                  st["x"].shape[1], st["q"], ldq, st["sf"],
                                                  st["sq"]))
        lib.check(lib.sgemm_fp4(type_, format_, M, N, K, st["q"], ldq, st["sf"], st["sq"],
                                b["codes"], b["ld"], b["sf"], b["scale"], st["y"], N))
        return (st["y"], st["s"]) if case["front"] == "norm" else st["y"]
    T, k, E, H, F = (case[n] for n in ("T", "k", "E", "H", "F"))
    ws = _workspace(st, lib.sgemm_experts_layer_workspace_size(T, k, H, F))
    lib.check(lib.sgemm_experts_layer(type_, case["weights"], T, k, E, H, F, st["x"], H, st["ids"],
                                      st["weights"], st["w1"], st["ld1"], 2 * F * st["ld1"],
                                      st["s1"], st["w2"], st["ld2"], H * st["ld2"], st["s2"],
                                      st["out"], H, ws, ws.numel()))
    return st["out"]


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------- floors

def work(case):
    op, es = case["op"], SIZE[case["type"]]
    if op in ("norm", "norm8", "grad"):
        M, H = case["M"], case["H"]
        if op == "norm":
            return dict(bytes=4 * M * H * es + H * es, flops=5 * M * H)
        if op == "norm8":
            return dict(bytes=3 * M * H * es + M * H + H * es + 4 * M, flops=6 * M * H)
        return dict(bytes=4 * M * H * es + H * (es + 4), flops=11 * M * H)
    if op in ("linear", "product"):
        M, N, K = case["M"], case["N"], case["K"]
        bits = 4 + 8 / BLOCK[case["format"]]
        b = N * K * bits / 8 + 4 * N + M * N * es
        if op == "product":
            b += M * K * bits / 8 + 4 * M
        else:
            b += M * K * es * {"plain": 1, "swiglu": 2, "norm": 3}[case["front"]]
        return dict(bytes=int(b), flops=2 * M * N * K)
    T, k, E, H, F = (case[n] for n in ("T", "k", "E", "H", "F"))
    live = T * k * (1 - case["drop"])
    used = E * (1 - (1 - 1 / E) ** live) if T > 1 else min(E, live)  # experts with a token
    each = 3 * H * F * (1 if case["weights"] == "i8" else 2)
    if case["weights"] == "i8":
        each += 4 * (2 * F + H)
    return dict(bytes=int(used * each + 2 * T * H * es + 8 * T * k), flops=int(6 * live * H * F))


# -------------------------------------------------------------- exact values

def exact(case, seed):
    """The definitions in 64 bits (codes included: a value next to a border may
    take the other code there)."""
    st = prepare(case, seed)
    op, f64 = case["op"], torch.float64

    def round4(u):
        grid = torch.tensor(LEVELS, dtype=f64, device=u.device)
        border = (grid[1:] + grid[:-1]) / 2
        a = u.abs()
        lo = torch.bucketize(a, border, right=False, out_int32=True)  # borders go down
        hi = torch.bucketize(a, border, right=True, out_int32=True)   # borders go up
        code = torch.where(lo % 2 == 0, lo, hi)
        return grid[code] * torch.sign(u)

    def quantize(v):
        M, K = v.shape
        n = BLOCK[case["format"]]
        val = torch.zeros_like(v)
        row = v.abs().max(dim=1, keepdim=True).values
        scale = torch.ones_like(row) if case["format"] == "mx" else row / 2688
        for k0 in range(0, K, n):
            part = v[:, k0:k0 + n]
            top = part.abs().max(dim=1, keepdim=True).values
            if case["format"] == "mx":
                e = torch.floor(torch.log2(torch.where(top > 0, top, 1.0))) - 2
                sf = torch.exp2(e)
            else:
                sf = (448 * top / torch.where(row > 0, row, 1.0)).float() \
                    .to(torch.float8_e4m3fn).to(f64)
            on = (sf > 0) & (scale > 0)
            div = torch.where(on, sf * scale, 1.0)
            val[:, k0:k0 + n] = torch.where(on, round4(part / div) * sf, 0.0)
        return val, scale[:, 0]

    def stream():
        s = (st["x"].to(f64) + st["r"].to(f64)).to(TYPES[case["type"]])
        d = s.to(f64)
        return s, d, 1 / torch.sqrt(d.pow(2).sum(1) / d.shape[1] + EPS)

    if op == "norm":
        s, d, rho = stream()
        return s, torch.einsum("mh,m,h->mh", d, rho, st["w"].to(f64))
    if op == "norm8":
        s, d, rho = stream()
        v = d * st["w"].to(f64)
        top = v.abs().max(dim=1).values
        q = torch.round(v / torch.where(top > 0, top, 1.0)[:, None] * 127).to(torch.int8)
        return s, q, top * rho / 127
    if op == "grad":
        s, dy, w = st["x"].to(f64), st["dy"].to(f64), st["w"].to(f64)
        rho = 1 / torch.sqrt(s.pow(2).sum(1) / s.shape[1] + EPS)
        n, g = s * rho[:, None], dy * w
        inner = torch.einsum("mh,mh->m", g, n) / s.shape[1]
        return st["ds"].to(f64) + rho[:, None] * (g - n * inner[:, None]), \
            torch.einsum("mh,mh->h", dy, n)
    if op in ("linear", "product"):
        K, format_ = case["K"], case["format"]
        s = None
        if op == "product":
            a = _dequantize(st["a"]["codes"], st["a"]["sf"], format_, K, f64)
            sa = st["a"]["scale"].to(f64)
        elif case["front"] == "norm":
            s, d, rho = stream()
            a, sa = quantize(d * st["w"].to(f64))
            sa = sa * rho
        else:
            v = st["x"].to(f64)
            if case["front"] == "swiglu":
                v = v[:, :K] * torch.sigmoid(v[:, :K]) * v[:, K:]
            a, sa = quantize(v)
        b = _dequantize(st["b"]["codes"], st["b"]["sf"], format_, K, f64)
        y = (a @ b.t()).mul_(sa[:, None]).mul_(st["b"]["scale"].to(f64))
        return y if s is None else (y, s)
    T, H, F = case["T"], case["H"], case["F"]
    x, ids, wts = st["x"].to(f64), st["ids"].tolist(), st["weights"].to(f64)
    out = torch.zeros(T, H, dtype=f64, device="cuda")
    for e in range(case["E"]):
        at = [(t, j) for t in range(T) for j in range(case["k"]) if ids[t][j] == e]
        if not at:
            continue
        w1, w2 = st["w1"][e, :, :H].to(f64), st["w2"][e, :, :F].to(f64)
        if st["s1"] is not None:
            w1, w2 = w1 * st["s1"][e].to(f64)[:, None], w2 * st["s2"][e].to(f64)[:, None]
        for t, j in at:
            gu = w1 @ x[t]
            out[t] += wts[t, j] * (w2 @ (gu[:F] * torch.sigmoid(gu[:F]) * gu[F:]))
    return out
