"""Cases, plain forms and exact values of the 8-bit product and expert operators.

Five operators of an expert layer and of linear layers served in 8 bits:

  route    token-to-expert choices -> rows sorted by expert (stable), the
           order both ways and each expert's first row
  combine  expert rows back to their tokens, weighted and summed
  grad     the gradients of both (a training step's way back)
  product  a linear layer in 8 bits: each token's row is quantised to 8-bit
           integers with one scale, then multiplied by 8-bit weights with a
           scale for each channel
  experts  the same for an expert layer: choices -> sort -> rows quantised in
           expert order -> each expert's own product

`own` selects what run() calls: False, elementary torch operations in 32 bits;
True, this library's entry points.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
TINY = 2.0 ** -100  # a row whose largest magnitude is below this counts as zero


def listed():
    return [
        # one decoding step of eight sequences
        dict(name="route_step", op="route", type="bf16", T=8, k=4, E=32, H=2048, drop=0.0),
        # a batch of prompts, many small experts
        dict(name="route_prompt", op="route", type="bf16", T=8192, k=8, E=64, H=4096, drop=0.0),
        # a decoding step of 64 sequences, few large experts
        dict(name="combine_step", op="combine", type="fp16", T=64, k=2, E=8, H=4096, drop=0.0),
        dict(name="combine_prompt", op="combine", type="bf16", T=8192, k=8, E=64, H=4096,
             drop=0.0),
        # sizes off every tile, a quarter of the choices dropped (experts over capacity)
        dict(name="grad_ragged", op="grad", type="fp32", T=777, k=3, E=10, H=1500, drop=0.25),
        # a training micro-batch
        dict(name="grad_train", op="grad", type="bf16", T=8192, k=4, E=64, H=2048, drop=0.05),
        # one token of one sequence through a square layer
        dict(name="product_token", op="product", type="bf16", M=1, N=4096, K=4096),
        # a small decoding batch on the benchmark's odd edge
        dict(name="product_few", op="product", type="fp16", M=37, N=4092, K=4092),
        # the ragged shape of the fp32 products
        dict(name="product_ragged", op="product", type="fp32", M=1000, N=1500, K=777),
        # a batch of prompts through a wide layer
        dict(name="product_prompt", op="product", type="bf16", M=8192, N=8192, K=4096),
        # a decoding step: a few rows for each expert, bound by the weights
        dict(name="experts_step", op="experts", type="bf16", T=16, k=4, E=32, K=2048, N=2048,
             drop=0.0),
        # prompts: hundreds of rows for each expert, unevenly
        dict(name="experts_prompt", op="experts", type="bf16", T=8192, k=4, E=32, K=2048, N=4096,
             drop=0.0),
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi, step):
    """As _log, every other time rounded to a multiple of `step`."""
    n = _log(rng, lo, hi)
    return n if rng.random() < 0.5 else min(hi, max(step, n // step * step))


def draw(rng):
    op = rng.choice(["route", "combine", "grad", "product", "experts"])
    type_ = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    tokens = _log(rng, 1, 8192 if type_ != "fp32" else 4096)  # fp32 rows are twice as long
    if op == "product":
        return dict(op=op, type=type_, M=tokens, N=_size(rng, 64, 8192, 64),
                    K=_size(rng, 64, 4096, 64))
    E = rng.choice([4, 8, 10, 16, 32, 60, 64, 128])
    k = rng.randint(1, min(8, E))
    drop = rng.choice([0.0, 0.0, 0.05, 0.3])
    if op == "experts":
        return dict(op=op, type=type_, T=tokens, k=min(k, 4), E=min(E, 64), K=_size(rng, 64, 2048, 64),
                    N=_size(rng, 64, 4096, 64), drop=drop)
    if op == "grad":  # moves three times the rows of one way
        return dict(op=op, type=type_, T=tokens, k=min(k, 4), E=E, H=_size(rng, 64, 2048, 64),
                    drop=drop)
    return dict(op=op, type=type_, T=tokens, k=k, E=E, H=_size(rng, 64, 4096, 64), drop=drop)


def _choices(case, gen):
    """A router's choices: k different experts a token, some experts chosen
    more often than others, dropped ones -1; and their weights."""
    T, k, E = case["T"], case["k"], case["E"]
    logits = torch.randn(T, E, device="cuda", generator=gen)
    logits += 0.7 * torch.randn(E, device="cuda", generator=gen)
    val, ids = torch.topk(logits, k, dim=1)
    weights = torch.softmax(val, dim=1)
    gone = torch.rand(T, k, device="cuda", generator=gen) < case["drop"]
    ids = torch.where(gone, -1, ids).to(torch.int32).contiguous()
    return ids, weights.contiguous()


def _order(ids, E):
    """Offsets, slots and positions of the stable sort by expert, dropped
    choices last."""
    key = ids.reshape(-1).long()
    key = torch.where((key < 0) | (key >= E), E, key)
    slots = torch.argsort(key, stable=True)
    positions = torch.empty_like(slots)
    positions[slots] = torch.arange(slots.numel(), device="cuda")
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(torch.bincount(key, minlength=E + 1)[:E], 0)
    return offsets, slots.to(torch.int32), positions.to(torch.int32)


def _tokens(shape, gen):
    """Activations: normal values, each token with a size of its own."""
    x = torch.randn(*shape, device="cuda", generator=gen)
    x *= torch.exp(0.5 * torch.randn(shape[0], 1, device="cuda", generator=gen))
    return x


def _pad16(n):
    return (n + 15) // 16 * 16


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = TYPES[case["type"]]
    op = case["op"]
    st = dict(case=case)
    if op == "product":
        M, N, K = case["M"], case["N"], case["K"]
        st["x"] = _tokens((M, K), gen).to(dt)
        groups = (1, N, K)
    elif op == "experts":
        st["ids"], _ = _choices(case, gen)
        st["x"] = _tokens((case["T"], case["K"]), gen).to(dt)
        M, N, K = case["T"] * case["k"], case["N"], case["K"]
        groups = (case["E"], N, K)
    if op in ("product", "experts"):
        # weights and their scales, laid out once: rows padded to 16 bytes
        E, N, K = groups
        ld = _pad16(K)
        w = torch.zeros(E, N, ld, dtype=torch.int8, device="cuda")
        for e in range(E):
            w[e, :, :K] = (40 * torch.randn(N, K, device="cuda", generator=gen)).round_() \
                .clamp_(-127, 127).to(torch.int8)
        st["w"], st["ldw"] = w, ld
        st["sw"] = (0.5 + torch.rand(E, N, device="cuda", generator=gen)) / (40 * math.sqrt(K))
        # what a user's program keeps between calls
        st["q"] = torch.zeros(max(M, 1), ld, dtype=torch.int8, device="cuda")
        st["sq"] = torch.zeros(M, device="cuda")
        st["y"] = torch.zeros(M, N, dtype=dt, device="cuda")
    else:
        T, k, E, H = case["T"], case["k"], case["E"], case["H"]
        st["ids"], st["weights"] = _choices(case, gen)
        if op == "route":
            st["x"] = _tokens((T, H), gen).to(dt)
            st["rows"] = torch.empty(T * k, H, dtype=dt, device="cuda")
        else:
            st["offsets"], st["slots"], st["positions"] = _order(st["ids"], E)
            st["rows"] = _tokens((T * k, H), gen).to(dt)
            if op == "combine":
                st["out"] = torch.empty(T, H, dtype=dt, device="cuda")
            else:
                st["dout"] = _tokens((T, H), gen).to(dt)
                st["dxrows"] = _tokens((T * k, H), gen).to(dt)
                st["drows"] = torch.empty_like(st["rows"])
                st["dweights"] = torch.empty(T, k, device="cuda")
                st["dx"] = torch.empty(T, H, dtype=dt, device="cuda")
    if op in ("route", "experts"):
        S = case["T"] * case["k"]
        st["offsets"] = torch.empty(case["E"] + 1, dtype=torch.int32, device="cuda")
        st["slots"] = torch.empty(S, dtype=torch.int32, device="cuda")
        st["positions"] = torch.empty(S, dtype=torch.int32, device="cuda")
    return st


# ------------------------------------------------------------- plain forms

def _plain_sort(ids, E):
    """The stable sort by counting: a choice's position is its expert's first
    row plus the earlier choices of the same expert."""
    key = ids.reshape(-1).long()
    key = torch.where((key < 0) | (key >= E), E, key)
    hot = (key[:, None] == torch.arange(E + 1, device=key.device)[None, :]).to(torch.int32)
    run_ = torch.cumsum(hot, 0, dtype=torch.int32)
    ends = torch.cumsum(run_[-1], 0, dtype=torch.int32)
    offsets = torch.cat([torch.zeros(1, dtype=torch.int32, device=key.device), ends[:E]])
    rank = torch.gather(run_, 1, key[:, None])[:, 0] - 1
    positions = offsets[key] + rank
    slots = torch.empty_like(positions)
    slots[positions.long()] = torch.arange(key.numel(), dtype=torch.int32, device=key.device)
    return offsets, slots, positions


def _plain_quantize(x):
    """Codes (as 32-bit floats) and scales of each row."""
    amax = x.abs().amax(1)
    full = torch.full_like(amax, 127.0)
    zero = amax < TINY
    q = torch.round(x * torch.where(zero, torch.zeros_like(amax), full / amax)[:, None])
    return q, torch.where(zero, torch.zeros_like(amax), amax / full)


def _plain_rows(x, slots, offsets, k):
    rows = x[slots.long() // k]
    live = torch.arange(rows.shape[0], device=x.device) < offsets[-1]
    return torch.where(live[:, None], rows, torch.zeros_like(rows))


def _run_plain(st):
    case = st["case"]
    op, dt = case["op"], TYPES[case["type"]]
    if op == "product":
        q, s = _plain_quantize(st["x"].float())
        w = st["w"][0, :, :case["K"]].float()
        return ((q @ w.t()) * s[:, None] * st["sw"][0][None, :]).to(dt)
    if op == "experts":
        E, K = case["E"], case["K"]
        offsets, slots, positions = _plain_sort(st["ids"], E)
        q, s = _plain_quantize(_plain_rows(st["x"].float(), slots, offsets, case["k"]))
        y = torch.zeros(q.shape[0], case["N"], dtype=dt, device=q.device)
        first = offsets.tolist()
        for e in range(E):
            a, b = first[e], first[e + 1]
            if b > a:
                acc = q[a:b] @ st["w"][e, :, :K].float().t()
                y[a:b] = (acc * s[a:b, None] * st["sw"][e][None, :]).to(dt)
        return y, offsets, slots, positions
    k, E = case["k"], case["E"]
    if op == "route":
        offsets, slots, positions = _plain_sort(st["ids"], E)
        return _plain_rows(st["x"], slots, offsets, k), offsets, slots, positions
    pos = st["positions"].long().view(case["T"], k)
    live = (pos < st["offsets"][-1])[:, :, None]
    picked = torch.where(live, st["rows"].float()[pos], 0.0)
    if op == "combine":
        return (picked * st["weights"][:, :, None]).sum(1).to(dt)
    dout = st["dout"].float()
    dw = (picked * dout[:, None, :]).sum(2)
    back = torch.where(live, st["weights"][:, :, None] * dout[:, None, :], 0.0)
    drows = torch.empty_like(st["rows"])
    drows[pos.view(-1)] = back.view(-1, case["H"]).to(dt)
    dx = torch.where(live, st["dxrows"].float()[pos], 0.0).sum(1).to(dt)
    return drows, dw, dx


# ------------------------------------------------ the library's entry points

def _run_own(st):
    import dense_fp32_matrix_03_gb300 as lib
    case = st["case"]
    op, type_ = case["op"], case["type"]
    if op == "product":
        M, N, K = case["M"], case["N"], case["K"]
        lib.check(lib.sgemm_i8_quantize_rows(type_, "none", M, K, st["x"], K, st["q"], st["ldw"],
                                             st["sq"]))
        lib.check(lib.sgemm_i8(type_, M, N, K, st["q"], st["ldw"], st["sq"], st["w"], st["ldw"],
                               st["sw"], st["y"], N))
        return st["y"]
    T, k, E = case["T"], case["k"], case["E"]
    if op in ("route", "experts"):
        lib.check(lib.sgemm_experts_sort(T, k, E, st["ids"], st["offsets"], st["slots"],
                                         st["positions"]))
    if op == "experts":
        N, K = case["N"], case["K"]
        lib.check(lib.sgemm_experts_dispatch_i8(type_, T, k, E, K, st["x"], K, st["positions"],
                                                st["offsets"], st["q"], st["ldw"], st["sq"]))
        lib.check(lib.sgemm_i8_experts(type_, T * k, N, K, E, st["offsets"], st["q"], st["ldw"],
                                       st["sq"], st["w"], st["ldw"], N * st["ldw"], st["sw"],
                                       st["y"], N))
        return st["y"], st["offsets"], st["slots"], st["positions"]
    H = case["H"]
    if op == "route":
        lib.check(lib.sgemm_experts_dispatch(type_, T, k, E, H, st["x"], H, st["positions"],
                                             st["offsets"], st["rows"], H))
        return st["rows"], st["offsets"], st["slots"], st["positions"]
    if op == "combine":
        lib.check(lib.sgemm_experts_combine(type_, T, k, E, H, st["rows"], H, st["positions"],
                                            st["offsets"], st["weights"], st["out"], H))
        return st["out"]
    lib.check(lib.sgemm_experts_combine_grad(type_, T, k, E, H, st["dout"], H, st["rows"], H,
                                             st["positions"], st["offsets"], st["weights"],
                                             st["drows"], H, st["dweights"]))
    lib.check(lib.sgemm_experts_dispatch_grad(type_, T, k, E, H, st["dxrows"], H,
                                              st["positions"], st["offsets"], st["dx"], H))
    return st["drows"], st["dweights"], st["dx"]


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------- floors

def work(case):
    op, es = case["op"], SIZE[case["type"]]
    if op == "product":
        M, N, K = case["M"], case["N"], case["K"]
        return dict(bytes=M * K * es + N * K + 4 * N + M * N * es, flops=2 * M * N * K)
    T, k, E = case["T"], case["k"], case["E"]
    S = T * k
    live = int(S * (1 - case["drop"]))
    if op == "experts":
        N, K = case["N"], case["K"]
        used = E * (1 - (1 - 1 / E) ** live)  # experts with a row, when choices are even
        return dict(bytes=int(4 * S + T * K * es + used * (N * K + 4 * N) + live * N * es
                              + 8 * S + 4 * E),
                    flops=2 * live * N * K)
    H = case["H"]
    if op == "route":
        return dict(bytes=4 * S + T * H * es + S * H * es + 8 * S + 4 * E, flops=0)
    if op == "combine":
        return dict(bytes=live * H * es + T * H * es + 8 * S, flops=2 * live * H)
    return dict(bytes=T * H * es + live * H * es + 8 * S + S * H * es + 4 * S  # combine's way back
                + live * H * es + T * H * es + 4 * S,                          # dispatch's
                flops=4 * live * H)


# -------------------------------------------------------------- exact values

def exact(case, seed):
    """The definitions, choice by choice for the order, in 64 bits for the
    numbers."""
    st = prepare(case, seed)
    op = case["op"]
    f64 = torch.float64

    def codes(x):
        x = x.to(f64)
        big = x.abs().max(dim=1, keepdim=True).values
        safe = torch.where(big < TINY, torch.ones_like(big), big)
        q = torch.round(x / safe * 127)
        q = torch.where(big < TINY, torch.zeros_like(q), q)
        return q, torch.where(big < TINY, torch.zeros_like(big), big / 127)

    if op == "product":
        q, s = codes(st["x"])
        y = q @ st["w"][0, :, :case["K"]].to(f64).t()
        return y.mul_(s).mul_(st["sw"][0].to(f64))
    T, k, E = case["T"], case["k"], case["E"]
    ids = st["ids"].cpu().numpy().reshape(-1).tolist()
    lists = [[] for _ in range(E + 1)]
    for s, e in enumerate(ids):
        lists[e if 0 <= e < E else E].append(s)
    first = [0]
    for e in range(E):
        first.append(first[-1] + len(lists[e]))
    order = [s for each in lists for s in each]
    where = [0] * len(order)
    for p, s in enumerate(order):
        where[s] = p
    offsets = torch.tensor(first, dtype=torch.int32)
    slots = torch.tensor(order, dtype=torch.int32)
    positions = torch.tensor(where, dtype=torch.int32)
    total = first[-1]
    source = slots.long().cuda() // k
    if op == "experts":
        y = torch.zeros(T * k, case["N"], dtype=f64, device="cuda")
        q, s = codes(st["x"])
        for e in range(E):
            a, b = first[e], first[e + 1]
            if a == b:
                continue
            t = source[a:b]
            y[a:b] = (q[t] @ st["w"][e, :, :case["K"]].to(f64).t()) * s[t] * st["sw"][e].to(f64)
        return y, offsets, slots, positions
    if op == "route":
        rows = st["x"].to(f64)[source]
        rows[total:] = 0
        return rows, offsets, slots, positions
    # one expert row at a time in the tokens' order: row of choice (t, j)
    T, H = case["T"], case["H"]
    w = st["weights"].to(f64)
    row_of = positions.long().cuda().view(T, k)
    if op == "combine":
        out = torch.zeros(T, H, dtype=f64, device="cuda")
        for j in range(k):
            on = row_of[:, j] < total
            out[on] += w[on, j, None] * st["rows"][row_of[on, j]].to(f64)
        return out
    drows = torch.zeros(T * k, H, dtype=f64, device="cuda")
    dw = torch.zeros(T, k, dtype=f64, device="cuda")
    dx = torch.zeros(T, H, dtype=f64, device="cuda")
    g = st["dout"].to(f64)
    for j in range(k):
        on = row_of[:, j] < total
        r = row_of[on, j]
        drows[r] = w[on, j, None] * g[on]
        dw[on, j] = torch.einsum("th,th->t", st["rows"][r].to(f64), g[on])
        dx[on] += st["dxrows"][r].to(f64)
    return drows, dw, dx
