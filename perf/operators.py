"""Measured cases of the gated delta rule (recurrent and chunked) and of the FP8 products around it.

Each case is one call a serving program makes. `run` computes it in plain torch operations in 32
bits, or, where `own` is set, by the library's entry points:

  gdr_decode   kda_gdr_decode   n new tokens for each of B sequences
  gdr_prefill  kda_gdr_prefill  packed prompts of different lengths
  linear_fp8   kda_linear_fp8   y = x W^T (+ r), both operands FP8 with a scale per block of 128
  quant_fp8    kda_quant_fp8    the operands of that product from BF16 or FP32

States live in slots: a call reads the slots src and writes the slots dst, so the same pass can be
repeated.
"""
import math

import torch

own = False

D = 128    # head dimension
C = 64     # tokens a chunk of the plain chunked form
E4M3_MAX = 448.0
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one conversation, one token: the latency of a call
        {"name": "gdr_decode_b1", "op": "gdr_decode", "B": 1, "n": 1, "H": 32, "Hk": 16, "dtype": "bf16", "packed": True},
        # the decode batch of the repository's benchmark at its 96 heads
        {"name": "gdr_decode_b256", "op": "gdr_decode", "B": 256, "n": 1, "H": 96, "Hk": 96, "dtype": "bf16", "packed": False},
        # four draft tokens to verify for each of an odd number of rows, FP32 rows, four value heads a key head
        {"name": "gdr_decode_b37_n4_f32", "op": "gdr_decode", "B": 37, "n": 4, "H": 16, "Hk": 4, "dtype": "f32", "packed": True},
        # a short turn of a chat
        {"name": "gdr_prefill_t100", "op": "gdr_prefill", "lens": "100", "H": 32, "Hk": 16, "dtype": "bf16", "packed": True},
        # the prompt length of the repository's benchmark
        {"name": "gdr_prefill_t8192", "op": "gdr_prefill", "lens": "8192", "H": 32, "Hk": 16, "dtype": "bf16", "packed": True},
        # a batch of unequal prompts, one of them empty, at the repository's 96 heads
        {"name": "gdr_prefill_varlen", "op": "gdr_prefill", "lens": "1,65,700,0,2048,311,1537,64", "H": 96, "Hk": 96, "dtype": "bf16", "packed": False},
        # FP32 rows, the correctness path
        {"name": "gdr_prefill_f32", "op": "gdr_prefill", "lens": "5,333,1024", "H": 8, "Hk": 8, "dtype": "f32", "packed": False},
        # the output projection of a small decode batch: the weights' bytes
        {"name": "linear_fp8_m16", "op": "linear_fp8", "M": 16, "N": 7168, "K": 12288, "res": True},
        # sizes that divide by no tile
        {"name": "linear_fp8_ragged", "op": "linear_fp8", "M": 777, "N": 1000, "K": 2064, "res": False},
        # one projection of a long prompt: the tensor cores' rate
        {"name": "linear_fp8_m8192", "op": "linear_fp8", "M": 8192, "N": 12288, "K": 7168, "res": False},
        # the activations of that prompt
        {"name": "quant_fp8_rows", "op": "quant_fp8", "M": 8192, "K": 7168, "block": 1, "dtype": "bf16"},
        # a weight matrix that divides by no block
        {"name": "quant_fp8_blocks", "op": "quant_fp8", "M": 1000, "K": 2064, "block": 128, "dtype": "f32"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["gdr_decode", "gdr_prefill", "gdr_prefill", "linear_fp8", "linear_fp8", "quant_fp8"])
    if op == "gdr_decode":
        H = rng.choice([4, 8, 16, 32, 48, 64, 96])
        return {"op": op, "B": _log(rng, 1, 256), "n": rng.choice([1, 1, 2, 3, 5, 8]), "H": H,
                "Hk": H // rng.choice([1, 2, 4]), "dtype": rng.choice(["bf16", "bf16", "f32"]),
                "packed": rng.random() < 0.5}
    if op == "gdr_prefill":
        H = rng.choice([4, 8, 16, 32, 48, 64, 96])
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        top = 8192 if dtype == "bf16" else 1500
        left = 8192 * 32 // H if dtype == "bf16" else 24000 // H
        lens = []
        for _ in range(rng.randint(1, 12)):
            lens.append(min(_log(rng, 1, top), max(1, left)))
            left -= lens[-1]
        return {"op": op, "lens": ",".join(str(x) for x in lens), "H": H, "Hk": H // rng.choice([1, 2, 4]),
                "dtype": dtype, "packed": rng.random() < 0.5}
    if op == "linear_fp8":
        while True:
            M, N, K = _log(rng, 1, 8192), 8 * _log(rng, 1, 2048), 16 * _log(rng, 1, 1024)
            if M * N * K <= 8192 * 12288 * 7168:
                return {"op": op, "M": M, "N": N, "K": K, "res": rng.random() < 0.5}
    while True:
        M, K = _log(rng, 1, 16384), 16 * _log(rng, 1, 1024)
        if M * K <= 8192 * 7168:
            return {"op": op, "M": M, "K": K, "block": rng.choice([1, 128]), "dtype": rng.choice(["bf16", "f32"])}


def _lens(case):
    return [int(x) for x in case["lens"].split(",")] if "lens" in case else [case["n"]] * case["B"]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    st = {"case": case}
    if case["op"] == "quant_fp8":
        # activations with a few large channels, weights scaled by their fan-in
        x = randn(case["M"], case["K"])
        x = x * torch.exp(randn(1, case["K"])) if case["block"] == 1 else x * case["K"] ** -0.5
        st["x"] = x.to(DT[case["dtype"]])
        return st
    if case["op"] == "linear_fp8":
        M, N, K = case["M"], case["N"], case["K"]
        st["xq"], st["xs"] = _quantise(randn(M, K) * torch.exp(0.5 * randn(M, 1)), 1)
        st["wq"], st["ws"] = _quantise(randn(N, K) * K ** -0.5, 128)
        # a checkpoint's block scales are any FP32 numbers
        st["ws"] = st["ws"] * (1.0 + 0.5 * torch.rand(st["ws"].shape, generator=gen, device=dev))
        st["r"] = randn(M, N).to(torch.bfloat16) if case["res"] else None
        return st
    H, Hk, dt = case["H"], case["Hk"], DT[case["dtype"]]
    lens = _lens(case)
    N, T = len(lens), sum(lens)
    # the mixer's inputs: after the activation (SiLU) for q, k, v, logits for the gates
    parts = [randn(T, Hk * D), randn(T, Hk * D), randn(T, H * D)]
    parts = [x * torch.sigmoid(x) for x in parts] + [randn(T, H), randn(T, H)]
    if case["packed"]:  # columns of one projection's output
        width = -(-sum(x.shape[1] for x in parts) // 8) * 8
        rows = torch.zeros(T, width, dtype=dt, device=dev)
        at = 0
        for i, x in enumerate(parts):
            rows[:, at:at + x.shape[1]] = x
            parts[i] = rows[:, at:at + x.shape[1]]
            at += x.shape[1]
    else:
        parts = [x.to(dt) for x in parts]
    st["q"], st["k"], st["v"], st["a"], st["b"] = parts
    st["A_log"] = torch.rand(H, generator=gen, device=dev) * math.log(16.0)
    st["dt_bias"] = randn(H) * math.sqrt(0.5)
    st["S"] = torch.zeros(2 * N, H, D, D, device=dev)
    st["S"][:N] = 0.05 * randn(N, H, D, D)
    src = torch.arange(N, device=dev, dtype=torch.int32)
    if "lens" in case:
        src[0] = -1  # the first sequence starts from nothing
    st["src"], st["dst"] = src, torch.arange(N, 2 * N, device=dev, dtype=torch.int32)
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    st["cu_host"] = cu
    st["cu"] = torch.tensor(cu, device=dev, dtype=torch.int32)
    return st


def _quantise(x, rows):
    """q = e4m3(x / s) with one scale s = 2^e for each block of `rows` x 128 values, the smallest with |x| <= 448 s."""
    M, K = x.shape
    nm, nk = -(-M // rows), -(-K // 128)
    blocks = torch.zeros(nm * rows, nk * 128, device=x.device)
    blocks[:M, :K] = x.float()
    blocks = blocks.view(nm, rows, nk, 128)
    amax = torch.where(torch.isfinite(blocks), blocks.abs(), 0.0).amax(dim=(1, 3))
    m, p = torch.frexp(amax)  # amax = m 2^p, m in [0.5, 1); 448 = 0.875 * 2^9
    e = (p - 9 + (m > 0.875).to(p.dtype)).clamp(min=-126)
    s = torch.where(amax > 0, ((e + 127) << 23).to(torch.int32).view(torch.float32), 1.0)
    q = (blocks / s[:, None, :, None]).view(nm * rows, nk * 128)[:M, :K]
    q = torch.where(torch.isfinite(q), q, float("nan"))
    return q.to(torch.float8_e4m3fn).contiguous(), s.contiguous()


def _gates(st):
    """Log decay and beta of every token and value head."""
    x = st["a"].float() + st["dt_bias"]
    softplus = x.clamp(min=0) + torch.log1p(torch.exp(-x.abs()))
    return -torch.exp(st["A_log"]) * softplus, 1.0 / (1.0 + torch.exp(-st["b"].float()))


def _heads(st):
    """q^ (scaled), k^ and v in 32 bits, [T, H, D]."""
    H, Hk = st["case"]["H"], st["case"]["Hk"]
    T = st["q"].shape[0]

    def unit(x):
        x = x.float().reshape(T, Hk, D)
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) + 1e-6)
        return x[:, :, None, :].expand(T, Hk, H // Hk, D).reshape(T, H, D)

    return unit(st["q"]) * D ** -0.5, unit(st["k"]), st["v"].float().reshape(T, H, D)


def _start(st):
    src = st["src"].long()
    return st["S"][src.clamp(min=0)] * (src >= 0).float()[:, None, None, None]


def _decode(st):
    B, n, H = st["case"]["B"], st["case"]["n"], st["case"]["H"]
    q, k, v = (x.view(B, n, H, D) for x in _heads(st))
    g, beta = (x.view(B, n, H) for x in _gates(st))
    S = _start(st)
    out = torch.empty(B, n, H, D, device=S.device)
    for t in range(n):
        S = S * torch.exp(g[:, t])[..., None, None]
        u = beta[:, t][..., None] * (v[:, t] - torch.matmul(k[:, t][:, :, None, :], S)[:, :, 0])
        S = S + k[:, t][..., :, None] * u[..., None, :]
        out[:, t] = torch.matmul(q[:, t][:, :, None, :], S)[:, :, 0]
    return out.reshape(B * n, H * D).to(st["q"].dtype), S


def _prefill(st):
    H, cu = st["case"]["H"], st["cu_host"]
    dev, N, T = st["q"].device, len(cu) - 1, cu[-1]
    first, where = [0], []  # chunks of each sequence; row of each chunk's tokens
    for s in range(N):
        n = cu[s + 1] - cu[s]
        first.append(first[-1] + -(-n // C))
        where += [cu[s] + i if i < n else -1 for i in range(-(-n // C) * C)]
    nc = first[-1]
    rows = torch.tensor(where, device=dev).view(nc, C)
    there = rows >= 0
    rows = rows.clamp(min=0)
    q, k, v = (torch.where(there[..., None, None], x[rows], 0.0).transpose(1, 2) for x in _heads(st))  # [nc, H, C, D]
    g, beta = (torch.where(there[..., None], x[rows], 0.0).transpose(1, 2) for x in _gates(st))        # [nc, H, C]
    G = g.double().cumsum(-1)
    low = torch.ones(C, C, dtype=torch.bool, device=dev).tril()
    decay = torch.exp(torch.where(low, G[..., :, None] - G[..., None, :], -math.inf)).float()
    A = (beta[..., None] * torch.matmul(k, k.transpose(-1, -2)) * decay).tril(-1)
    inv = torch.eye(C, device=dev).repeat(nc, H, 1, 1)  # (I + A)^-1 by forward substitution
    for t in range(1, C):
        inv[..., t, :t] = -torch.matmul(A[..., t, None, :t], inv[..., :t, :t])[..., 0, :]
    eG = torch.exp(G).float()[..., None]
    W = torch.matmul(inv, beta[..., None] * eG * k)
    U0 = torch.matmul(inv, beta[..., None] * v)
    P = torch.matmul(q, k.transpose(-1, -2)) * decay
    Qg = q * eG
    Kd = k * torch.exp(G[..., -1:] - G).float()[..., None]
    last = torch.exp(G[..., -1]).float()[..., None, None]
    S = _start(st)
    out = torch.zeros(nc, H, C, D, device=dev)
    counts = [first[s + 1] - first[s] for s in range(N)]
    for c in range(max(counts, default=0)):
        on = [s for s in range(N) if counts[s] > c]
        at, ss = torch.tensor([first[s] + c for s in on], device=dev), torch.tensor(on, device=dev)
        S0 = S[ss]
        U = U0[at] - torch.matmul(W[at], S0)
        out[at] = torch.matmul(Qg[at], S0) + torch.matmul(P[at], U)
        S[ss] = last[at] * S0 + torch.matmul(Kd[at].transpose(-1, -2), U)
    o = torch.zeros(T, H, D, device=dev)
    o[rows[there]] = out.transpose(1, 2)[there]
    return o.view(T, H * D).to(st["q"].dtype), S


def _linear(st):
    def whole(q, s, rows):
        M, K = q.shape
        return q.float() * s.repeat_interleave(rows, 0)[:M].repeat_interleave(128, 1)[:, :K]

    y = torch.matmul(whole(st["xq"], st["xs"], 1), whole(st["wq"], st["ws"], 128).t())
    return (y if st["r"] is None else y + st["r"].float()).to(torch.bfloat16)


def _own(st):
    import linear_attention_mixer_gb300 as K

    case, op = st["case"], st["case"]["op"]
    if op == "quant_fp8":
        if "q8" not in st:
            M, Kd, rows = case["M"], case["K"], case["block"]
            st["q8"] = torch.empty(M, Kd, dtype=torch.float8_e4m3fn, device=st["x"].device)
            st["s8"] = torch.empty(-(-M // rows), -(-Kd // 128), dtype=torch.float32, device=st["x"].device)
        K.kda_quant_fp8(st["x"], st["q8"], st["s8"], block_rows=case["block"])
        return st["q8"], st["s8"]
    if op == "linear_fp8":
        if "y" not in st:
            M, N, Kd = case["M"], case["N"], case["K"]
            st["y"] = torch.empty(M, N, dtype=torch.bfloat16, device=st["xq"].device)
            st["work"] = torch.empty(K.kda_linear_fp8_workspace_bytes(M, N, Kd), dtype=torch.uint8, device=st["xq"].device)
        K.kda_linear_fp8(st["xq"], st["xs"], st["wq"], st["ws"], st["y"], st["work"], r=st["r"])
        return st["y"]
    if "cfg" not in st:
        st["cfg"] = K.kda_gdr_config(case["H"], case["Hk"], D, K.KDA_BF16 if case["dtype"] == "bf16" else K.KDA_F32)
        st["params"] = K.kda_gdr_params_from(st["A_log"], st["dt_bias"])
        st["out"] = torch.empty(st["q"].shape[0], case["H"] * D, dtype=st["q"].dtype, device=st["q"].device)
        if op == "gdr_prefill":
            st["work"] = torch.empty(K.kda_gdr_workspace_bytes(st["cfg"], st["cu_host"]), dtype=torch.uint8, device=st["q"].device)
    rows = (st["q"], st["k"], st["v"], st["a"], st["b"], st["out"])
    if op == "gdr_decode":
        K.kda_gdr_decode(st["cfg"], st["params"], st["S"], st["src"], st["dst"], case["n"], *rows)
    else:
        K.kda_gdr_prefill(st["cfg"], st["params"], st["S"], st["src"], st["dst"], st["cu"], st["cu_host"], *rows, st["work"])
    return st["out"], st["S"][len(st["cu_host"]) - 1:]


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "quant_fp8":
        return _quantise(state["x"], state["case"]["block"])
    if op == "linear_fp8":
        return _linear(state)
    return _decode(state) if op == "gdr_decode" else _prefill(state)


def work(case):
    if case["op"] == "quant_fp8":
        M, K, b = case["M"], case["K"], case["block"]
        return {"bytes": M * K * (DT[case["dtype"]].itemsize + 1) + 4 * -(-M // b) * -(-K // 128), "flops": 2 * M * K}
    if case["op"] == "linear_fp8":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": M * K + N * K + 4 * -(-K // 128) * (M + -(-N // 128)) + M * N * (4 if case["res"] else 2),
                "flops": 2 * M * N * K}
    H, Hk, lens = case["H"], case["Hk"], _lens(case)
    T, e = sum(lens), DT[case["dtype"]].itemsize
    read = len(lens) - (1 if "lens" in case else 0)  # states read
    return {"bytes": T * e * (2 * Hk * D + 2 * H * D + 2 * H) + 4 * H * D * D * (read + len(lens)),
            "flops": 6 * T * H * D * D}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "quant_fp8":
        return _exact_quant(st["x"].double(), case["block"])
    if case["op"] == "linear_fp8":
        x, w = st["xq"].double(), st["wq"].double()
        y = torch.zeros(case["M"], case["N"], dtype=torch.float64, device=x.device)
        for b in range(st["xs"].shape[1]):
            part = x[:, 128 * b:128 * b + 128] @ w[:, 128 * b:128 * b + 128].t()
            rows = torch.arange(case["N"], device=x.device) // 128
            y += part * st["xs"][:, b, None].double() * st["ws"][rows, b].double()
        return y if st["r"] is None else y + st["r"].double()
    H, Hk, lens = case["H"], case["Hk"], _lens(case)
    N, steps = len(lens), max(lens)
    if steps * (2e-4 + N * H * D * D * 8 * 9 / 4e12) > 15:
        return None
    dev = st["q"].device
    dt = torch.float64
    group = torch.arange(H, device=dev) // (H // Hk)
    cu = torch.tensor(st["cu_host"], device=dev)
    S = torch.zeros(N, H, D, D, dtype=dt, device=dev)
    for s, slot in enumerate(st["src"].tolist()):
        if slot >= 0:
            S[s] = st["S"][slot].to(dt)
    out = torch.zeros(st["q"].shape[0], H, D, dtype=dt, device=dev)
    rate = torch.exp(st["A_log"].to(dt))
    long = sorted(range(N), key=lambda s: -lens[s])  # the token loop runs over the sequences that are still going
    order = torch.tensor(long, device=dev)
    S = S[order]
    for t in range(steps):
        n = sum(lens[s] > t for s in long)
        row = cu[order[:n]] + t
        k = st["k"][row].to(dt).view(n, Hk, D)[:, group]
        q = st["q"][row].to(dt).view(n, Hk, D)[:, group]
        k = k * (k.square().sum(-1, keepdim=True) + 1e-6).rsqrt()
        q = q * (q.square().sum(-1, keepdim=True) + 1e-6).rsqrt() / math.sqrt(D)
        alpha = torch.exp(-rate * torch.nn.functional.softplus(st["a"][row].to(dt) + st["dt_bias"].to(dt), threshold=60.0))
        beta = torch.sigmoid(st["b"][row].to(dt))
        Z = S[:n]
        Z *= alpha[..., None, None]
        miss = st["v"][row].to(dt).view(n, H, D) - torch.einsum("nhk,nhkv->nhv", k, Z)
        Z += torch.einsum("nhk,nhv->nhkv", k * beta[..., None], miss)
        out[row] = torch.einsum("nhk,nhkv->nhv", q, Z)
    back = torch.empty_like(S)
    back[order] = S
    return out.view(-1, H * D), back


def _exact_quant(x, rows):
    M, K = x.shape
    nm, nk = -(-M // rows), -(-K // 128)
    s = torch.ones(nm, nk, dtype=torch.float64, device=x.device)
    full = torch.zeros(nm * rows, nk * 128, dtype=torch.float64, device=x.device)
    full[:M, :K] = x.abs()
    top = full.view(nm, rows, nk, 128).amax(3).amax(1)
    # the smallest power of two with top <= 448 s: the logarithm's ceiling, then put right by one step where it rounded
    s = torch.exp2(torch.ceil(torch.log2(top.clamp(min=1e-300) / E4M3_MAX))).clamp(min=2.0 ** -126)
    s = torch.where(top > E4M3_MAX * s, 2 * s, torch.where(top <= E4M3_MAX * s / 2, (s / 2).clamp(min=2.0 ** -126), s))
    s = torch.where(top > 0, s, torch.ones_like(s))
    z = x / s.repeat_interleave(rows, 0)[:M].repeat_interleave(128, 1)[:, :K]
    # e4m3: four significant bits, the smallest step 2^-9, ties to even
    _, p = torch.frexp(z)
    step = torch.exp2((p.double() - 4).clamp(min=-9.0))
    return torch.round(z / step) * step, s
