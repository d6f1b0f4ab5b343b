"""Measured cases of the gated linear recurrence (token by token, packed prompts, training) and of the block norms.

Each case is one call, or one training step, of a user's program. `run` computes it in plain torch operations, or,
where `own` is set, by the library's entry points:

  glr_decode      kda_glr_decode           n new tokens for each of B sequences
  glr_prefill     kda_glr_prefill          packed prompts of different lengths
  glr_train       kda_glr_prefill, then kda_glr_backward   outputs, and gradients of rows, parameters and states
  block_norm      kda_block_norm           residual + gate * scale * norm(block's output), and the next block's norm
  block_norm_back kda_block_norm_backward  the gradients of that

The recurrence, for each channel c of dim (all parameters FP32 [dim]):
  gk = -exp(A_log) sigmoid(a + a_bias),  alpha = exp(gk),  beta = sigmoid(b + b_bias)
  h = alpha h + sqrt(1 - alpha^2) beta x,  out = h, or h silu(g) with an output gate
The block norms, for each row of dim channels (rms(z) = sqrt(mean(z^2) + eps)):
  x' = x + scale sigmoid(g) post_w y / rms(y),  h = pre_w x' / rms(x')
with h in the rows' type, or in E4M3 with a power-of-two scale for each 128 columns (the values that these stand for are
returned, in BF16, which holds them).
"""
import math

import torch

own = False

EPS = 1e-6
E4M3_MAX = 448.0
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one conversation, one token: the latency of a call
        {"name": "glr_decode_b1", "op": "glr_decode", "B": 1, "n": 1, "D": 4096, "dtype": "bf16", "gate": True, "packed": True},
        # the decode batch of the repository's benchmark at its 96 x 128 channels, four draft tokens each
        {"name": "glr_decode_b256_n4", "op": "glr_decode", "B": 256, "n": 4, "D": 12288, "dtype": "bf16", "gate": True, "packed": False},
        # a short turn of a chat
        {"name": "glr_prefill_t100", "op": "glr_prefill", "lens": "100", "D": 4096, "dtype": "bf16", "gate": True, "packed": True},
        # one long document
        {"name": "glr_prefill_t65536", "op": "glr_prefill", "lens": "65536", "D": 4096, "dtype": "bf16", "gate": False, "packed": False},
        # a batch of unequal prompts, one of them empty, at the hidden width of the repository's layers
        {"name": "glr_prefill_varlen", "op": "glr_prefill", "lens": "1,65,700,0,2048,311,1537,64", "D": 7168, "dtype": "f32", "gate": False, "packed": True},
        # a training step over one long sequence
        {"name": "glr_train_t8192", "op": "glr_train", "lens": "8192", "D": 4096, "dtype": "bf16", "gate": True, "packed": False},
        # a training step over ragged FP32 sequences of an odd width
        {"name": "glr_train_ragged", "op": "glr_train", "lens": "5,333,1024,63", "D": 1004, "dtype": "f32", "gate": False, "packed": False},
        # the norms around one decode token's block
        {"name": "block_norm_m1", "op": "block_norm", "M": 1, "D": 7168, "dtype": "bf16", "gate": False, "fp8": False},
        # those of a prompt as long as the repository's benchmark
        {"name": "block_norm_m8192", "op": "block_norm", "M": 8192, "D": 7168, "dtype": "bf16", "gate": True, "fp8": False},
        # a decode batch whose next projection takes FP8 rows
        {"name": "block_norm_fp8", "op": "block_norm", "M": 512, "D": 7168, "dtype": "bf16", "gate": False, "fp8": True},
        # training on as many rows
        {"name": "block_norm_back_m8192", "op": "block_norm_back", "M": 8192, "D": 7168, "dtype": "bf16", "gate": True},
        # FP32 rows whose sizes divide by nothing
        {"name": "block_norm_back_ragged", "op": "block_norm_back", "M": 777, "D": 1004, "dtype": "f32", "gate": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _width(rng, hi, dtype):
    """A row's channels: whole 16 bytes."""
    unit = 8 if dtype == "bf16" else 4
    return unit * _log(rng, 64 // unit, hi // unit)


def _lengths(rng, total):
    """Lengths of packed sequences, `total` tokens at most: a few of any length, or many short ones."""
    if rng.random() < 0.3:
        count, top = _log(rng, 8, 300), _log(rng, 2, 200)
        got = [rng.randint(0, top) for _ in range(count)]
    else:
        got = [_log(rng, 1, 65536) for _ in range(rng.randint(1, 9))]
    out = []
    for n in got:
        out.append(min(n, total))
        total -= out[-1]
    return ",".join(str(x) for x in out) if any(out) else "1"


def draw(rng):
    op = rng.choice(["glr_decode", "glr_prefill", "glr_prefill", "glr_train", "block_norm", "block_norm", "block_norm_back"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    case = {"op": op, "dtype": dtype, "gate": rng.random() < 0.5}
    if op.startswith("block_norm"):
        case["M"], case["D"] = _log(rng, 1, 16384), _width(rng, 16384, dtype)
        case["M"] = min(case["M"], 8192 * 7168 // case["D"])
        if op == "block_norm":
            case["fp8"] = rng.random() < 0.3
            if case["fp8"]:
                case["M"], case["D"] = min(case["M"], 1024), 16 * (case["D"] // 16)
        return case
    case["D"], case["packed"] = _width(rng, 12288, dtype), rng.random() < 0.5
    if op == "glr_decode":
        case["B"], case["n"] = _log(rng, 1, 256), rng.choice([1, 1, 2, 3, 5, 8])
        return case
    most = {"glr_prefill": 65536 * 4096, "glr_train": 8192 * 4096}[op] // (1 if dtype == "bf16" else 2)
    case["lens"] = _lengths(rng, min(65536, most // case["D"]))
    return case


def _lens(case):
    return [int(x) for x in case["lens"].split(",")] if "lens" in case else [case["n"]] * case["B"]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    D, dt = case["D"], DT[case["dtype"]]

    def randn(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=gen, device=dev, dtype=dtype)

    st = {"case": case, "g": None}
    if case["op"].startswith("block_norm"):
        M = case["M"]
        # a residual stream with a few large channels, a block's output of another size, weights near one, small scales
        names = {"block_norm": ["x", "y"], "block_norm_back": ["x1", "y", "dx1", "dh"]}[case["op"]]
        st |= {n: randn(M, D, dtype=dt) for n in names + (["g"] if case["gate"] else [])}
        wide = torch.exp(randn(1, D)).to(dt)
        st[names[0]] *= wide
        st["y"] *= 0.3
        st["post_w"], st["pre_w"] = 1.0 + 0.2 * randn(D), 1.0 + 0.2 * randn(D)
        st["scale"] = 0.1 + 0.05 * randn(D)
        return st
    lens = _lens(case)
    N, T = len(lens), sum(lens)
    names = ["x", "a", "b"] + (["g"] if case["gate"] else [])
    if case["packed"]:  # columns of one projection's output
        st["rows"] = randn(T, len(names) * D, dtype=dt)
        st |= {n: st["rows"][:, i * D:i * D + D] for i, n in enumerate(names)}
    else:
        st |= {n: randn(T, D, dtype=dt) for n in names}
    # decays of one to a thousand tokens; biases that open the gates unequally
    st["A_log"] = math.log(0.002) + torch.rand(D, generator=gen, device=dev) * math.log(1000.0)
    st["a_bias"], st["b_bias"] = 0.7 * randn(D), 0.7 * randn(D)
    st["S"] = torch.zeros(2 * N, D, device=dev)
    st["S"][:N] = 0.5 * randn(N, D)
    src = torch.arange(N, device=dev, dtype=torch.int32)
    if "lens" in case:
        src[0] = -1  # the first sequence starts from nothing
    st["src"], st["dst"] = src, torch.arange(N, 2 * N, device=dev, dtype=torch.int32)
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    st["cu_host"], st["cu"] = cu, torch.tensor(cu, device=dev, dtype=torch.int32)
    if case["op"] == "glr_train":
        st["dout"] = randn(T, D, dtype=dt)
        st["dS_last"] = randn(N, D)
    return st


# ---------------------------------------------------------------- the recurrence in plain form

def _sigmoid(x):
    return 1.0 / (1.0 + torch.exp(-x))


def _gates(st):
    """gk, alpha, sqrt(1 - alpha^2) and beta of every row, in 32 bits, gk in 64."""
    gk = -torch.exp(st["A_log"].double()) * _sigmoid(st["a"].double() + st["a_bias"])
    m = torch.sqrt(-torch.expm1(2.0 * gk)).float()
    return gk, m, _sigmoid(st["b"].float() + st["b_bias"])


def _scan(A, h, first):
    """h_t = A_t h_(t-1) + h_t in place, along the rows, afresh at the rows `first`: by doubling, in 64 bits (sums over
    many tokens, decays near one)."""
    A[first] = 0.0
    s = 1
    while s < h.shape[0]:
        h[s:] += A[s:] * h[:-s]  # the right side is computed before it is added
        A[s:] = A[s:] * A[:-s]
        s *= 2
    return h


def _start(st):
    src = st["src"].long()
    return st["S"][src.clamp(min=0)] * (src >= 0).float()[:, None]


def _bounds(st):
    """Sequences that are not empty, and their first and last rows."""
    cu = st["cu"].long()
    some = cu[1:] > cu[:-1]
    return some, cu[:-1][some], cu[1:][some] - 1


def _states(st, gk, u):
    """The state after every row, in 64 bits, and each sequence's last one."""
    some, first, last = _bounds(st)
    h0 = _start(st).double()
    A, h = torch.exp(gk), u.double()
    h[first] += A[first] * h0[some]
    _scan(A, h, first)
    S = h0
    S[some] = h[last]
    return h, S


def _forward(st):
    gk, m, beta = _gates(st)
    u = m * beta * st["x"].float()
    del m, beta
    h, S = _states(st, gk, u)
    if st["g"] is not None:
        z = st["g"].float()
        h = h.float() * (z * _sigmoid(z))
    return h.to(st["x"].dtype), S.float()


def _train(st):
    some, first, last = _bounds(st)
    dt = st["x"].dtype
    gk, m, beta = _gates(st)
    x = st["x"].float()
    h, S = _states(st, gk, m * beta * x)
    before = torch.empty_like(h)  # the state in front of each row
    before[1:] = h[:-1]
    before[first] = _start(st).double()[some]
    out, dh, dg = h, st["dout"].float(), None
    if st["g"] is not None:
        z = st["g"].float()
        s = _sigmoid(z)
        out = h.float() * (z * s)
        dg = (dh * h.float() * s * (1.0 + z * (1.0 - s))).to(dt)
        dh = dh * (z * s)
    # lambda_t = dh_t + alpha_(t+1) lambda_(t+1), from the last row of each sequence
    lam = dh.double()
    lam[last] += st["dS_last"].double()[some]
    A = torch.zeros_like(lam)
    A[:-1] = torch.exp(gk[1:])
    lam = _scan(A.flip(0), lam.flip(0), lam.shape[0] - 1 - last).flip(0)
    alpha = torch.exp(gk)
    dS = st["dS_last"].double()
    dS[some] = alpha[first] * lam[first]
    mx = (lam * m).float()
    dx, dbeta = mx * beta, mx * x
    db = dbeta * beta * (1.0 - beta)
    # through alpha: h lambda; through sqrt(1 - alpha^2): its derivative by gk is -alpha^2 / m, and gk / m goes to 0 with gk
    by_gk = lam * before * alpha * gk - (lam * (beta * x)) * alpha * alpha * torch.where(gk < 0, gk / m.double(), 0.0)
    da = by_gk * (1.0 - _sigmoid(st["a"].double() + st["a_bias"]))
    return {"out": out.to(dt), "S": S.float(), "dx": dx.to(dt), "da": da.to(dt), "db": db.to(dt), "dg": dg, "dA_log": by_gk.sum(0).float(),
            "da_bias": da.sum(0).float(), "db_bias": db.double().sum(0).float(), "dS_first": dS.float()}


# ---------------------------------------------------------------- the block norms in plain form

def _rstd(z):
    return 1.0 / torch.sqrt((z * z).mean(-1, keepdim=True) + EPS)


def _norms(st):
    y = st["y"].float()
    z = st["post_w"] * (y * _rstd(y)) * st["scale"]
    x1 = st["x"].float() + (z if st["g"] is None else _sigmoid(st["g"].float()) * z)
    h = st["pre_w"] * (x1 * _rstd(x1))
    x1 = x1.to(st["x"].dtype)
    return x1, (_stands_for(*_quantise(h)) if st["case"]["fp8"] else h.to(st["x"].dtype))


def _quantise(h):
    """q = e4m3(h / s), s = 2^e the smallest with |h| <= 448 s over each 128 columns of a row."""
    M, D = h.shape
    blocks = torch.zeros(M, -(-D // 128) * 128, device=h.device)
    blocks[:, :D] = h
    blocks = blocks.view(M, -1, 128)
    amax = blocks.abs().amax(dim=2)
    m, p = torch.frexp(amax)  # amax = m 2^p, m in [0.5, 1); 448 = 0.875 * 2^9
    e = (p - 9 + (m > 0.875).to(p.dtype)).clamp(min=-126)
    s = torch.where(amax > 0, ((e + 127) << 23).to(torch.int32).view(torch.float32), 1.0)
    q = (blocks / s[..., None]).view(M, -1)[:, :D]
    return q.to(torch.float8_e4m3fn).contiguous(), s


def _stands_for(q, s):
    v, whole = q.to(torch.bfloat16), q.shape[1] // 128 * 128
    v[:, :whole].unflatten(1, (-1, 128)).mul_(s[:, :whole // 128, None])
    if whole < q.shape[1]:
        v[:, whole:].mul_(s[:, -1:])
    return v


def _norms_back(st):
    dt = st["y"].dtype
    x1, y, dh = st["x1"].float(), st["y"].float(), st["dh"].float()
    r = _rstd(x1)
    n = x1 * r
    w = dh * st["pre_w"]
    dx = st["dx1"].float() + r * (w - n * (w * n).mean(-1, keepdim=True))
    dpre = (dh * n).double().sum(0)
    r = _rstd(y)
    n = y * r
    gate = 1.0 if st["g"] is None else _sigmoid(st["g"].float())
    q = (dx * gate * n).double().sum(0)
    w = dx * gate * (st["scale"] * st["post_w"])
    dy = r * (w - n * (w * n).mean(-1, keepdim=True))
    dg = None if st["g"] is None else (w * n * (1.0 - gate)).to(dt)
    return {"dx": dx.to(dt), "dy": dy.to(dt), "dg": dg, "dpost_w": (q * st["scale"]).float(), "dscale": (q * st["post_w"]).float(),
            "dpre_w": dpre.float()}


# ---------------------------------------------------------------- the library

def _own(st):
    import linear_attention_mixer_gb300 as K

    case, op = st["case"], st["case"]["op"]
    io = K.KDA_BF16 if case["dtype"] == "bf16" else K.KDA_F32
    if op == "block_norm":
        if "cfg" not in st:
            st["cfg"] = K.kda_block_norm_config(case["D"], io)
            st["params"] = K.kda_block_norm_params_from(st["post_w"], st["scale"], st["pre_w"])
            st["x1"], st["h"], st["hs"] = torch.empty_like(st["x"]), torch.empty_like(st["x"]), None
            if case["fp8"]:
                st["h"] = torch.empty_like(st["x"], dtype=torch.float8_e4m3fn)
                st["hs"] = torch.empty(case["M"], -(-case["D"] // 128), device=st["x"].device)
        K.kda_block_norm(st["cfg"], st["params"], st["x"], y=st["y"], g=st["g"], x_out=st["x1"], h=st["h"], hs=st["hs"])
        return st["x1"], (_stands_for(st["h"], st["hs"]) if case["fp8"] else st["h"])
    if op == "block_norm_back":
        if "cfg" not in st:
            st["cfg"] = K.kda_block_norm_config(case["D"], io)
            st["params"] = K.kda_block_norm_params_from(st["post_w"], st["scale"], st["pre_w"])
            st["out"] = {n: torch.empty_like(st["y"]) for n in ("dx", "dy")} | {"dg": None if st["g"] is None else torch.empty_like(st["g"])}
            st["out"] |= {n: torch.empty_like(st["scale"]) for n in ("dpost_w", "dscale", "dpre_w")}
            st["work"] = torch.empty(K.kda_block_norm_workspace_bytes(st["cfg"], case["M"]), dtype=torch.uint8, device=st["y"].device)
        K.kda_block_norm_backward(st["cfg"], st["params"], st["x1"], st["dh"], st["dx1"], st["out"]["dx"], st["work"], y=st["y"], g=st["g"],
                                  dy=st["out"]["dy"], dg=st["out"]["dg"], dpost_w=st["out"]["dpost_w"], dscale=st["out"]["dscale"],
                                  dpre_w=st["out"]["dpre_w"])
        return st["out"]
    train = op == "glr_train"
    if "cfg" not in st:
        st["cfg"] = K.kda_glr_config(case["D"], io)
        st["params"] = K.kda_glr_params_from(st["A_log"], st["a_bias"], st["b_bias"])
        st["out"] = torch.empty(st["x"].shape, dtype=st["x"].dtype, device=st["x"].device)
        st["starts"] = None
        if op != "glr_decode":
            st["work"] = torch.empty(K.kda_glr_workspace_bytes(st["cfg"], st["cu_host"]), dtype=torch.uint8, device=st["x"].device)
        if train:
            st["starts"] = torch.empty(K.kda_glr_chunks(st["cu_host"]), case["D"], device=st["x"].device)
            st["grads"] = {n: None if n == "dg" and st["g"] is None else torch.empty_like(st["out"]) for n in ("dx", "da", "db", "dg")}
            st["grads"] |= {n: torch.empty_like(st["A_log"]) for n in ("dA_log", "da_bias", "db_bias")}
            st["grads"]["dS_first"] = torch.empty_like(st["dS_last"])
    rows = (st["x"], st["a"], st["b"], st["g"])
    S = st["S"][st["src"].numel():]
    if op == "glr_decode":
        K.kda_glr_decode(st["cfg"], st["params"], st["S"], st["src"], st["dst"], case["n"], *rows, st["out"])
        return st["out"], S
    K.kda_glr_prefill(st["cfg"], st["params"], st["S"], st["src"], st["dst"], st["cu"], st["cu_host"], *rows, st["out"], st["work"],
                      starts=st["starts"])
    if not train:
        return st["out"], S
    K.kda_glr_backward(st["cfg"], st["params"], st["cu"], st["cu_host"], st["starts"], *rows, st["dout"], work=st["work"],
                       dS_last=st["dS_last"], **st["grads"])
    return {"out": st["out"], "S": S, **st["grads"]}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    return {"block_norm": _norms, "block_norm_back": _norms_back, "glr_train": _train}.get(op, _forward)(state)


def work(case):
    D, e = case["D"], DT[case["dtype"]].itemsize
    if case["op"] == "block_norm":
        M, rows = case["M"], 3 + case["gate"]
        h = M * (D + 4 * -(-D // 128)) if case["fp8"] else M * D * e
        return {"bytes": rows * M * D * e + h + 3 * 4 * D, "flops": (12 + 4 * case["gate"]) * M * D}
    if case["op"] == "block_norm_back":
        return {"bytes": (6 + 2 * case["gate"]) * case["M"] * D * e + 6 * 4 * D, "flops": (24 + 6 * case["gate"]) * case["M"] * D}
    lens = _lens(case)
    T, N, rows = sum(lens), len(lens), 4 + case["gate"]
    states = 2 * N - ("lens" in case)
    if case["op"] == "glr_train":
        return {"bytes": (8 + 2 * case["gate"]) * T * D * e + 4 * D * (states + 2 * N + 6), "flops": (40 + 16 * case["gate"]) * T * D}
    return {"bytes": rows * T * D * e + 4 * D * (states + 3), "flops": (16 + 5 * case["gate"]) * T * D}


# ---------------------------------------------------------------- from the definition, in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    f64 = {k: v.to(torch.float64) if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in st.items()}
    if case["op"].startswith("block_norm"):
        return _exact_norms(f64, case)
    lens = _lens(case)
    cu = torch.tensor(st["cu_host"], device=st["x"].device)
    longest = sorted(range(len(lens)), key=lambda s: -lens[s])  # the token loop runs over the sequences that are still going
    order = torch.tensor(longest, device=st["x"].device)
    live = [sum(n > t for n in lens) for t in range(max(lens))]
    with torch.enable_grad():
        leaf = {n: f64[n].clone().requires_grad_(case["op"] == "glr_train") for n in ("x", "a", "b", "A_log", "a_bias", "b_bias")}
        f64.pop("rows", None)
        alpha = torch.exp(-torch.exp(leaf["A_log"]) * torch.sigmoid(leaf["a"] + leaf["a_bias"]))
        # 1 - alpha^2 without its difference: exp(z) - 1 = 2 exp(z / 2) sinh(z / 2)
        z = -torch.exp(leaf["A_log"]) * torch.sigmoid(leaf["a"] + leaf["a_bias"])
        u = torch.sqrt(-2.0 * torch.exp(z) * torch.sinh(z)) * torch.sigmoid(leaf["b"] + leaf["b_bias"]) * leaf["x"]
    decay, add = alpha.detach(), u.detach()
    state = torch.zeros(len(lens), case["D"], dtype=torch.float64, device=decay.device)
    for s, slot in enumerate(st["src"].tolist()):
        if slot >= 0:
            state[s] = f64["S"][slot]
    state = state[order]
    h, before = torch.empty_like(add), torch.empty_like(add) if case["op"] == "glr_train" else None
    for t, n in enumerate(live):
        row = cu[order[:n]] + t
        if before is not None:
            before[row] = state[:n]
        state[:n] = decay[row] * state[:n] + add[row]
        h[row] = state[:n]
    S = torch.empty_like(state)
    S[order] = state
    gate = None if st["g"] is None else f64["g"].clone().requires_grad_(True)
    if case["op"] != "glr_train":
        return (h if gate is None else h * torch.nn.functional.silu(gate.detach())), S
    dh, dg, out = f64["dout"], None, h
    if gate is not None:
        with torch.enable_grad():
            silu = torch.nn.functional.silu(gate)
            dg, = torch.autograd.grad(silu, gate, dh * h)
        out, dh = h * silu.detach(), dh * silu.detach()
    carry, lam = f64["dS_last"][order].clone(), torch.empty_like(h)
    for t in range(len(live) - 1, -1, -1):
        n = live[t]
        row = cu[order[:n]] + t
        lam[row] = dh[row] + carry[:n]
        carry[:n] = decay[row] * lam[row]
    dS = torch.empty_like(carry)
    dS[order] = carry
    got = torch.autograd.grad([alpha, u], list(leaf.values()), [lam * before, lam])
    grads = dict(zip(("dx", "da", "db", "dA_log", "da_bias", "db_bias"), got))
    return {"out": out, "S": S, "dg": dg, "dS_first": dS, **grads}


def _exact_norms(s, case):
    def normed(z):
        return torch.nn.functional.normalize(z, dim=-1, eps=0.0) * math.sqrt(z.shape[-1]) / torch.sqrt(1.0 + EPS / z.square().mean(-1, keepdim=True))

    def stream(y, g, post_w, scale):
        z = normed(y) * post_w * scale
        return z if g is None else torch.sigmoid(g) * z

    if case["op"] == "block_norm":
        x1 = s["x"] + stream(s["y"], s["g"], s["post_w"], s["scale"])
        h = normed(x1) * s["pre_w"]
        return x1, (_exact_quant(h) if case["fp8"] else h)
    leaf = {n: s[n].clone().requires_grad_(True) for n in ("x1", "y", "g", "post_w", "scale", "pre_w") if s[n] is not None}
    with torch.enable_grad():
        dnorm, dpre = torch.autograd.grad(normed(leaf["x1"]) * leaf["pre_w"], [leaf["x1"], leaf["pre_w"]], s["dh"])
        dx = s["dx1"] + dnorm
        z = stream(leaf["y"], leaf.get("g"), leaf["post_w"], leaf["scale"])
        got = torch.autograd.grad(z, [leaf[n] for n in ("y", "post_w", "scale", "g") if n in leaf], dx)
    return {"dx": dx, "dy": got[0], "dpost_w": got[1], "dscale": got[2], "dg": got[3] if "g" in leaf else None, "dpre_w": dpre}


def _exact_quant(h):
    M, D = h.shape
    full = torch.zeros(M, -(-D // 128) * 128, dtype=torch.float64, device=h.device)
    full[:, :D] = h.abs()
    top = full.view(M, -1, 128).amax(2)
    # the smallest power of two with top <= 448 s: the logarithm's ceiling, then put right by one step where it rounded
    s = torch.exp2(torch.ceil(torch.log2(top.clamp(min=1e-300) / E4M3_MAX))).clamp(min=2.0 ** -126)
    s = torch.where(top > E4M3_MAX * s, 2 * s, torch.where(top <= E4M3_MAX * s / 2, (s / 2).clamp(min=2.0 ** -126), s))
    s = torch.where(top > 0, s, torch.ones_like(s)).repeat_interleave(128, 1)[:, :D]
    z = h / s
    # e4m3: four significant bits, the smallest step 2^-9, ties to even
    _, p = torch.frexp(z)
    step = torch.exp2((p.double() - 4).clamp(min=-9.0))
    return torch.round(z / step) * step * s
