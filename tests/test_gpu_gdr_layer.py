"""The gated delta rule layer, and the KDA layer with FP8 projections, as a serving program runs them:
quantise, project, mix, project back, over a packed prefill and the decode steps that continue it. Each
product is checked against FP64 on the operands that the library itself produced (an FP8 code may turn on
the last bit of what was quantised), the mixer against its oracle on the projection's own output.

Tolerances: the products' as in test_gpu_fp8.py and test_gpu_linear.py (a rounding of the result to BF16,
2^-8, and FP32 sums, 2^-16 of the absolute terms); the mixer's as in test_gpu_gdr.py."""
import numpy as np
import pytest
import torch

import kda_inputs as KI
import linear_attention_mixer_gb300 as K
from linear_attention_mixer_gb300 import layer as L
from oracle import fp8 as O8
from oracle.gdr import gdr
from tests.test_gpu_gdr import near, near_state

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module", autouse=True)
def _built():
    from linear_attention_mixer_gb300 import build
    build.build()
    torch.cuda.set_device(0)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda().to(torch.bfloat16)


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def check_product(x, w, y, r=None):
    """y against x w^T (+ r) of the device tensors, x quantised as the layer does for an Fp8Weight."""
    xh = host(x)
    if isinstance(w, L.Fp8Weight):
        ref, mag = O8.linear(*O8.quantise(xh, 1), host(w.q), host(w.s), None if r is None else host(r))
    else:
        wh = host(w)
        ref, mag = xh @ wh.T + (0 if r is None else host(r)), np.abs(xh) @ np.abs(wh).T + (0 if r is None else np.abs(host(r)))
    bad = np.abs(host(y) - ref) > 2.0 ** -8 * np.abs(ref) + 2.0 ** -16 * mag
    assert not bad.any(), int(bad.sum())


def gdr_layer(H, Hk, hidden, fp8, seed):
    cfg = K.kda_gdr_config(H, Hk)
    rng = np.random.default_rng([seed, H, Hk])
    W = L.gdr_width(cfg)
    used = (2 * Hk + H) * D + 2 * H
    w_in = np.zeros((W, hidden))
    w_in[:used] = rng.standard_normal((used, hidden)) * hidden ** -0.5
    w_o = rng.standard_normal((hidden, H * D)) * (H * D) ** -0.5
    A_log, dt_bias = rng.uniform(0, 2.7, H).astype(np.float32), rng.standard_normal(H).astype(np.float32)
    form = L.fp8_weight if fp8 else (lambda w: w)
    params = K.kda_gdr_params_from(torch.from_numpy(A_log).cuda(), torch.from_numpy(dt_bias).cuda())
    return cfg, L.GdrLayerWeights(form(dev(w_in)), form(dev(w_o)), params), A_log, dt_bias, rng


def check_mixer(cfg, run, rows, S0, A_log, dt_bias, S1, chunked):
    """Rows `rows` of the runner's last call: its mixer's output and new state from its own projection."""
    H, Hk = cfg.num_heads, cfg.num_qk_heads
    p = host(run.proj[rows])
    q, k, v, a, b = np.split(p[:, :(2 * Hk + H) * D + 2 * H], np.cumsum([Hk * D, Hk * D, H * D, H]), axis=1)
    n = len(p)
    o, S, mag, _ = gdr(q.reshape(n, Hk, D), k.reshape(n, Hk, D), v.reshape(n, H, D), a, b, A_log, dt_bias, S0)
    near(run.o[rows], o.reshape(n, -1), mag.reshape(n, -1), True, chunked)
    near_state(S1, S, chunked)


@pytest.mark.parametrize("fp8", [False, True])
def test_prefill_then_decode(fp8):
    H, Hk, hidden, lens = 8, 4, 320 if fp8 else 256, [70, 5, 129]  # the BF16 product takes multiples of 128
    cfg, lw, A_log, dt_bias, rng = gdr_layer(H, Hk, hidden, fp8, 1)
    T, N = sum(lens), len(lens)
    run = L.GdrLayerRunner(cfg, hidden, T, "cuda", fp8)
    S = torch.zeros(N + 1, H, D, D, device="cuda")
    S[N] = float("nan")
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    slot = torch.arange(N, dtype=torch.int32, device="cuda")
    x, y = dev(rng.standard_normal((T, hidden))), torch.empty(T, hidden, dtype=torch.bfloat16, device="cuda")
    run.prefill(lw, S, torch.full((N,), -1, dtype=torch.int32, device="cuda"), slot, torch.from_numpy(cu).cuda(), cu, x, y)
    torch.cuda.synchronize()
    check_product(x, lw.w_in, run.proj[:T])
    for s in range(N):
        check_mixer(cfg, run, slice(cu[s], cu[s + 1]), np.zeros((H, D, D)), A_log, dt_bias, S[s], True)
    check_product(run.o[:T], lw.w_o, y, x)
    x = y[torch.from_numpy(cu[1:] - 1).cuda().long()]
    for n in (1, 1, 3):  # two steps, then three draft tokens of which sequence 1 goes on in a slot of its own
        S0 = host(S)
        dst = slot.clone()
        if n == 3:
            x, dst[1] = x.repeat_interleave(3, 0).contiguous(), N
        y = torch.empty_like(x)
        run.decode(lw, S, slot, dst, n, x, y)
        torch.cuda.synchronize()
        check_product(x, lw.w_in, run.proj[:N * n])
        for s in range(N):
            check_mixer(cfg, run, slice(s * n, s * n + n), S0[s], A_log, dt_bias, S[int(dst[s])], False)
        check_product(run.o[:N * n], lw.w_o, y, x)
        if n == 3:
            assert np.array_equal(host(S[1]), S0[1])
        x = y


@pytest.mark.parametrize("H,Hk", [(3, 1), (5, 5)])
def test_heads_that_are_no_multiple_of_8(H, Hk):
    cfg, lw, A_log, dt_bias, rng = gdr_layer(H, Hk, 128, True, 6)
    run = L.GdrLayerRunner(cfg, 128, 70, "cuda", True)
    S = torch.zeros(1, H, D, D, device="cuda")
    slot = torch.zeros(1, dtype=torch.int32, device="cuda")
    S0 = np.zeros((H, D, D))
    for n in (70, 2):
        x, y = dev(rng.standard_normal((n, 128))), torch.empty(n, 128, dtype=torch.bfloat16, device="cuda")
        if n == 70:
            run.prefill(lw, S, slot, slot, torch.tensor([0, n], dtype=torch.int32, device="cuda"), [0, n], x, y)
        else:
            run.decode(lw, S, slot, slot, n, x, y)
        torch.cuda.synchronize()
        check_product(x, lw.w_in, run.proj[:n])
        check_mixer(cfg, run, slice(0, n), S0, A_log, dt_bias, S[0], n == 70)
        check_product(run.o[:n], lw.w_o, y, x)
        S0 = host(S[0])


@pytest.mark.parametrize("fp8", [False, True])
def test_fewer_rows_than_the_runner_was_made_for(fp8):
    """Row counts whose products are split along K, in a runner for a number of rows whose products are not."""
    cfg, lw, A_log, dt_bias, rng = gdr_layer(8, 4, 512, fp8, 8)
    run = L.GdrLayerRunner(cfg, 512, 256, "cuda", fp8)
    for B in (1, 17, 60, 129, 256):
        S = torch.zeros(B, 8, D, D, device="cuda")
        slot = torch.arange(B, dtype=torch.int32, device="cuda")
        x, y = dev(rng.standard_normal((B, 512))), torch.empty(B, 512, dtype=torch.bfloat16, device="cuda")
        run.decode(lw, S, slot, slot, 1, x, y)
        torch.cuda.synchronize()
        check_product(x, lw.w_in, run.proj[:B])
        for s in (0, B - 1):
            check_mixer(cfg, run, slice(s, s + 1), np.zeros((8, D, D)), A_log, dt_bias, S[s], False)
        check_product(run.o[:B], lw.w_o, y, x)


def test_captured_decode_step():
    cfg, lw, A_log, dt_bias, rng = gdr_layer(8, 8, 256, True, 2)
    B = 5
    run = L.GdrLayerRunner(cfg, 256, B, "cuda", True)
    S = torch.zeros(B, 8, D, D, device="cuda")
    slot = torch.arange(B, dtype=torch.int32, device="cuda")
    x, y = dev(rng.standard_normal((B, 256))), torch.empty(B, 256, dtype=torch.bfloat16, device="cuda")
    run.decode(lw, S, slot, slot, 1, x, y)
    torch.cuda.synchronize()
    want, S1 = y.clone(), S.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run.decode(lw, S, slot, slot, 1, x, y)
    S.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(S, S1)


def test_a_captured_prefill_outlives_a_larger_one():
    cfg, lw, _, _, rng = gdr_layer(2, 1, 256, False, 4)
    run = L.GdrLayerRunner(cfg, 256, 1000, "cuda")
    S, slot = torch.zeros(2, 2, D, D, device="cuda"), torch.arange(1, dtype=torch.int32, device="cuda")
    fresh = slot - 1
    bufs = {n: (dev(rng.standard_normal((n, 256))), torch.empty(n, 256, dtype=torch.bfloat16, device="cuda"),
                torch.tensor([0, n], dtype=torch.int32, device="cuda")) for n in (100, 1000)}

    def prefill(n):
        x, y, cu = bufs[n]
        run.prefill(lw, S, fresh, slot, cu, [0, n], x, y)

    g = torch.cuda.CUDAGraph()
    prefill(100)
    torch.cuda.synchronize()
    want, S1 = bufs[100][1].clone(), S.clone()
    with torch.cuda.graph(g):
        prefill(100)
    old = run.ws
    address, size = old.data_ptr(), old.numel()
    del old
    prefill(1000)
    assert run.ws.data_ptr() != address
    # what is allocated now does not get the memory that the graph writes to
    other = [torch.full((size,), 7, dtype=torch.uint8, device="cuda") for _ in range(8)]
    bufs[100][1].zero_()
    S.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(bufs[100][1], want) and torch.equal(S, S1)
    assert all(bool((t == 7).all()) for t in other)


def test_a_prefill_whose_workspace_must_grow_is_not_captured():
    cfg, lw, _, _, rng = gdr_layer(2, 1, 256, False, 5)
    run = L.GdrLayerRunner(cfg, 256, 100, "cuda")
    S, slot = torch.zeros(1, 2, D, D, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    x, y = dev(rng.standard_normal((100, 256))), torch.empty(100, 256, dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([0, 100], dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        with pytest.raises(RuntimeError):
            run.prefill(lw, S, slot, slot, cu, [0, 100], x, y)
    run.prefill(lw, S, slot, slot, cu, [0, 100], x, y)
    torch.cuda.synchronize()
    assert bool(torch.isfinite(y.float()).all())


@pytest.mark.parametrize("handle", [False, True])
def test_a_prefill_captured_on_another_stream_than_the_current_one(handle):
    """The stream that the call is given decides: a captured workspace is kept when it is replaced, and does not grow
    during the capture."""
    cfg, lw, _, _, rng = gdr_layer(2, 1, 256, False, 7)
    run = L.GdrLayerRunner(cfg, 256, 1000, "cuda")
    S, slot = torch.zeros(2, 2, D, D, device="cuda"), torch.arange(1, dtype=torch.int32, device="cuda")
    fresh = slot - 1
    bufs = {n: (dev(rng.standard_normal((n, 256))), torch.empty(n, 256, dtype=torch.bfloat16, device="cuda"),
                torch.tensor([0, n], dtype=torch.int32, device="cuda")) for n in (100, 1000)}
    side = torch.cuda.Stream()
    given = side.cuda_stream if handle else side

    def prefill(n, **kw):
        x, y, cu = bufs[n]
        run.prefill(lw, S, fresh, slot, cu, [0, n], x, y, **kw)

    prefill(100)
    torch.cuda.synchronize()
    want, S1 = bufs[100][1].clone(), S.clone()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        g.capture_begin()
    assert torch.cuda.current_stream() != side
    prefill(100, stream=given)
    with pytest.raises(RuntimeError, match="must grow"):
        prefill(1000, stream=given)
    with torch.cuda.stream(side):
        with pytest.raises(RuntimeError, match="must grow"):  # nor does a call beside the capture end it
            prefill(1000, stream=torch.cuda.default_stream())
        g.capture_end()
    address, size = run.ws.data_ptr(), run.ws.numel()
    prefill(1000)
    assert run.ws.data_ptr() != address
    other = [torch.full((size,), 7, dtype=torch.uint8, device="cuda") for _ in range(8)]
    bufs[100][1].zero_()
    S.zero_()
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(bufs[100][1], want) and torch.equal(S, S1)
    assert all(bool((t == 7).all()) for t in other)


def test_kda_layer_with_fp8_projections(oracle_mod):
    """The stacked projection and W_o of a KDA layer in FP8, decode and prefill; the mixer between them is
    the one that test_gpu_linear.py checks."""
    H, hidden, B, T = 2, 256, 3, 70
    p = KI.make_params(H, D, 4, 5)
    from tests.kda_testutil import dev_params
    rng = np.random.default_rng(5)
    mat = lambda n, k: dev(rng.standard_normal((n, k)) * k ** -0.5)
    lw = L.KdaLayerWeights(L.fp8_weight(mat(4 * H * D, hidden)), mat(D, hidden), mat(H * D, D), mat(H, hidden),
                           L.fp8_weight(mat(hidden, H * D)), dev_params(p))
    cfg = K.kda_config(H, D, K.KDA_BF16)
    st = K.kda_state_alloc(cfg, B)
    try:
        run = L.KdaLayerRunner(cfg, hidden, T, "cuda", fp8=True)
        slots = torch.arange(B, dtype=torch.int32, device="cuda")
        for n in (T, B):
            x, y = dev(rng.standard_normal((n, hidden))), torch.empty(n, hidden, dtype=torch.bfloat16, device="cuda")
            if n == T:
                cu = np.array([0, 40, 40, T], dtype=np.int32)
                run.prefill(lw, st, slots, torch.from_numpy(cu).cuda(), cu, x, y)
            else:
                run.decode(lw, st, slots, x, y)
            torch.cuda.synchronize()
            qkvg = run.qkvg.view(-1)[:4 * n * H * D].view(4, n, H * D)
            check_product(x, lw.w_qkvg, torch.cat(list(qkvg), dim=1))
            assert bool(torch.isfinite(run.o[:n].float()).all())
            check_product(run.o[:n], lw.w_o, y, x)
        assert K.kda_state_poll_error(st) == 0
    finally:
        K.kda_state_free(st)


def test_refusals():
    cfg, lw, _, _, rng = gdr_layer(8, 4, 128, True, 3)
    run = L.GdrLayerRunner(cfg, 128, 4, "cuda", fp8=False)
    S, slot = torch.zeros(4, 8, D, D, device="cuda"), torch.arange(4, dtype=torch.int32, device="cuda")
    x = dev(rng.standard_normal((4, 128)))
    with pytest.raises(TypeError):  # FP8 weights in a BF16 runner
        run.decode(lw, S, slot, slot, 1, x, torch.empty_like(x))
    run = L.GdrLayerRunner(cfg, 128, 2, "cuda", fp8=True)
    with pytest.raises(ValueError):  # more rows than it was made for
        run.decode(lw, S, slot, slot, 1, x, torch.empty_like(x))
    with pytest.raises(ValueError):
        L.GdrLayerRunner(K.kda_gdr_config(8, 4, io_dtype=K.KDA_F32), 128, 2, "cuda")
