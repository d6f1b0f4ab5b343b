"""The gated linear recurrence (kda_glr_decode, kda_glr_prefill, kda_glr_backward) against its FP64 token loop.

Tolerances are those that oracle/glr.py derives beside each result, and half a step of the rows' type for what is
rounded to it: 2^-8 of the value in BF16 (2^-133, half its smallest number, near zero), 2^-24 in FP32.
"""
import numpy as np
import pytest
import torch

import kda_inputs as KI
import linear_attention_mixer_gb300 as K
from oracle.glr import glr, grad

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from linear_attention_mixer_gb300 import build
    build.build()
    torch.cuda.set_device(0)


def np64(t):
    return t.detach().cpu().double().numpy()


def near(got, ref, err, bf16=False):
    got = np64(got)
    bound = err + (2.0 ** -8 * (np.abs(ref) + err) + 2.0 ** -133 if bf16 else 2.0 ** -24 * np.abs(ref)) + 1e-37
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), (int(bad.sum()), float(np.nanmax(np.abs(got - ref) / bound)))


class Problem:
    """Seeded rows of packed sequences, on the host (as the row type rounds them) and on the device."""

    def __init__(self, lens, D, bf16=True, gate=True, packed=False, seed=0, edit=None, slow=False):
        rng = np.random.default_rng([seed, len(lens), D])
        self.lens, self.D, self.bf16, self.gate = list(lens), D, bf16, gate
        T, N = sum(lens), len(lens)
        self.T, self.N = T, N
        self.cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        self.names = ("x", "a", "b", "g") if gate else ("x", "a", "b")
        h = {n: rng.standard_normal((T, D)).astype(np.float32) for n in self.names + ("dout",)}
        h["A_log"] = (np.log(0.002) + rng.uniform(0, np.log(1000.0), D)).astype(np.float32) - (6 if slow else 0)
        h["a_bias"], h["b_bias"] = (rng.standard_normal((2, D)) * 0.7).astype(np.float32)
        h["h0"], h["dS"] = (rng.standard_normal((2, N, D)) * 0.5).astype(np.float32)
        if edit:
            edit(h)
        with np.errstate(invalid="ignore"):
            self.h = h | {n: KI.bf16_round(h[n]) if bf16 else h[n] for n in self.names + ("dout",)}
        self.dt = torch.bfloat16 if bf16 else torch.float32
        self.dev = {n: torch.from_numpy(self.h[n]).cuda().to(self.dt if n in self.names + ("dout",) else torch.float32) for n in self.h}
        if packed:  # columns of one wide tensor, with columns between and behind that belong to nobody
            step = D + 8
            wide = torch.full((T, len(self.names) * step + 16), float("nan"), dtype=self.dt, device="cuda")
            for i, n in enumerate(self.names):
                wide[:, i * step:i * step + D] = self.dev[n]
                self.dev[n] = wide[:, i * step:i * step + D]
        self.cfg = K.kda_glr_config(D, K.KDA_BF16 if bf16 else K.KDA_F32)
        self.params = K.kda_glr_params_from(*(self.dev[n] for n in ("A_log", "a_bias", "b_bias")))
        self.out = torch.full((T + 3, D), -7.0, dtype=self.dt, device="cuda")
        self.starts = torch.full((K.kda_glr_chunks(self.cu), D), float("nan"), device="cuda")
        self.work = torch.empty(K.kda_glr_workspace_bytes(self.cfg, self.cu), dtype=torch.uint8, device="cuda").fill_(0xFF)
        self.cu_dev = torch.from_numpy(self.cu).cuda()
        self.S = torch.full((2 * N + 2, D), 3.0, device="cuda")
        self.S[:N] = self.dev["h0"]
        self.src = torch.arange(N, dtype=torch.int32, device="cuda")
        self.dst = self.src + N
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def rows(self):
        return tuple(self.dev[n] if n in self.dev else None for n in "xabg")

    def prefill(self, starts=True, sync=True, **kw):
        K.kda_glr_prefill(self.cfg, self.params, self.S, self.src, self.dst, self.cu_dev, self.cu, *self.rows(), self.out[:self.T], self.work,
                          starts=self.starts if starts else None, err=self.err, **kw)
        if sync:
            torch.cuda.synchronize()

    def make_grads(self):
        g = {n: torch.full((self.T + 2, self.D), -7.0, dtype=self.dt, device="cuda") for n in ("dx", "da", "db") + (("dg",) if self.gate else ())}
        g |= {n: torch.full((self.D,), float("nan"), device="cuda") for n in ("dA_log", "da_bias", "db_bias")}
        g["dS"] = torch.full((self.N, self.D), float("nan"), device="cuda")
        return g

    def backward(self, g=None, dS=True, sync=True, **kw):
        g = g or self.make_grads()
        row = {n: g[n][:self.T] if n in g else None for n in ("dx", "da", "db", "dg")}
        K.kda_glr_backward(self.cfg, self.params, self.cu_dev, self.cu, self.starts, *self.rows(), self.dev["dout"], work=self.work,
                           dS_last=self.dev["dS"] if dS else None, dS_first=g["dS"], dA_log=g["dA_log"], da_bias=g["da_bias"],
                           db_bias=g["db_bias"], err=self.err, **row, **kw)
        if sync:
            torch.cuda.synchronize()
        return g

    def args(self, s, h0=None):
        r = slice(self.cu[s], self.cu[s + 1])
        return tuple(self.h[n][r] if n in self.h else None for n in "xabg") + tuple(self.h[n] for n in ("A_log", "a_bias", "b_bias")) + \
            (self.h["h0"][s] if h0 is None else h0,)

    def check(self, h0s=None):
        for s in range(self.N):
            f = glr(*self.args(s, None if h0s is None else h0s[s]))
            near(self.out[self.cu[s]:self.cu[s + 1]], f["out"], f["out_err"], self.bf16)
            near(self.S[int(self.dst[s])], f["S"], f["S_err"])
        assert bool((self.out[self.T:] == -7.0).all())
        assert int(self.err.item()) == 0

    def check_grads(self, g, dS=True):
        sums = {n: [0.0, 0.0] for n in ("dA_log", "da_bias", "db_bias")}
        for s in range(self.N):
            r = slice(self.cu[s], self.cu[s + 1])
            f = grad(*self.args(s), self.h["dout"][r], self.h["dS"][s] * (1.0 if dS else 0.0))
            for n in ("dx", "da", "db") + (("dg",) if self.gate else ()):
                near(g[n][r], f[n], f[n + "_err"], self.bf16)
            near(g["dS"][s], f["dS"], f["dS_err"])
            for n in sums:
                sums[n][0] += f[n]
                sums[n][1] += f[n + "_err"]
        for n, (v, e) in sums.items():
            near(g[n], v, e + 2.0 ** -24 * self.N * e + 2.0 ** -22 * np.abs(v))
        for n in ("dx", "da", "db"):
            assert bool((g[n][self.T:] == -7.0).all())


SHAPES = [([1], 64, True, True, False), ([5], 8, True, False, True), ([16], 72, True, True, True), ([17, 1, 0, 40], 200, True, False, False),
          ([2], 4, False, True, False), ([100, 31], 68, False, False, True), ([0, 0, 129], 1004, False, True, False), ([0], 16, True, True, False),
          ([128], 128, True, True, False), ([600, 127, 1], 136, True, True, True), ([1025], 64, False, False, False),
          ([2100, 3], 320, True, False, False), ([4100], 8, False, True, True)]


@pytest.mark.parametrize("lens,D,bf16,gate,packed", SHAPES)
def test_prefill_and_backward(lens, D, bf16, gate, packed):
    p = Problem(lens, D, bf16, gate, packed)
    p.prefill()
    p.check()
    p.check_grads(p.backward())


@pytest.mark.parametrize("lens,D,bf16,gate,packed,slow", [([20000], 72, True, True, False, True), ([9000, 3, 0, 16384], 64, False, False, True, False),
                                                          ([0, 33000, 1025], 8, True, False, True, True), ([5000, 12288, 4097], 200, True, True, False, False),
                                                          ([70001], 4, False, True, False, True)])
def test_long_sequences_of_few_channels(lens, D, bf16, gate, packed, slow):
    """Sequences in parts that are worked on at once, also into the slots that they came from."""
    p = Problem(lens, D, bf16, gate, packed, seed=17, slow=slow)
    p.dst = p.src
    p.prefill()
    p.check()
    got = p.backward()
    p.check_grads(got)
    first = p.out.clone()
    p.S[:p.N] = p.dev["h0"]
    p.prefill(starts=False)
    again = p.backward()
    assert torch.equal(first, p.out) and all(torch.equal(got[n], again[n]) for n in got)


@pytest.mark.parametrize("D,bf16", [(12288, True), (7168, False)])
def test_wide_rows(D, bf16):
    p = Problem([150, 20], D, bf16, seed=1)
    p.prefill()
    p.check()
    p.check_grads(p.backward())


@pytest.mark.parametrize("count,top,D,bf16,gate,packed", [(700, 8, 40, True, True, False), (300, 16, 256, True, False, True), (2000, 2, 72, False, True, False),
                                                         (150, 64, 1024, True, True, True), (90, 200, 520, False, True, False), (30, 33, 2048, False, False, True)])
def test_many_short_sequences(count, top, D, bf16, gate, packed):
    """Both ways of a prefill, and blocks of one warp and of four in the backward."""
    lens = list(np.random.default_rng(5).integers(0, top + 1, count))
    p = Problem(lens, D, bf16, gate, packed, seed=2)
    p.prefill()
    p.check()
    got = p.backward()
    p.check_grads(got)
    first = p.out.clone()
    p.prefill(starts=False)
    again = p.backward()
    assert torch.equal(first, p.out) and all(torch.equal(got[n], again[n]) for n in got)


def test_a_long_memory():
    """1 - alpha down to 1e-6: the steady state needs more than alpha in FP32."""
    def edit(h):
        h["a"][:] = 0.25  # the same decay at every token, so that an error of alpha adds up
        h["x"] += 1.0
    p = Problem([3000], 64, False, False, seed=3, edit=edit, slow=True)
    p.prefill()
    p.check()
    p.check_grads(p.backward())


def test_without_starts_and_without_a_final_gradient():
    p = Problem([70, 9], 96, True, True, seed=4)
    p.prefill(starts=False)
    p.check()
    q = Problem([70, 9], 96, True, True, seed=4)
    q.prefill()
    assert torch.equal(p.out, q.out) and torch.equal(p.S, q.S)
    q.check_grads(q.backward(dS=False), dS=False)


def test_gates_at_their_ends():
    """a or b infinite or far out: a state kept, dropped, or closed to the input; and an output gate far out."""
    rng = np.random.default_rng(6)

    def edit(h):
        for n in "ab":
            m = rng.integers(0, 9, h[n].shape)
            for i, v in enumerate((-np.inf, np.inf, -60.0, 60.0, -95.0)):
                h[n][m == i] = v
        h["g"][rng.integers(0, 5, h["g"].shape) == 0] = -70.0
        h["g"][rng.integers(0, 5, h["g"].shape) == 0] = 90.0
        h["A_log"][::3] = 6.0
    p = Problem([200, 33], 72, False, True, seed=6, edit=edit)
    p.prefill()
    p.check()
    p.check_grads(p.backward())


def test_only_kept_states():
    """a = -inf and nothing let in: out repeats the state to the bit."""
    def edit(h):
        h["a"][:] = -np.inf
        h["b"][::2] = -np.inf
    p = Problem([300], 64, False, False, seed=7, edit=edit)
    p.prefill()
    assert bool((p.out[:300] == p.dev["h0"]).all()) and torch.equal(p.S[1], p.dev["h0"][0])


def test_what_is_not_finite_stays_behind():
    """A NaN reaches its own channel of its own sequence, from its token on."""
    for name in "xab":
        p = Problem([150, 150], 64, True, False, seed=8)
        q = Problem([150, 150], 64, True, False, seed=8)
        q.dev[name][90, 5] = float("nan")
        p.prefill()
        q.prefill()
        same = torch.ones(300, 64, dtype=torch.bool, device="cuda")
        same[90:150, 5] = False
        assert torch.equal(p.out[:300][same], q.out[:300][same])
        assert bool(q.out[90:150, 5].isnan().all()) and bool(q.S[2, 5].isnan()) and torch.equal(p.S[3], q.S[3])


def test_slots():
    """Zero states, forks and states taken back; a slot read twice; rows with bad ids are left alone."""
    p = Problem([20, 20, 20], 64, True, True, seed=9)
    p.src[:] = torch.tensor([-1, 1, 1], dtype=torch.int32)
    p.dst[:] = torch.tensor([0, 5, 3], dtype=torch.int32)
    p.prefill()
    p.check([np.zeros(64), p.h["h0"][1], p.h["h0"][1]])
    for src, dst in ((-2, 3), (8, 3), (0, -1), (0, 8)):
        q = Problem([20, 20, 20], 64, True, True, seed=9)
        q.src[1], q.dst[1] = src, dst
        S = q.S.clone()
        q.prefill()
        assert int(q.err.item()) == K.KDA_ERR_DEVICE
        assert bool((q.out[20:40] == -7.0).all())
        for s in (0, 2):
            f = glr(*q.args(s))
            near(q.out[20 * s:20 * s + 20], f["out"], f["out_err"], True)
            S[3 + s] = q.S[3 + s]
        assert torch.equal(S, q.S)


def test_bounds_that_do_not_rise():
    """Sequences whose bounds are wrong on the device are left alone."""
    for cu in ([0, 30, 20, 60], [0, 20, 40, 61], [5, 20, 40, 60], [0, 20, 2 ** 30, 60], [-16, 20, 40, 60]):
        p = Problem([20, 20, 20], 64, True, True, seed=10)
        p.prefill()
        good = p.out.clone()
        p.out[:] = -7.0
        p.cu_dev.copy_(torch.tensor(cu, dtype=torch.int32))
        p.prefill()
        assert int(p.err.item()) == K.KDA_ERR_DEVICE
        p.err.zero_()
        for s in range(3):
            if cu[s:s + 2] == [20 * s, 20 * s + 20] and not any(a < 20 * s + 20 and b > 20 * s for a, b in zip(cu[:s], cu[1:])):
                assert torch.equal(p.out[20 * s:20 * s + 20], good[20 * s:20 * s + 20])
        p.starts.zero_()
        p.backward()
        assert int(p.err.item()) == K.KDA_ERR_DEVICE


@pytest.mark.parametrize("n", [1, 2, 5, 8])
@pytest.mark.parametrize("B,D,bf16,gate,packed", [(1, 8, True, True, False), (3, 4096, True, False, True), (7, 68, False, True, True),
                                                   (300, 64, False, False, False)])
def test_decode(n, B, D, bf16, gate, packed):
    p = Problem([n] * B, D, bf16, gate, packed, seed=11)
    p.src[0] = -1
    K.kda_glr_decode(p.cfg, p.params, p.S, p.src, p.dst, n, *p.rows(), p.out[:p.T], err=p.err)
    torch.cuda.synchronize()
    p.check([np.zeros(D)] + list(p.h["h0"][1:]))


def test_decode_in_place_after_a_prefill():
    """A prompt, then its tokens one by one and three at a time in the same slot: as one sequence."""
    p = Problem([57], 80, True, True, seed=12)
    q = Problem([50], 80, True, True, seed=12)
    for n in "xabg":
        q.dev[n] = p.dev[n][:50]
    q.params = p.params
    q.S[0] = p.S[0]
    q.prefill()
    slot = q.dst
    at = 50
    for n in (1, 3, 3):
        K.kda_glr_decode(p.cfg, p.params, q.S, slot, slot, n, *(p.dev[c][at:at + n] for c in "xabg"), p.out[at:at + n])
        at += n
    torch.cuda.synchronize()
    p.out[:50] = q.out[:50]
    p.S[1] = q.S[1]
    p.check()


def test_twice_the_same_and_on_another_stream():
    p = Problem([900, 40], 128, True, True, seed=13)
    p.prefill()
    first = (p.out.clone(), p.S.clone(), p.backward())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    p.out.fill_(-7.0)
    torch.cuda.synchronize()
    p.prefill(stream=s, sync=False)
    g = p.make_grads()
    torch.cuda.synchronize()
    p.backward(g, stream=s.cuda_stream)
    assert torch.equal(first[0], p.out) and torch.equal(first[1], p.S)
    for n in g:
        assert torch.equal(first[2][n], g[n]), n


def test_captured_and_replayed():
    """A training step and a decode step in one graph, replayed on other rows."""
    p = Problem([130, 7], 72, True, True, seed=14)
    g = p.make_grads()
    p.prefill()
    p.backward(g)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.prefill(sync=False)
        p.backward(g, sync=False)
    q = Problem([130, 7], 72, True, True, seed=15)
    for n in p.names + ("dout", "h0", "dS"):
        p.dev[n].copy_(q.dev[n])
        p.h[n] = q.h[n]
    p.S[:2] = q.dev["h0"]
    graph.replay()
    torch.cuda.synchronize()
    p.check()
    p.check_grads(g)


def test_offsets_beyond_32_bits():
    """Rows whose distance makes the last one lie more than 2^31 elements behind the first."""
    T, D, stride = 70, 64, 1 << 25
    p = Problem([T], D, True, False, seed=16)
    wide = torch.empty(T * stride, dtype=torch.bfloat16, device="cuda").as_strided((T, 4 * D), (stride, 1))
    for i, n in enumerate("xab"):
        wide[:, i * D:i * D + D] = p.dev[n]
        p.dev[n] = wide[:, i * D:i * D + D]
    out = wide[:, 3 * D:]
    K.kda_glr_prefill(p.cfg, p.params, p.S, p.src, p.dst, p.cu_dev, p.cu, *p.rows(), out, p.work, starts=p.starts, err=p.err)
    p.out[:T] = out
    torch.cuda.synchronize()
    p.check()
    p.check_grads(p.backward())


def test_no_sequences():
    cfg = K.kda_glr_config(64)
    prm = K.kda_glr_params_from(*(torch.zeros(64, device="cuda") for _ in range(3)))
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    cu = torch.zeros(1, dtype=torch.int32, device="cuda")
    row = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    S, ws, sums = torch.ones(1, 64, device="cuda"), torch.empty(256, dtype=torch.uint8, device="cuda"), [torch.ones(64, device="cuda") for _ in range(3)]
    K.kda_glr_prefill(cfg, prm, S, none, none, cu, [0], row, row, row, None, row, ws)
    K.kda_glr_decode(cfg, prm, S, none, none, 1, row, row, row, None, row)
    K.kda_glr_backward(cfg, prm, cu, [0], torch.empty(0, 64, device="cuda"), row, row, row, None, row, row, row, row, None, ws,
                       dA_log=sums[0], da_bias=sums[1], db_bias=sums[2])
    torch.cuda.synchronize()
    assert bool((S == 1).all()) and all(bool((s == 0).all()) for s in sums)


def test_refusals_of_the_binding():
    p = Problem([20, 5], 64, True, True, seed=18)
    x, a, b, g = p.rows()
    out = p.out[:p.T]

    def prefill(S=p.S, src=p.src, dst=p.dst, cu=p.cu_dev, cuh=p.cu, x=x, a=a, b=b, g=g, out=out, ws=p.work, starts=p.starts, prm=p.params, err=p.err):
        K.kda_glr_prefill(p.cfg, prm, S, src, dst, cu, cuh, x, a, b, g, out, ws, starts=starts, err=err)

    def backward(**e):
        v = p.make_grads() | {"starts": p.starts, "dS_last": p.dev["dS"], "dout": p.dev["dout"], "x": x} | e
        K.kda_glr_backward(p.cfg, p.params, p.cu_dev, p.cu, v["starts"], v["x"], a, b, g, v["dout"], v["dx"][:p.T], v["da"][:p.T], v["db"][:p.T], v["dg"][:p.T],
                           p.work, dS_last=v["dS_last"], dA_log=v["dA_log"])

    other = K.kda_glr_params_from(*(torch.zeros(72, device="cuda") for _ in range(3)))
    by_hand = K.kda_glr_params(p.params.A_log, p.params.a_bias, p.params.b_bias)
    for e in ({"x": x.float()}, {"x": x[:-1]}, {"a": a.t()}, {"b": b.cpu()}, {"g": g[:, :32]}, {"out": torch.zeros(p.T, 128, dtype=p.dt, device="cuda")[:, ::2]},
              {"S": p.S[:, :32]}, {"S": p.S.double()}, {"src": p.src.long()}, {"dst": p.dst[:1]}, {"cu": p.cu_dev[:-1]}, {"cuh": [0, 20]}, {"cuh": [0, 20, 26]},
              {"starts": p.starts[:1]}, {"starts": p.starts.half()}, {"ws": p.work[:100]}, {"ws": p.work.cpu()}, {"prm": other}, {"prm": by_hand}, {"err": p.src.cpu()},
              {"x": None}, {"x": 3}, {"cuh": [0, 30, 25]}):
        with pytest.raises((TypeError, ValueError, AttributeError, K.KdaError)):
            prefill(**e)
    for e in ({"x": x.float()}, {"dout": p.dev["dout"][:3]}, {"starts": p.starts[:1]}, {"dS_last": p.dev["dS"][:1]}, {"dA_log": torch.zeros(63, device="cuda")}):
        with pytest.raises((TypeError, ValueError, K.KdaError)):
            backward(**e)
    with pytest.raises(ValueError):
        K.kda_glr_params_from(*(torch.zeros(n, device="cuda") for n in (64, 64, 72)))
    with pytest.raises(TypeError):
        K.kda_glr_params_from(*(torch.zeros(64, device="cuda", dtype=torch.float64) for _ in range(3)))
    for n in (0, 9):
        with pytest.raises((K.KdaError, ValueError)):
            K.kda_glr_decode(p.cfg, p.params, p.S, p.src, p.dst, n, *p.rows(), out)
    p.prefill()  # nothing was touched
    p.check()


FIRST = """
import torch
import linear_attention_mixer_gb300 as K
f32 = dict(device="cuda")
cfg, T, D, cu_h = K.kda_glr_config(72), 700, 72, [0, 700]
v = [torch.randn(D, **f32) for _ in range(3)]
prm = K.kda_glr_params_from(*v)
rows = [torch.randn(T, D, **f32).bfloat16() for _ in range(5)]
out, dx, da, db, dg = (torch.empty_like(rows[0]) for _ in range(5))
S, slot, cu = torch.zeros(1, D, **f32), torch.zeros(1, dtype=torch.int32, **f32), torch.tensor(cu_h, dtype=torch.int32, **f32)
ws = torch.empty(K.kda_glr_workspace_bytes(cfg, cu_h), dtype=torch.uint8, **f32)
starts, dA = torch.empty(K.kda_glr_chunks(cu_h), D, **f32), torch.empty(D, **f32)
nc, np_ = K.kda_block_norm_config(D), K.kda_block_norm_params_from(*v)
h, x1 = torch.empty_like(out), torch.empty_like(out)

def step():
    K.kda_glr_prefill(cfg, prm, S, slot, slot, cu, cu_h, *rows[:4], out, ws, starts=starts)
    K.kda_glr_backward(cfg, prm, cu, cu_h, starts, *rows, dx, da, db, dg, ws, dA_log=dA)
    K.kda_block_norm(nc, np_, rows[0], y=out, x_out=x1, h=h)

torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    step()
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in (out, dx, da, db, dg, dA, h, x1)]
S.zero_()
step()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, (out, dx, da, db, dg, dA, h, x1)))
print("same")
"""


def test_the_first_call_of_a_process_is_captured():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stderr[-2000:]
