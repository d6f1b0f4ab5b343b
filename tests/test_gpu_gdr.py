"""The gated delta rule (kda_gdr_decode, kda_gdr_prefill) against its FP64 token recurrence.

Tolerances, from the arithmetic (half a step of BF16 is 2^-8 of the value, of FP32 2^-24):
  out, BF16 rows, recurrent: the rounding of the result, 2^-8 |o|, and FP32 sums of at most 128 + a few
      terms, below 2^-12 mag (mag: the sums of absolute values, oracle/gdr.py).
  out, BF16 rows, chunked: that, and the products Q S0 with S0 rounded to BF16 (2^-8 of the sum of
      absolute terms) and P U with both rounded (2 x 2^-8): at most 2^-7 mag (1 + 2^-8).
  state, chunked: every product that feeds the state splits its inexact factors into two BF16 (2^-16 of
      the value is lost) and drops lo x lo (2^-16): five such losses between S0 and S, so 5 x 2^-16 of
      the state in the 2-norm where its terms do not cancel, and of oracle/gdr.py's bound where they do.
  FP32 rows and the recurrent state: each of the three sums over 128 terms is 16 + 3 additions deep,
      fewer than 64 roundings a token with the gates: 64 x 2^-24 = 2^-18 in the 2-norm; elements of out
      within 2^-18 mag.
"""
import numpy as np
import pytest
import torch

import kda_inputs as KI
import linear_attention_mixer_gb300 as K
from oracle.gdr import gdr

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module", autouse=True)
def _built():
    from linear_attention_mixer_gb300 import build
    build.build()
    torch.cuda.set_device(0)


class Problem:
    """Seeded rows of packed sequences on the host (values already rounded to the row type) and the device."""

    def __init__(self, lens, H, Hk, bf16=True, seed=0, packed=True, states=None, edit=None, l2norm=True):
        rng = np.random.default_rng([seed, len(lens), H, Hk])
        self.lens, self.H, self.Hk, self.bf16, self.l2norm = list(lens), H, Hk, bf16, l2norm
        T = self.T = sum(lens)
        self.cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        silu = lambda x: x / (1 + np.exp(-x))
        scale = 1.0 if l2norm else D ** -0.5
        h = {"q": silu(rng.standard_normal((T, Hk * D))) * scale, "k": silu(rng.standard_normal((T, Hk * D))) * scale,
             "v": silu(rng.standard_normal((T, H * D))), "a": rng.standard_normal((T, H)),
             "b": rng.standard_normal((T, H))}
        h = {n: x.astype(np.float32) for n, x in h.items()}
        if edit:
            edit(h)
        with np.errstate(invalid="ignore"):
            self.h = {n: KI.bf16_round(x) if bf16 else x for n, x in h.items()}
        self.A_log = rng.uniform(0, np.log(16.0), H).astype(np.float32)
        self.dt_bias = (rng.standard_normal(H) * 0.7).astype(np.float32)
        N = len(lens)
        self.S0 = (rng.standard_normal((N, H, D, D)) * 0.05).astype(np.float32) if states is None else states
        dt = torch.bfloat16 if bf16 else torch.float32
        dev = {n: torch.from_numpy(x).to(dt).cuda() for n, x in self.h.items()}
        if packed:  # columns of one wide tensor, with columns between and behind that belong to nobody
            at, cols = 0, {}
            for n in ("a", "q", "b", "k", "v"):
                if n in "qkv":
                    at = -(-at // 8) * 8
                cols[n] = at
                at += dev[n].shape[1] + 1
            wide = torch.full((T, -(-at // 8) * 8 + 8), float("nan"), dtype=dt, device="cuda")
            for n, c in cols.items():
                wide[:, c:c + dev[n].shape[1]] = dev[n]
                dev[n] = wide[:, c:c + dev[n].shape[1]]
        self.dev = dev
        self.cfg = K.kda_gdr_config(H, Hk, D, K.KDA_BF16 if bf16 else K.KDA_F32)
        self.cfg.qk_l2norm = int(l2norm)
        self.params = K.kda_gdr_params_from(torch.from_numpy(self.A_log).cuda(), torch.from_numpy(self.dt_bias).cuda())
        self.out = torch.full((T + 3, H * D), -7.0, dtype=dt, device="cuda")

    def slots(self, spare=2):
        N = len(self.lens)
        S = torch.full((2 * N + spare, self.H, D, D), 3.0, device="cuda")
        S[:N] = torch.from_numpy(self.S0).cuda()
        return S, torch.arange(N, dtype=torch.int32, device="cuda"), torch.arange(N, 2 * N, dtype=torch.int32, device="cuda")

    def rows(self):
        return tuple(self.dev[n] for n in "qkvab") + (self.out[:self.T],)

    def prefill(self, S, src, dst, **kw):
        ws = torch.empty(K.kda_gdr_workspace_bytes(self.cfg, self.cu), dtype=torch.uint8, device="cuda").fill_(0xFF)
        K.kda_gdr_prefill(self.cfg, self.params, S, src, dst, torch.from_numpy(self.cu).cuda(), self.cu, *self.rows(), ws, **kw)
        torch.cuda.synchronize()

    def decode(self, S, src, dst, n, **kw):
        K.kda_gdr_decode(self.cfg, self.params, S, src, dst, n, *self.rows(), **kw)
        torch.cuda.synchronize()

    def ref(self, s, S0=None, head=None):
        """Oracle of sequence s: o [T, H d], S, mag."""
        r = slice(self.cu[s], self.cu[s + 1])
        n = self.lens[s]
        g = lambda x, m: self.h[x][r].reshape(n, m, D)
        o, S, mag, self.col = gdr(g("q", self.Hk), g("k", self.Hk), g("v", self.H), self.h["a"][r], self.h["b"][r], self.A_log,
                        self.dt_bias, self.S0[s] if S0 is None else S0, self.l2norm)
        return o.reshape(n, self.H * D), S, mag.reshape(n, self.H * D)


def near(got, ref, mag, bf16, chunked):
    got = got.float().cpu().numpy().astype(np.float64)
    if not bf16:
        bound = 2.0 ** -18 * mag
    else:
        bound = 2.0 ** -8 * np.abs(ref) + (2.0 ** -7 * (1 + 2.0 ** -8) if chunked else 2.0 ** -12) * mag
    bad = ~(np.abs(got - ref) <= bound + 1e-30)
    assert not bad.any(), (int(bad.sum()), float(np.nanmax(np.abs(got - ref) / (bound + 1e-30))))


def near_state(got, ref, chunked):
    got = got.cpu().numpy().astype(np.float64)
    tol = 5 * 2.0 ** -16 if chunked else 2.0 ** -18
    e, n = np.linalg.norm(got - ref), np.linalg.norm(ref)
    assert e <= tol * n + 1e-30, (e / n if n else e, tol)


def near_columns(got, ref, col, chunked):
    """near_state for keys that make the state's terms cancel: per value column, against oracle/gdr.py's bound."""
    e = np.linalg.norm(got.cpu().numpy().astype(np.float64) - ref, axis=1)
    tol = 5 * 2.0 ** -16 if chunked else 2.0 ** -18
    assert (e <= tol * col).all(), float((e / (tol * col)).max())


def check(p, S, src, dst, S0s, chunked):
    for s in range(len(p.lens)):
        o, Sr, mag = p.ref(s, S0s[s])
        near(p.out[p.cu[s]:p.cu[s + 1]], o, mag, p.bf16, chunked)
        near_state(S[int(dst[s])], Sr, chunked)
    assert bool((p.out[p.T:] == -7.0).all())  # rows behind the last sequence


@pytest.mark.parametrize("n", [1, 2, 8])
@pytest.mark.parametrize("B,H,Hk,bf16,packed", [(1, 2, 1, True, True), (5, 4, 4, True, False), (3, 6, 2, False, True),
                                                 (1, 3, 3, False, False)])
def test_decode(n, B, H, Hk, bf16, packed):
    p = Problem([n] * B, H, Hk, bf16, seed=1, packed=packed)
    S, src, dst = p.slots()
    keep = S.clone()
    p.decode(S, src, dst, n)
    check(p, S, src, dst, p.S0, False)
    assert torch.equal(S[:B], keep[:B]) and torch.equal(S[2 * B:], keep[2 * B:])  # sources and spare slots


@pytest.mark.parametrize("lens", [[1], [63], [64], [65], [128], [200], [0, 1, 0, 130, 64, 2, 0]])
@pytest.mark.parametrize("H,Hk,bf16,packed", [(2, 1, True, True), (3, 3, True, False), (4, 1, True, True), (9, 1, True, False),
                                               (4, 2, False, True)])
def test_prefill(lens, H, Hk, bf16, packed):
    p = Problem(lens, H, Hk, bf16, seed=2, packed=packed)
    S, src, dst = p.slots()
    keep = S.clone()
    p.prefill(S, src, dst)
    check(p, S, src, dst, p.S0, bf16)
    N = len(lens)
    assert torch.equal(S[:N], keep[:N]) and torch.equal(S[2 * N:], keep[2 * N:])


@pytest.mark.parametrize("lens,bf16", [([3, 70, 1, 129, 64, 65, 0, 33, 90], True), ([3, 70, 1, 129, 64, 65, 0, 33, 90], False),
                                       ([200], True)])
def test_many_heads(lens, bf16):
    """Many short sequences (more blocks than SMs: 64 value columns each) and one of as many heads (32 columns)."""
    p = Problem(lens, 32, 16, bf16, seed=3)
    S, src, dst = p.slots()
    p.prefill(S, src, dst)
    check(p, S, src, dst, p.S0, bf16)


@pytest.mark.parametrize("bf16", [True, False])
def test_many_sequences(bf16):
    """More sequences than a block has threads, empty ones and ones of several chunks among them."""
    p = Problem([(0, 1, 3, 0, 2)[i % 5] for i in range(400)] + [0] * 70 + [130, 1, 0, 65] + [1, 0] * 20, 2, 1, bf16, seed=19)
    S, src, dst = p.slots()
    p.prefill(S, src, dst)
    check(p, S, src, dst, p.S0, bf16)


@pytest.mark.parametrize("bf16", [True, False])
def test_fresh_in_place_and_forked_rows(bf16):
    """src -1 starts from zeros without reading a slot, src == dst updates in place, one src may serve two rows."""
    p = Problem([70, 20, 65, 65], 2, 2, bf16, seed=4)
    S, src, dst = p.slots()
    S[5] = float("nan")
    src = torch.tensor([-1, 1, 2, 2], dtype=torch.int32, device="cuda")
    dst = torch.tensor([5, 1, 6, 7], dtype=torch.int32, device="cuda")
    p.prefill(S, src, dst)
    zero = np.zeros_like(p.S0[0])
    check(p, S, src, dst, [zero, p.S0[1], p.S0[2], p.S0[2]], bf16)
    p = Problem([1, 1], 2, 2, bf16, seed=5)
    S, _, _ = p.slots()
    S[1] = float("inf")
    p.decode(S, torch.tensor([-1, 0], dtype=torch.int32, device="cuda"), torch.tensor([1, 0], dtype=torch.int32, device="cuda"), 1)
    check(p, S, None, [1, 0], [zero, p.S0[0]], False)


def test_prefill_then_decode_equals_one_prefill_of_all():
    p = Problem([150], 4, 2, True, seed=6)
    S, src, dst = p.slots()
    p.prefill(S, src, dst)
    o, Sr, mag = p.ref(0)
    for cut in (64, 100):
        S2 = S.clone()
        S2[0] = torch.from_numpy(p.S0[0]).cuda()
        out = torch.empty_like(p.out)
        ws = torch.empty(K.kda_gdr_workspace_bytes(p.cfg, [0, cut]), dtype=torch.uint8, device="cuda")
        rows = [x[:cut] for x in p.rows()[:5]] + [out[:cut]]
        K.kda_gdr_prefill(p.cfg, p.params, S2, src, src, torch.tensor([0, cut], dtype=torch.int32, device="cuda"), [0, cut], *rows, ws)
        for t in range(cut, 150, 5):
            n = min(5, 150 - t)
            rows = [x[t:t + n] for x in p.rows()[:5]] + [out[t:t + n]]
            K.kda_gdr_decode(p.cfg, p.params, S2, src, src, n, *rows)
        torch.cuda.synchronize()
        near(out[:150], o, mag, True, True)
        near_state(S2[0], Sr, True)


@pytest.mark.parametrize("bf16", [True, False])
def test_raw_keys(bf16):
    p = Problem([100, 31], 2, 1, bf16, seed=7, l2norm=False)
    S, src, dst = p.slots()
    p.prefill(S, src, dst)
    check(p, S, src, dst, p.S0, bf16)


@pytest.mark.parametrize("bf16", [True, False])
def test_gate_extremes(bf16):
    """Decays that reset the state (alpha 0) and that keep it (alpha 1), beta 0 and 1, in every position of a chunk."""
    def edit(h):
        rng = np.random.default_rng(9)
        T, H = h["a"].shape
        h["a"][:] = rng.choice([-60.0, -3.0, 0.0, 3.0, 60.0, 3e38, -np.inf], size=(T, H))
        h["b"][:] = rng.choice([-100.0, -2.0, 0.0, 100.0, np.inf], size=(T, H))
    p = Problem([190, 7], 3, 1, bf16, seed=8, edit=edit)
    S, src, dst = p.slots()
    p.prefill(S, src, dst)
    check(p, S, src, dst, p.S0, bf16)
    def edit_one(h):
        h["a"][:], h["b"][:] = -30.0, 30.0  # nothing decays, everything is replaced: the state only grows or turns
        h["k"][:] = np.abs(h["k"]) + 0.3    # and the keys are strongly correlated
    p = Problem([256], 2, 2, bf16, seed=10, edit=edit_one)
    S, src, dst = p.slots()
    p.prefill(S, src, dst)
    o, Sr, mag = p.ref(0)
    near(p.out[:256], o, mag, bf16, bf16)
    near_columns(S[1], Sr, p.col, bf16)


def test_zero_rows():
    """Zero keys and queries (their norm is sqrt(eps)) and zero values."""
    def edit(h):
        h["k"][3:40], h["q"][20:70], h["v"][5:90] = 0, 0, 0
    for bf16 in (True, False):
        p = Problem([130], 2, 1, bf16, seed=11, edit=edit)
        S, src, dst = p.slots()
        p.prefill(S, src, dst)
        check(p, S, src, dst, p.S0, bf16)


def test_what_is_not_finite_stays_in_its_sequence():
    """NaN and infinity in one sequence's rows reach that sequence alone, whatever shares its 64-row tiles."""
    def edit(h):
        for n in "qkvab":
            h[n][70:75] = np.nan
            h[n][75:80] = np.inf
    p = Problem([70, 10, 60], 2, 1, True, seed=12, edit=edit)
    S, src, dst = p.slots()
    p.prefill(S, src, dst)
    for s in (0, 2):
        o, Sr, mag = p.ref(s)
        near(p.out[p.cu[s]:p.cu[s + 1]], o, mag, True, True)
        near_state(S[int(dst[s])], Sr, True)
    assert bool(torch.isnan(S[int(dst[1])]).any())


def test_bad_slots_and_lengths_are_recorded():
    p = Problem([66, 5, 9], 2, 2, True, seed=13)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for bad_src, bad_dst in ((-2, 4), (99, 4), (1, -1), (1, 99)):
        S, src, dst = p.slots()
        keep = S.clone()
        src[1], dst[1] = bad_src, bad_dst
        p.out.fill_(-7.0)
        err.zero_()
        p.prefill(S, src, dst, err=err)
        assert err.item() == K.KDA_ERR_DEVICE
        assert bool((p.out[66:71] == -7.0).all()) and torch.equal(S[4], keep[4])
        near_state(S[3], p.ref(0)[1], True)
        near_state(S[5], p.ref(2)[1], True)
    # a device cu_seqlens that is not the host's: nothing is written
    for wrong in ([0, 66, 71, 79], [0, 66, 60, 80], [1, 66, 71, 80], [0, 6, 71, 80], [0, 66, 71, 1 << 30]):
        S, src, dst = p.slots()
        keep = S.clone()
        p.out.fill_(-7.0)
        err.zero_()
        ws = torch.empty(K.kda_gdr_workspace_bytes(p.cfg, p.cu), dtype=torch.uint8, device="cuda")
        K.kda_gdr_prefill(p.cfg, p.params, S, src, dst, torch.tensor(wrong, dtype=torch.int32, device="cuda"), p.cu, *p.rows(), ws, err=err)
        torch.cuda.synchronize()
        if wrong != [0, 6, 71, 80]:  # this one has as many chunks and tokens: another valid split of the same rows
            assert err.item() == K.KDA_ERR_DEVICE, wrong
            assert bool((p.out == -7.0).all()) and torch.equal(S, keep)
    p = Problem([1, 1], 2, 2, True, seed=14)
    S, src, dst = p.slots()
    dst[0] = 50
    err.zero_()
    p.decode(S, src, dst, 1, err=err)
    assert err.item() == K.KDA_ERR_DEVICE and bool((p.out[0] == -7.0).all())
    near_state(S[3], p.ref(1)[1], False)


def test_fp32_sequences_refuse_a_cu_seqlens_that_is_wrong_anywhere():
    p = Problem([6] * 40, 2, 2, False, seed=16)  # more sequences than a warp has lanes
    ws = torch.empty(K.kda_gdr_workspace_bytes(p.cfg, p.cu), dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for at, value in ((0, 1), (40, 239), (7, 30), (36, 217), (39, 1 << 30), (20, -1)):
        wrong = p.cu.copy()
        wrong[at] = value
        S, src, dst = p.slots()
        keep = S.clone()
        p.out.fill_(-7.0)
        err.zero_()
        K.kda_gdr_prefill(p.cfg, p.params, S, src, dst, torch.from_numpy(wrong).cuda(), p.cu, *p.rows(), ws, err=err)
        torch.cuda.synchronize()
        if (at, value) == (36, 217):  # .. 210, 217, 222 ..: it rises from 0 to 240, another split of the same tokens
            assert err.item() == 0
            p.cu, p.lens = wrong, [int(n) for n in np.diff(wrong)]
            check(p, S, src, dst, p.S0, False)
            p.cu, p.lens = np.arange(0, 241, 6, dtype=np.int32), [6] * 40
            continue
        assert err.item() == K.KDA_ERR_DEVICE, (at, value)
        assert bool((p.out == -7.0).all()) and torch.equal(S, keep), (at, value)


def test_a_call_whose_rows_are_all_skipped_keeps_its_place_in_the_stream():
    """The workspace is taken for something else right behind a call that has nothing to do but its first
    kernel's part: what is written there later stays."""
    p = Problem([4096], 16, 4, True, seed=18)
    S, src, dst = p.slots()
    keep = S.clone()
    dst[0] = -1
    cu = torch.from_numpy(p.cu).cuda()
    ws = torch.empty(K.kda_gdr_workspace_bytes(p.cfg, p.cu), dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for i in range(20):
        K.kda_gdr_prefill(p.cfg, p.params, S, src, dst, cu, p.cu, *p.rows(), ws, err=err)
        ws.fill_(i)
        assert bool((ws == i).all()), i
    assert err.item() == K.KDA_ERR_DEVICE and torch.equal(S, keep) and bool((p.out == -7.0).all())


def test_repeats_bit_for_bit_on_a_side_stream_and_in_a_graph():
    p = Problem([130, 64, 1], 4, 2, True, seed=15)
    S, src, dst = p.slots()
    p.prefill(S, src, dst)
    S1, o1 = S.clone(), p.out.clone()
    ws = torch.empty(K.kda_gdr_workspace_bytes(p.cfg, p.cu), dtype=torch.uint8, device="cuda")
    cu = torch.from_numpy(p.cu).cuda()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    S[3:6] = 0
    p.out.fill_(-7.0)
    torch.cuda.synchronize()
    K.kda_gdr_prefill(p.cfg, p.params, S, src, dst, cu, p.cu, *p.rows(), ws, stream=st)
    st.synchronize()
    assert torch.equal(S, S1) and torch.equal(p.out, o1)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        K.kda_gdr_prefill(p.cfg, p.params, S, src, dst, cu, p.cu, *p.rows(), ws)
        K.kda_gdr_decode(p.cfg, p.params, S, dst, dst, 1, *(x[:3] for x in p.rows()[:5]), p.out[p.T:p.T + 3])
    for seed in (15, 16):  # replayed on other data in the same tensors
        p2 = Problem([130, 64, 1], 4, 2, True, seed=seed)
        for n in "qkvab":
            p.dev[n].copy_(p2.dev[n])
        p.h = p2.h
        S[:3] = torch.from_numpy(p2.S0).cuda()
        p.S0 = p2.S0
        p.out.fill_(-7.0)
        K_A = torch.from_numpy(p2.A_log).cuda()
        p.params._keep[0].copy_(K_A)
        p.params._keep[1].copy_(torch.from_numpy(p2.dt_bias).cuda())
        p.A_log, p.dt_bias = p2.A_log, p2.dt_bias
        g.replay()
        torch.cuda.synchronize()
        for s in range(3):
            o, Sr, mag = p.ref(s)
            near(p.out[p.cu[s]:p.cu[s + 1]], o, mag, True, True)
            first = lambda x, m: p.h[x][s:s + 1].reshape(1, m, -1)
            o, Sr, mag, _ = gdr(first("q", 2), first("k", 2), first("v", 4), p.h["a"][s:s + 1], p.h["b"][s:s + 1], p.A_log, p.dt_bias, Sr)
            near(p.out[p.T + s:p.T + s + 1], o.reshape(1, -1), mag.reshape(1, -1), True, True)
            near_state(S[3 + s], Sr, True)


def test_slots_past_32_bits():
    """A state whose offset in bytes and in elements passes 2^32."""
    H = 64
    slots = 2 ** 32 // (H * D * D) + 2
    S = torch.empty(slots, H, D, D, device="cuda")
    p = Problem([65], H, 32, True, seed=17)
    S[slots - 2] = torch.from_numpy(p.S0[0]).cuda()
    i = lambda x: torch.tensor([x], dtype=torch.int32, device="cuda")
    p.prefill(S, i(slots - 2), i(slots - 1))
    near_state(S[slots - 1], p.ref(0)[1], True)
    q = Problem([1], H, 32, True, seed=18)
    S[slots - 2] = torch.from_numpy(q.S0[0]).cuda()
    q.decode(S, i(slots - 2), i(slots - 1), 1)
    near_state(S[slots - 1], q.ref(0)[1], False)


def test_no_rows():
    p = Problem([0, 0], 2, 1, True, seed=19)
    S, src, dst = p.slots()
    p.prefill(S, src, dst)
    assert torch.equal(S[2:4], S[:2])
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    rows = tuple(x[:0] for x in p.rows())
    K.kda_gdr_decode(p.cfg, p.params, S, none, none, 1, *rows)
    K.kda_gdr_prefill(p.cfg, p.params, S, none, none, torch.zeros(1, dtype=torch.int32, device="cuda"), [0], *rows,
                      torch.empty(256, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()


def test_parameters_made_by_hand_are_refused():
    p = Problem([1], 2, 1, True, seed=20)
    S, src, dst = p.slots()
    p.params = K.kda_gdr_params(p.params.A_log, p.params.dt_bias)  # no count and no device to check
    with pytest.raises(ValueError):
        p.decode(S, src, dst, 1)


def test_binding_refusals():
    p = Problem([4], 2, 1, True, seed=20)
    S, src, dst = p.slots()
    q, k, v, a, b, out = p.rows()
    call = lambda *rows, S=S, src=src, n=4: K.kda_gdr_decode(p.cfg, p.params, S, src, dst, n, *rows)
    for bad in ((q.float(), k, v, a, b, out), (q.cpu(), k, v, a, b, out)):
        with pytest.raises(TypeError):
            call(*bad)
    for bad in ((q[:3], k, v, a, b, out), (q, k, v[:, :128], a, b, out), (q, k, v, a.t().contiguous().t(), b, out)):
        with pytest.raises(ValueError):
            call(*bad)
    with pytest.raises(ValueError):
        call(q, k, v, a, b, out, S=S[:, :1])
    with pytest.raises(ValueError):
        call(q, k, v, a, b, out, src=torch.zeros(2, dtype=torch.int32, device="cuda"))
    for bad in ((v[:, 1:129], k, v, a, b, out),):  # not 16-byte aligned
        with pytest.raises(K.KdaError) as e:
            call(*bad)
        assert e.value.status == K.KDA_ERR_INVALID
    odd = torch.zeros(4, 131, dtype=torch.bfloat16, device="cuda")[:, :128]
    with pytest.raises(K.KdaError):
        call(odd, k, v, a, b, out)
    with pytest.raises(K.KdaError):
        K.kda_gdr_prefill(p.cfg, p.params, S, src, dst, torch.from_numpy(p.cu).cuda(), p.cu, q, k, v, a, b, out,
                          torch.empty(100, dtype=torch.uint8, device="cuda"))
