"""The gated linear recurrence over states that are kept long, and over states that fall far within a window.

One decay for each channel at all tokens (a = 0, b = 0), so that what a decay is off by adds up. Bound, relative and in the 2-norm
over the channels: e = alpha - 1 and m are off by 2^-20 or less each (an exponential and a product of gk, a polynomial and a root, a few
2^-24 each), which a state, a sum of alpha^k m x, has at most twice: 2^-18. Each step rounds the state and its increment by 2^-24
or less of it, n steps with signs that follow the inputs (an increment is many steps of FP32 here) by 2^-24 sqrt(2 n), four times that
to be certain. A scan takes a state over 64 tokens or more at once (and starts from 0 within them), so n = T / 64 there: 1.5e-5 for 65536
tokens; n = T token by token: 9e-5. A loop with alpha itself in FP32 has the same sign at each token and misses both, which is asserted.
"""
import numpy as np
import pytest
import torch

import linear_attention_mixer_gb300 as K
from tests.test_gpu_glr import Problem, np64

pytestmark = pytest.mark.gpu
T = 65536
SCAN, TOKENS = (2.0 ** -18 + 4 * 2.0 ** -24 * np.sqrt(2 * n) for n in (T // 64, T))


@pytest.fixture(scope="module", autouse=True)
def _built():
    from linear_attention_mixer_gb300 import build
    build.build()
    torch.cuda.set_device(0)


def long_memory(rate, D, rest=0):
    """T tokens with 1 - alpha from rate to 2 rate over the channels, and `rest` empty sequences behind them."""
    def edit(h):
        h["a"][:] = h["b"][:] = 0.0
        h["a_bias"][:] = h["b_bias"][:] = 0.0
        h["A_log"][:] = np.log(2 * rate * np.linspace(1, 2, D))
    return Problem([T] + [0] * rest, D, False, False, seed=40, edit=edit)


def loop(p, rows, start, dtype):
    """The state behind the T tokens of rows (m beta x, or dout) from start, by alpha as `dtype` has it."""
    gk = -np.exp(p.h["A_log"].astype(np.float64)) * 0.5
    e, al = np.expm1(gk), np.exp(gk).astype(dtype)
    m = np.sqrt(-e * (2.0 + e)) * 0.5
    u = (rows * m).astype(dtype)
    h = start.astype(dtype)
    for t in range(T):
        h = al * h + u[t]
    return h.astype(np.float64)


def loop_back(p, dtype):
    al = np.exp(-np.exp(p.h["A_log"].astype(np.float64)) * 0.5).astype(dtype)
    c, d = p.h["dS"][0].astype(dtype), p.h["dout"].astype(dtype)
    for t in range(T - 1, -1, -1):
        c = al * (d[t] + c)
    return c.astype(np.float64)


def off(got, ref):
    return np.linalg.norm(got - ref) / np.linalg.norm(ref)


@pytest.mark.parametrize("rest", [0, 152])
@pytest.mark.parametrize("rate", [1e-5, 1e-6, 1e-7])
def test_states_that_are_kept_long(rate, rest):
    """The sequence in parts, and (with other sequences beside it) in one part, by clusters."""
    p = long_memory(rate, 64, rest)
    x, h0 = p.h["x"][:T].astype(np.float64), p.h["h0"][0].astype(np.float64)
    S, dS = loop(p, x, h0, np.float64), loop_back(p, np.float64)
    assert off(loop(p, x, h0, np.float32), S) > TOKENS and off(loop_back(p, np.float32), dS) > TOKENS
    p.prefill()
    g = p.backward()
    assert int(p.err.item()) == 0
    got = np64(p.S[int(p.dst[0])])
    assert off(got, S) <= SCAN, off(got, S)
    assert off(np64(g["dS"][0]), dS) <= SCAN, off(np64(g["dS"][0]), dS)
    if rest == 0:  # the same tokens, eight at a time
        state = p.dev["h0"][:1].clone()
        slot, out = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.empty(8, 64, device="cuda")
        for t in range(0, T, 8):
            K.kda_glr_decode(p.cfg, p.params, state, slot, slot, 8, *(None if r is None else r[t:t + 8] for r in p.rows()), out)
        torch.cuda.synchronize()
        assert off(np64(state[0]), S) <= TOKENS and off(got, np64(state[0])) <= SCAN + TOKENS


@pytest.mark.parametrize("lens", [[130, 40], [1100], [9000]])
@pytest.mark.parametrize("level", [1.0, 6e4])
def test_states_that_fall_far(lens, level):
    """Nothing comes in: what is left of a state is right relative to itself, however little; and so for the gradient."""
    def edit(h):
        h["x"][:] = 0.0
        h["x"][::509] = 1.0
        h["a"] *= 0.1
        h["h0"] *= level
        h["dS"] *= level
        h["dout"][:] = 0.0
        D = h["A_log"].shape[0]
        h["A_log"][:] = np.log(2 * np.geomspace(1e-4, 12.0, D))
        h["a_bias"][:] = 0.0
    p = Problem(lens, 64, False, False, seed=41, edit=edit)
    p.prefill()
    p.check()
    p.check_grads(p.backward())
