"""How exact the outputs of the chunked gated delta rule are, in a bound that the loss of any one low part of P or U
would break.

The chunked form takes Q S0 with S0 rounded to BF16 and P U with P and U in two BF16 parts each (high x high, low x
high, high x low). Half a step of BF16 is 2^-8, so an output is off by at most
    2^-8 |o|      its own rounding,
    2^-8 m0       S0's (m0: the terms of Q S0 in absolute value, see test_gpu_gdr_long.py),
    3 x 2^-16 mag what the two parts and the dropped low x low lose in P U, and
    5 x 2^-16     the losses between S0 and U (test_gpu_gdr.py), relative to terms that mag bounds but for the
                  cancellation in T's rows:
2^-13 mag in all, and 2^-12 with a factor of two for that cancellation. From a zero state a single chunk has m0 = 0.
Terms of mag mostly cancel in o, and 2^-8 of one of its high parts is 16 times the last bound."""
import numpy as np
import pytest
import torch

import linear_attention_mixer_gb300 as K
from tests.test_gpu_gdr import D, Problem
from tests.test_gpu_gdr_long import recurrence

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from linear_attention_mixer_gb300 import build
    build.build()
    torch.cuda.set_device(0)


def plain(h):
    pass


def slow(h):  # little decay
    h["a"] -= 4.0


def leaning(h):  # keys with a common part, little decay
    h["k"][:] += 0.5
    h["a"] -= 4.0


def aligned(h):  # all keys positive, nothing decays, everything is replaced
    h["a"][:], h["b"][:] = -30.0, 30.0
    h["k"][:] = np.abs(h["k"]) + 0.3


def strongly(h):  # nearly one key
    h["a"][:], h["b"][:] = -30.0, 30.0
    h["k"][:] = 1.0 + 0.1 * h["k"]


def excess(p, S0=None):
    """Largest |error| over the bound, and the error's norm over the output's."""
    S, src, dst = p.slots()
    p.prefill(S, src, dst)
    o, mag, m0, _ = recurrence(p, S0)
    e = np.abs(p.out[:p.T].float().cpu().numpy().astype(np.float64) - o)
    bound = 2.0 ** -8 * (np.abs(o) + m0) + 2.0 ** -12 * mag
    return float((e / (bound + 1e-30)).max()), float(np.linalg.norm(e) / np.linalg.norm(o))


@pytest.mark.parametrize("edit", [plain, slow, leaning, aligned, strongly])
@pytest.mark.parametrize("lens,H,Hk", [([64], 4, 2), ([33], 3, 3), ([64, 50, 17, 63] * 20, 16, 8)])  # 32 and 64 columns
def test_one_chunk_from_a_zero_state(lens, H, Hk, edit):
    p = Problem(lens, H, Hk, True, seed=60, edit=edit, states=np.zeros((len(lens), H, D, D), np.float32))
    x, norm = excess(p)
    print(edit.__name__, x, norm)
    assert x <= 1


@pytest.mark.parametrize("edit", [plain, slow, leaning, aligned, strongly])
@pytest.mark.parametrize("lens,H,Hk", [([700], 4, 2), ([300, 129, 640, 64] * 5, 16, 8)])
def test_several_chunks(lens, H, Hk, edit):
    p = Problem(lens, H, Hk, True, seed=61, edit=edit)
    x, norm = excess(p)
    print(edit.__name__, x, norm)
    assert x <= 1
