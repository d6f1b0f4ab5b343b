"""What is not finite in a row of the chunked gated delta rule reaches no earlier token, no other value column than the
recurrence takes it to, and no other sequence: the outputs and the state are finite where the FP64 recurrence's are,
within the tolerances of test_gpu_gdr.py, and nowhere else."""
import numpy as np
import pytest
import torch

import linear_attention_mixer_gb300 as K
from tests.test_gpu_gdr import D, Problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from linear_attention_mixer_gb300 import build
    build.build()
    torch.cuda.set_device(0)


def compare(got, ref, mag, share):
    """got is finite exactly where ref is, and there within 2^-8 |ref| + share mag."""
    got = got.float().cpu().numpy().astype(np.float64)
    fin = np.isfinite(ref)
    assert np.array_equal(np.isfinite(got), fin), (int((np.isfinite(got) != fin).sum()), int(fin.sum()))
    bad = fin & ~(np.abs(np.where(fin, got - ref, 0)) <= 2.0 ** -8 * np.abs(np.where(fin, ref, 0)) + share * np.where(fin, mag, 0) + 1e-30)
    assert not bad.any(), int(bad.sum())


def check(p, S, dst):
    with np.errstate(all="ignore"):
        for s in range(len(p.lens)):
            o, Sr, mag = p.ref(s)
            compare(p.out[p.cu[s]:p.cu[s + 1]], o, mag, 2.0 ** -7 * (1 + 2.0 ** -8))
            fin = np.isfinite(Sr)
            got = S[int(dst[s])].cpu().numpy().astype(np.float64)
            assert np.array_equal(np.isfinite(got), fin)
            e, n = np.linalg.norm(np.where(fin, got - Sr, 0)), np.linalg.norm(np.where(fin, Sr, 0))
            assert e <= 5 * 2.0 ** -16 * n + 1e-30, (e, n)
    assert bool((p.out[p.T:] == -7.0).all())


# tokens at the edges of 8- and 16-row tiles and of chunks, in the first chunk, later ones and the ragged last
@pytest.mark.parametrize("t", [0, 1, 8, 15, 16, 63, 64, 77, 134])
@pytest.mark.parametrize("name,value", [("v", np.nan), ("v", np.inf), ("k", np.nan), ("k", -np.inf), ("q", np.nan),
                                         ("a", np.nan), ("b", np.nan)])
@pytest.mark.parametrize("lens,H,Hk", [([135], 2, 1), ([135] + [130, 64, 7, 200] * 5, 8, 4)])  # 32 and 64 columns
def test_one_value(lens, H, Hk, name, value, t):
    def edit(h):
        h[name][t, 5 % h[name].shape[1]] = value
    p = Problem(lens[:3] if len(lens) > 1 and t not in (15, 77) else lens, H, Hk, True, seed=50, edit=edit)
    S, src, dst = p.slots()
    p.prefill(S, src, dst)
    check(p, S, dst)


@pytest.mark.parametrize("lens,H", [([135], 2), ([135] + [130, 64, 7, 200] * 5, 16)])
def test_several_values_in_place(lens, H):
    """Several bad tokens, in different heads, rows and sequences, and a state that is not finite itself; src == dst."""
    N = len(lens)
    cu = np.concatenate([[0], np.cumsum(lens)])
    def edit(h):
        h["v"][20, 3], h["v"][20, 200], h["v"][90, 130] = np.nan, np.inf, -np.inf
        h["a"][101, 1] = np.nan
        for s in range(1, N, 3):
            h["k"][(cu[s] + cu[s + 1]) // 2, 7] = np.nan
    p = Problem(lens, H, H // 2, True, seed=51, edit=edit)
    if N > 1:
        p.S0[2, 1, 4, 9] = np.inf
    S, src, _ = p.slots()
    keep = S.clone()
    p.prefill(S, src, src)
    check(p, S, np.arange(N))
    assert torch.equal(S[N:], keep[N:])


def test_a_state_that_is_not_finite_is_copied_for_an_empty_sequence():
    """.. and nothing is read for it: its row would be the one behind the last."""
    p = Problem([70, 0], 2, 1, True, seed=52)
    p.S0[1, 0, 3, 3] = np.nan
    S, src, dst = p.slots()
    p.prefill(S, src, dst)
    assert torch.equal(S[3].view(torch.int32), S[1].view(torch.int32))


def test_a_long_sequence_goes_on_after_it():
    """Hundreds of tokens behind the bad one, walked token by token in its 16 columns only."""
    def edit(h):
        h["v"][700, 40] = np.nan
    p = Problem([1000], 2, 2, True, seed=53, edit=edit)
    S, src, dst = p.slots()
    p.prefill(S, src, dst)
    check(p, S, dst)
