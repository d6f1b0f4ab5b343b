"""The chunked gated delta rule in its steady state: sequences of many chunks (every stage of the rings and every
hand-over buffer is used many times over, with both parities of its barriers) and batches of more items than the
first kernel has blocks, in both forms of the second kernel, against the FP64 token recurrence.

The recurrence runs here for all sequences at once, on the GPU in torch's FP64; it is checked against
oracle/gdr.py. The tolerances are those of test_gpu_gdr.py."""
import numpy as np
import pytest
import torch

import linear_attention_mixer_gb300 as K
from tests.test_gpu_gdr import D, Problem, near, near_state

pytestmark = pytest.mark.gpu
C = 64


@pytest.fixture(scope="module", autouse=True)
def _built():
    from linear_attention_mixer_gb300 import build
    build.build()
    torch.cuda.set_device(0)


def recurrence(p, S0=None):
    """Of every sequence of p: o [T, H d], S [N, H, d, d], mag as oracle/gdr.py, and m0, the part of mag that comes
    from the state at the start of the token's chunk: |q^| . (decays since then) |S at its start|."""
    H, Hk, N = p.H, p.Hk, len(p.lens)
    f64 = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda().double()
    q, k, v = (f64(p.h[n]).view(p.T, -1, D) for n in "qkv")
    if p.l2norm:
        q = q / (q.square().sum(-1, keepdim=True) + 1e-6).sqrt()
        k = k / (k.square().sum(-1, keepdim=True) + 1e-6).sqrt()
    q = (q * D ** -0.5).repeat_interleave(H // Hk, 1)
    k = k.repeat_interleave(H // Hk, 1)
    x = f64(p.h["a"]) + f64(p.dt_bias)
    alpha = torch.exp(-torch.exp(f64(p.A_log)) * (x.clamp(min=0) + torch.log1p(torch.exp(-x.abs()))))
    beta = torch.sigmoid(f64(p.h["b"]))
    order = sorted(range(N), key=lambda s: -p.lens[s])  # those that are still going come first
    first = torch.from_numpy(p.cu[:N].astype(np.int64)).cuda()[order]
    S = f64(p.S0 if S0 is None else S0)[order]
    M = S.abs()
    M0 = M.clone()
    o, mag, m0 = (torch.zeros(p.T, H, D, dtype=torch.float64, device="cuda") for _ in range(3))
    for t in range(max(p.lens)):
        n = sum(x > t for x in p.lens)
        r = first[:n] + t
        al, kt, qt = alpha[r][..., None, None], k[r][..., None], q[r][..., None, :]
        if t % C == 0:
            M0[:n] = S[:n].abs()
        Z = S[:n] * al
        u = beta[r][..., None, None] * (v[r][..., None, :] - kt.transpose(-1, -2) @ Z)
        S[:n] = Z + kt * u
        M[:n] = M[:n] * al + kt.abs() * u.abs()
        M0[:n] *= al
        o[r] = (qt @ S[:n])[..., 0, :]
        mag[r] = (qt.abs() @ M[:n])[..., 0, :]
        m0[r] = (qt.abs() @ M0[:n])[..., 0, :]
    back = torch.empty_like(S)
    back[order] = S
    return tuple(x.view(p.T, -1).cpu().numpy() for x in (o, mag, m0)) + (back.cpu().numpy(),)


def check(p, S, dst):
    o, mag, _, Sr = recurrence(p)
    for s in range(len(p.lens)):
        r = slice(p.cu[s], p.cu[s + 1])
        near(p.out[r], o[r], mag[r], True, True)
        near_state(S[int(dst[s])], Sr[s], True)
    assert bool((p.out[p.T:] == -7.0).all())


def run(p):
    S, src, dst = p.slots()
    keep = S.clone()
    p.prefill(S, src, dst)
    N = len(p.lens)
    assert torch.equal(S[:N], keep[:N]) and torch.equal(S[2 * N:], keep[2 * N:])
    return S, dst


def test_the_recurrence():
    p = Problem([70, 0, 5, 130], 4, 2, True, seed=40)
    o, mag, m0, S = recurrence(p)
    for s in range(4):
        r = slice(p.cu[s], p.cu[s + 1])
        orr, Sr, magr = p.ref(s)
        for got, ref in ((o[r], orr), (mag[r], magr), (S[s], Sr)):
            assert np.allclose(got, ref, rtol=1e-11, atol=1e-13)
        assert (m0[r] >= 0).all() and (m0[r][:1] <= mag[r][:1] * (1 + 1e-12)).all()



# one sequence is fewer blocks than SMs at 32 columns; the batches are several waves of blocks at either width
LONG = [([20 * C + 37], 2, 1), ([17 * C], 10, 2), ([31 * C + 1], 3, 3), ([9 * C + 5, 12 * C, 1, 10 * C + 63, 0, 700] * 4, 16, 8),
        ([600, 333, 1025] * 12, 18, 2), ([64 * C], 32, 16)]


@pytest.mark.parametrize("lens,H,Hk", LONG)
def test_many_chunks(lens, H, Hk):
    p = Problem(lens, H, Hk, True, seed=41)
    S, dst = run(p)
    check(p, S, dst)


@pytest.mark.parametrize("H,Hk", [(6, 3), (18, 2)])  # more than four value heads a key head in the second
def test_more_items_than_blocks(H, Hk):
    """The first kernel's blocks (three an SM) take three items or more each."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    chunks = -(-(2 * 3 * sms + 50) // Hk)
    rng = np.random.default_rng(5)
    lens = []
    while sum(-(-n // C) for n in lens) < chunks:
        lens.append(int(rng.integers(1, 9 * C)))
    p = Problem(lens, H, Hk, True, seed=42)
    S, dst = run(p)
    check(p, S, dst)


def test_a_prompt_of_8192_tokens():
    p = Problem([8192], 4, 2, True, seed=43)
    S, dst = run(p)
    check(p, S, dst)
