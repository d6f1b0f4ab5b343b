"""What is not finite in one row of the gated linear recurrence: forward it reaches its own channel of its own sequence from its token
on, and in the gradients what the formulas make of it - everything else is the same to the bit as without it. Sequences in parts, by
clusters, by single blocks and by a thread each."""
import numpy as np
import pytest
import torch

from tests.test_gpu_glr import Problem

pytestmark = pytest.mark.gpu
CHANNEL = 5


@pytest.fixture(scope="module", autouse=True)
def _built():
    from linear_attention_mixer_gb300 import build
    build.build()
    torch.cuda.set_device(0)


# lengths; the sequence that has it, and its token there
LONG = [([9000, 300], 0, 4700), ([300, 9000, 70], 1, 8999), ([5000] + [0] * 152 + [600], 0, 2500), ([700, 40], 0, 100), ([700, 40], 1, 39)]
SHORT = [([16] * 40, 7, 9), ([2] * 300, 9, 0)]


def clean_and_not(lens, D, bf16, gate, row, name, value):
    """The same problem without and with the value in one row, after a prefill and a backward."""
    got = []
    for bad in (False, True):
        p = Problem(lens, D, bf16, gate, seed=50)
        p.dst = p.src + p.N
        if bad:
            p.dev[name][row, CHANNEL] = value
        p.prefill()
        got.append((p, p.backward()))
    return got


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("name", ["x", "a", "b", "g", "dout"])
@pytest.mark.parametrize("lens,s,t", LONG + SHORT)
def test_one_row(lens, s, t, name, value):
    D, bf16 = 72, name != "x"
    cu = np.concatenate([[0], np.cumsum(lens)])
    row = int(cu[s] + t)
    (p, g), (q, h) = clean_and_not(lens, D, bf16, True, row, name, value)
    assert int(q.err.item()) == 0
    rows = torch.arange(int(cu[-1]), device="cuda")
    inside = (rows >= int(cu[s])) & (rows < int(cu[s + 1]))
    behind, before, here = inside & (rows > row), inside & (rows < row), rows == row
    none = torch.zeros_like(here)
    # where a value may be another: the states behind it, and what they enter; the gradients before it, through lam
    kept = {"out": behind | here, "dx": before | here, "da": inside, "db": before | here, "dg": behind | here}
    if name == "x":  # lam does not know x
        kept |= {"dx": none, "da": behind | here, "db": here}
    if name == "b":  # nor b, whose dx and db are this token's
        kept |= {"dx": here, "da": behind | here, "db": here}
    if name == "g":
        kept["out"] = here
        kept["da"] = before | here
        kept["dg"] = here
    if name == "dout":
        kept["out"] = none
        kept["da"] = before | here
        kept["dg"] = here
    for n, where in kept.items():
        a, b = (p.out[:p.T], q.out[:q.T]) if n == "out" else (g[n][:p.T], h[n][:p.T])
        same = torch.ones(p.T, D, dtype=torch.bool, device="cuda")
        same[:, CHANNEL] = ~where
        assert torch.equal(a[same], b[same]), n
        assert bool((q.out[q.T:] == -7.0).all())
    other = torch.ones(p.N, D, dtype=torch.bool, device="cuda")
    other[s, CHANNEL] = False
    assert torch.equal(p.S[p.N:2 * p.N][other], q.S[p.N:2 * p.N][other]) and torch.equal(g["dS"][other], h["dS"][other])
    columns = torch.arange(D, device="cuda") != CHANNEL
    for n in ("dA_log", "da_bias", "db_bias"):
        assert torch.equal(g[n][columns], h[n][columns]), n
    # and it does get there
    if np.isnan(value):
        if name in "xab":
            assert bool(q.out[:q.T][behind | here, CHANNEL].isnan().all()) and bool(q.S[q.N + s, CHANNEL].isnan())
        if name in ("a", "g", "dout"):
            assert bool(h["dx"][:q.T][before | here, CHANNEL].isnan().all()) and bool(h["dS"][s, CHANNEL].isnan())
        assert bool(h["db"][row, CHANNEL].isnan()) and bool(h["dA_log"][CHANNEL].isnan())
