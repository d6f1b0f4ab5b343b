"""Waits that give up in the gated linear recurrence's scan, whose blocks wait for one another within a cluster: the kernel file is
built once more with limits that run out at once in chosen warps and lanes. The call has to end by itself, record
KDA_ERR_TIMEOUT, leave alone what it does not own, and leave the library usable."""
import pytest
import torch

from linear_attention_mixer_gb300 import kda as K
from tests.test_gpu_give_up import EVEN, EVERY, ODD, compiled
from tests.test_gpu_glr import Problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from linear_attention_mixer_gb300 import build
    build.build()
    torch.cuda.set_device(0)


@pytest.fixture(scope="module")
def glr_lib(tmp_path_factory):
    return compiled(tmp_path_factory.mktemp("glr"), "glr_give_up", "kda_glr_scan.cu", "KDA_GLR_WAIT_LIMIT", ["kda_glr.cu"])


@pytest.mark.parametrize("lens,D,bf16,gate", [([3000], 72, True, True), ([1500, 40, 700], 200, False, False), ([9000], 64, True, False)])
def test_prefill_and_backward(glr_lib, monkeypatch, lens, D, bf16, gate):
    def problem():
        p = Problem(lens, D, bf16, gate, seed=30)
        p.dst = p.src + p.N
        return p

    good = problem()
    good.prefill()
    with monkeypatch.context() as m:
        m.setattr(K, "lib", lambda: glr_lib)
        for warps, lanes in [(0, 0), (1, EVERY), (2, ODD), (8, EVEN), (0xF, 1 << 31), (0xFF, EVERY), (0xFF, ODD)]:
            assert glr_lib.wl_set(warps, lanes) == 0
            p = problem()
            p.prefill()
            assert p.err.item() == (K.KDA_ERR_TIMEOUT if warps else K.KDA_OK), (hex(warps), hex(lanes))
            assert bool((p.out[p.T:] == -7.0).all()) and torch.equal(p.S[:p.N], p.dev["h0"]) and bool((p.S[2 * p.N:] == 3.0).all())
            if not warps:
                assert torch.equal(p.out, good.out) and torch.equal(p.S, good.S)
            p.starts.copy_(good.starts)
            p.err.zero_()
            g = p.backward()
            assert p.err.item() == (K.KDA_ERR_TIMEOUT if warps else K.KDA_OK), (hex(warps), hex(lanes))
            for n in ("dx", "da", "db"):
                assert bool((g[n][p.T:] == -7.0).all())
    p = problem()
    p.prefill()
    p.check()
    p.check_grads(p.backward())
