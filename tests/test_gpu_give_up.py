"""Waits that give up, in kernels whose warps wait for one another. The kernel files are built once more with
limits that run out at once in chosen warps and lanes (tests/cuda/wait_limits.cuh): the call has to end by
itself, record KDA_ERR_TIMEOUT, leave alone what it does not own, and leave the library usable.

Lanes apart matter: a limit may run out in one lane of a warp and not in the next."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

from linear_attention_mixer_gb300 import kda as K
from oracle import fp8 as O8
from tests import test_gpu_fp8 as F8
from tests.test_gpu_gdr import Problem, check

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "linear_attention_mixer_gb300", "csrc")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from linear_attention_mixer_gb300 import build
    build.build()
    torch.cuda.set_device(0)


def compiled(tmp, name, source, macro, others=()):
    """A library of `source` with its wait limit replaced, and the other sources as they are; what else it calls
    comes from libkda.so, which is loaded first so that its own calls stay in it."""
    K.lib()
    nvcc = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    flags = ["-gencode", "arch=compute_103a,code=sm_103a", "-O3", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr"]
    jobs, objs = [], []
    for s in (source, *others):
        objs.append(str(tmp / (s + ".o")))
        edit = ["-include", os.path.join(HERE, "cuda", "wait_limits.cuh"), f"-D{macro}=(wl_limit())"] if s == source else []
        jobs.append(subprocess.Popen([nvcc, *flags, *edit, "-c", os.path.join(CSRC, s), "-o", objs[-1]]))
    assert all(j.wait() == 0 for j in jobs)
    out = tmp / f"lib{name}.so"
    subprocess.run([nvcc, "-shared", *objs, K.LIB_PATH, "-Xlinker", "-Bsymbolic", "-Xlinker", "-rpath=" + os.path.dirname(K.LIB_PATH), "-o", str(out)],
                   check=True)
    L = ctypes.CDLL(str(out))
    for fn, res, args in K.SIGNATURES:
        f = getattr(L, fn)  # its own, or libkda's behind it
        f.restype, f.argtypes = res, args
    L.wl_set.argtypes = [ctypes.c_uint32, ctypes.c_uint32]
    return L


@pytest.fixture(scope="module")
def gdr_lib(tmp_path_factory):
    return compiled(tmp_path_factory.mktemp("gdr"), "gdr_give_up", "kda_gdr_prefill.cu", "KDA_GDR_WAIT_LIMIT", ["kda_gdr.cu"])


EVERY, ODD, EVEN = 0xFFFFFFFF, 0xAAAAAAAA, 0x55555555
# warps 0-3 carry the state, 4-7 form the output, lane 0 of warp 8 copies
GDR = [(1 << 0, EVERY), (1 << 0, ODD), (1 << 3, EVEN), (0xF, 1 << 31), (1 << 4, EVERY), (1 << 5, ODD), (0xF0, EVEN),
       (1 << 8, EVERY), (0x1FF, EVERY), (0xFF, ODD)]


@pytest.mark.parametrize("lens,H", [([650], 2), ([330] * 8, 32)])  # 32 and 64 value columns a block
def test_prefill(gdr_lib, monkeypatch, lens, H):
    p = Problem(lens, H, H // 2, True, seed=30)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    N = len(lens)
    with monkeypatch.context() as m:
        m.setattr(K, "lib", lambda: gdr_lib)
        for warps, lanes in [(0, 0)] + GDR:
            assert gdr_lib.wl_set(warps, lanes) == 0
            S, src, dst = p.slots()
            keep = S.clone()
            p.out.fill_(-7.0)
            err.zero_()
            p.prefill(S, src, dst, err=err)
            assert err.item() == (K.KDA_ERR_TIMEOUT if warps else K.KDA_OK), (hex(warps), hex(lanes))
            assert torch.equal(S[:N], keep[:N]) and torch.equal(S[2 * N:], keep[2 * N:])
            assert bool((p.out[p.T:] == -7.0).all())
            if not warps:
                check(p, S, src, dst, p.S0, True)
            if warps == 0x1FF:  # no warp saw its rows
                assert torch.equal(S, keep) and bool((p.out == -7.0).all())
    S, src, dst = p.slots()
    err.zero_()
    p.prefill(S, src, dst, err=err)
    assert err.item() == K.KDA_OK
    check(p, S, src, dst, p.S0, True)


@pytest.fixture(scope="module")
def fp8_lib(tmp_path_factory):
    return compiled(tmp_path_factory.mktemp("fp8"), "fp8_give_up", "kda_fp8.cu", "KDA_F8_WAIT_LIMIT")


def modes(epi):
    """Epilogue warps 0 .. epi - 1, then lane 0 of the copying warp and of the one that issues the products."""
    return [(1, EVERY), (1, ODD), (1 << (epi - 1), EVEN), ((1 << epi) - 1, 1 << 31), (1 << epi, EVERY), (2 << epi, EVERY),
            ((4 << epi) - 1, EVERY), ((1 << epi) - 1, ODD)]


# one k range and several, 128 and 256 columns a tile
@pytest.mark.parametrize("M,N,Kd", [(130, 264, 2064), (16, 1024, 4096), (1200, 4104, 1040)])
def test_fp8_product(fp8_lib, monkeypatch, M, N, Kd):
    ops = F8.operands(M, N, Kd, 4)
    args = [F8.dev8(ops[0]), torch.from_numpy(ops[1]).cuda(), F8.dev8(ops[2]), torch.from_numpy(ops[3]).cuda()]
    y = torch.empty(M * N + 64, dtype=torch.bfloat16, device="cuda")
    work = torch.zeros(K.kda_linear_fp8_workspace_bytes(M, N, Kd), dtype=torch.uint8, device="cuda")

    def call():
        y.fill_(-7.0)
        work.zero_()
        K.kda_linear_fp8(*args, y[:M * N], work)
        torch.cuda.synchronize()
        assert bool((y[M * N:] == -7.0).all())
        return int(work[:4].view(torch.int32).item())

    assert call() == K.KDA_OK
    want = y.clone()
    F8.near(want[:M * N].float().cpu().numpy().astype(np.float64).reshape(M, N), *O8.linear(*ops))
    with monkeypatch.context() as m:
        m.setattr(K, "lib", lambda: fp8_lib)
        for epi in (4, 8):  # whichever the tile's width is: other numbers of warps are covered by the masks too
            for warps, lanes in [(0, 0)] + modes(epi):
                assert fp8_lib.wl_set(warps, lanes) == 0
                got = call()
                if warps == 0:
                    assert got == K.KDA_OK and torch.equal(y, want)
                elif warps & 1:  # the first epilogue warp always waits for a product
                    assert got == K.KDA_ERR_TIMEOUT, (hex(warps), hex(lanes))
    assert call() == K.KDA_OK and torch.equal(y, want)


@pytest.fixture(scope="module")
def linear_lib(tmp_path_factory):
    return compiled(tmp_path_factory.mktemp("lin"), "linear_give_up", "kda_linear.cu", "KDA_LN_WAIT_LIMIT")


@pytest.mark.parametrize("M,N,Kd", [(300, 384, 1024), (16, 256, 8192)])
def test_product(linear_lib, monkeypatch, M, N, Kd):
    gen = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn(M, Kd, generator=gen, device="cuda").to(torch.bfloat16)
    w = (torch.randn(N, Kd, generator=gen, device="cuda") * Kd ** -0.5).to(torch.bfloat16)
    y = torch.empty(M * N + 64, dtype=torch.bfloat16, device="cuda")
    work = torch.zeros(K.kda_linear_workspace_bytes(M, N, Kd), dtype=torch.uint8, device="cuda")

    def call():
        y.fill_(-7.0)
        work.zero_()
        K.kda_linear(x, w, y[:M * N].view(M, N), work)
        torch.cuda.synchronize()
        assert bool((y[M * N:] == -7.0).all())
        return int(work[:4].view(torch.int32).item())

    assert call() == K.KDA_OK
    want = y.clone()
    with monkeypatch.context() as m:
        m.setattr(K, "lib", lambda: linear_lib)
        for warps, lanes in [(0, 0)] + modes(4):
            assert linear_lib.wl_set(warps, lanes) == 0
            got = call()
            assert (got == K.KDA_OK and torch.equal(y, want)) if warps == 0 else got == K.KDA_ERR_TIMEOUT or not warps & 1
    assert call() == K.KDA_OK and torch.equal(y, want)
