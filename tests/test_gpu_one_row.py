"""One token, or one row, through the C entry points of the gated linear recurrence and the block norms: the distance to a next one is
not used, whatever it is."""
import ctypes

import pytest
import torch

import linear_attention_mixer_gb300 as K
from tests import test_gpu_block_norm as BN
from tests import test_gpu_glr as G

pytestmark = pytest.mark.gpu
STRIDES = [0, 3, -7, -2 ** 62, 2 ** 62]
b = ctypes.byref


@pytest.fixture(scope="module", autouse=True)
def _built():
    from linear_attention_mixer_gb300 import build
    build.build()
    torch.cuda.set_device(0)


def at(t):
    return None if t is None else t.data_ptr()


@pytest.mark.parametrize("stride", STRIDES)
@pytest.mark.parametrize("lens,D,bf16,gate", [([1], 72, True, True), ([0, 1, 0], 68, False, False)])
def test_one_token(lens, D, bf16, gate, stride):
    L, p = K.lib(), G.Problem(lens, D, bf16, gate, seed=60)
    r = K.kda_glr_rows(*(at(t) for t in (*p.rows(), p.out)), *[stride] * 5)
    cu = p.cu.ctypes.data_as(ctypes.c_void_p)
    call = (b(p.cfg), b(p.params), p.S.data_ptr(), p.S.shape[0])
    assert L.kda_glr_prefill(*call, p.src.data_ptr(), p.dst.data_ptr(), p.cu_dev.data_ptr(), cu, p.N, b(r), p.starts.data_ptr(), p.work.data_ptr(), p.work.nbytes,
                             p.err.data_ptr(), None) == K.KDA_OK, K.kda_last_error()
    torch.cuda.synchronize()
    p.check()
    g = p.make_grads()
    back = K.kda_glr_grad_rows(*(at(t) for t in (*p.rows(), p.dev["dout"], g["dx"], g["da"], g["db"], g.get("dg"))), *[stride] * 9)
    assert L.kda_glr_backward(b(p.cfg), b(p.params), p.cu_dev.data_ptr(), cu, p.N, p.starts.data_ptr(), b(back), p.dev["dS"].data_ptr(), g["dS"].data_ptr(),
                              *(g[n].data_ptr() for n in ("dA_log", "da_bias", "db_bias")), p.work.data_ptr(), p.work.nbytes, p.err.data_ptr(), None) == K.KDA_OK
    torch.cuda.synchronize()
    p.check_grads(g)
    s = lens.index(1)
    p.S[:p.N] = p.dev["h0"]
    p.out.fill_(-7.0)
    assert L.kda_glr_decode(*call, p.src[s:].data_ptr(), p.dst[s:].data_ptr(), 1, 1, b(r), p.err.data_ptr(), None) == K.KDA_OK
    torch.cuda.synchronize()
    p.check()


@pytest.mark.parametrize("stride", STRIDES)
@pytest.mark.parametrize("D,bf16,gate", [(136, True, True), (1004, False, False), (8200, True, False)])
def test_one_row(D, bf16, gate, stride):
    L, p = K.lib(), BN.Problem(1, D, bf16, gate, seed=61)
    d, x1, h = p.dev, p.new(), p.new()
    r = K.kda_block_norm_rows(*(at(t) for t in (d["x"], d["y"], d["g"], x1, h, None)), *[stride] * 5)
    assert L.kda_block_norm(b(p.cfg), b(p.params), 1, b(r), None) == K.KDA_OK, K.kda_last_error()
    torch.cuda.synchronize()
    want = p.forward()
    assert torch.equal(x1, want[0]) and torch.equal(h, want[1])
    g = {n: p.new() for n in ("dx", "dy") + (("dg",) if gate else ())}
    s = {n: torch.full((D,), float("nan"), device="cuda") for n in ("dpost_w", "dscale", "dpre_w")}
    work = torch.empty(K.kda_block_norm_workspace_bytes(p.cfg, 1), dtype=torch.uint8, device="cuda")
    back = K.kda_block_norm_grad_rows(*(at(t) for t in (d["x"], d["dh"], d["dx1"], d["y"], d["g"], g["dx"], g["dy"], g.get("dg"))), *[stride] * 8)
    assert L.kda_block_norm_backward(b(p.cfg), b(p.params), 1, b(back), *(s[n].data_ptr() for n in s), work.data_ptr(), work.nbytes, None) == K.KDA_OK
    torch.cuda.synchronize()
    want = p.backward()
    assert all(torch.equal(t, want[n]) for n, t in (g | s).items())
