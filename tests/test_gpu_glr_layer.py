"""The gated linear recurrence layer (layer.GlrLayerRunner): a stack of two, prompts and then tokens, each step against FP64
from what the step before it wrote.

Products: FP32 sums of 64-wide blocks and the rounding to BF16, 2^-8 of the value and 2^-12 of the sums of absolute terms
(FP8 operands are exact in what they stand for). The recurrence and the norms as in their own tests.
"""
import numpy as np
import pytest
import torch

import linear_attention_mixer_gb300 as K
from linear_attention_mixer_gb300 import layer as L
from oracle import block_norm, fp8 as F8
from oracle.glr import glr

pytestmark = pytest.mark.gpu
HIDDEN, D = 256, 192


@pytest.fixture(scope="module", autouse=True)
def _built():
    from linear_attention_mixer_gb300 import build
    build.build()
    torch.cuda.set_device(0)


def np64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def near(got, ref, err, half=2.0 ** -8):
    bound = err + half * (np.abs(ref) + err) + 2.0 ** -133
    bad = ~(np.abs(np64(got) - ref) <= bound)
    assert not bad.any(), (int(bad.sum()), float((np.abs(np64(got) - ref) / bound).max()))


class Stack:
    def __init__(self, gate, fp8, rows, seed=0, layers=2):
        rng = np.random.default_rng(seed)
        self.gate, self.fp8, self.cfg = gate, fp8, K.kda_glr_config(D)
        vec = lambda n, lo, hi: rng.uniform(lo, hi, n).astype(np.float32)  # noqa: E731
        cuda = lambda v: torch.from_numpy(v).cuda()  # noqa: E731
        mat = lambda n, k: (cuda(rng.standard_normal((n, k)).astype(np.float32)) * k ** -0.5).to(torch.bfloat16)  # noqa: E731
        self.vecs, self.layers = [], []
        for _ in range(layers):
            v = dict(A_log=vec(D, -6, 0.6), a_bias=vec(D, -1, 1), b_bias=vec(D, -1, 1), post_w=vec(HIDDEN, 0.8, 1.2), scale=vec(HIDDEN, 0.1, 0.5), pre_w=vec(HIDDEN, 0.8, 1.2))
            d = {n: cuda(x) for n, x in v.items()}
            w_in, w_o = mat(L.glr_width(self.cfg, gate), HIDDEN), mat(HIDDEN, D)
            self.vecs.append(v)
            self.layers.append(L.GlrLayerWeights(L.fp8_weight(w_in) if fp8 else w_in, L.fp8_weight(w_o) if fp8 else w_o,
                                                 K.kda_glr_params_from(d["A_log"], d["a_bias"], d["b_bias"]),
                                                 K.kda_block_norm_params_from(d["post_w"], d["scale"], d["pre_w"])))
        self.run = L.GlrLayerRunner(self.cfg, HIDDEN, rows, "cuda", gate=gate, fp8=fp8)
        self.S = torch.zeros(layers, 6, D, device="cuda")
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def h(self, n):
        return np64(self.run.h[:n]) if not self.fp8 else F8.whole(np64(self.run.h[:n]), np64(self.run.hs[:n]), 1)

    def product(self, x, w, y):
        w64 = F8.whole(np64(w.q), np64(w.s), 128) if self.fp8 else np64(w)
        if self.fp8 and x is not None:
            q, s = F8.quantise(x, 1)
            x = F8.whole(q, s, 1)
        near(y, x @ w64.T, 2.0 ** -12 * (np.abs(x) @ np.abs(w64).T))

    def check_norm(self, i, x, y, x_out, n, last):
        v = self.vecs[i]
        r = block_norm.forward(x, y, None, *(v[k].astype(np.float64) for k in ("post_w", "scale", "pre_w")))
        if x_out is not None:
            near(x_out, r["x1"], r["x1_err"])
        if not last:
            half = 2.0 ** -4 if self.fp8 else 2.0 ** -8
            err = r["h_err"] + (2.0 ** -10 * np.repeat(np64(self.run.hs[:n]), 128, 1)[:, :HIDDEN] if self.fp8 else 0)
            bad = ~(np.abs(self.h(n) - r["h"]) <= err + half * (np.abs(r["h"]) + err))
            assert not bad.any()

    def step(self, x, lens, src, dst, decode):
        """Both layers over rows x, sequences of lens tokens from slots src to dst; every step checked. The stream after them."""
        n, run = x.shape[0], self.run
        si, di = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in (src, dst))
        cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        run.enter(self.layers[0].norm, x)
        torch.cuda.synchronize()
        self.check_norm(0, np64(x), None, None, n, False)
        for i, lw in enumerate(self.layers):
            h, S0, x0 = self.h(n), np64(self.S[i]), np64(x)
            last = i == len(self.layers) - 1
            out = torch.empty_like(x) if i == 0 else x  # the second in place
            if decode:
                run.decode(lw, self.S[i], si, di, lens[0], x, out, last=last, err=self.err)
            else:
                run.prefill(lw, self.S[i], si, di, torch.from_numpy(cu).cuda(), cu, x, out, last=last, err=self.err)
            torch.cuda.synchronize()
            p = np64(run.proj[:n])
            w64 = F8.whole(np64(lw.w_in.q), np64(lw.w_in.s), 128) if self.fp8 else np64(lw.w_in)
            near(run.proj[:n], h @ w64.T, 2.0 ** -12 * (np.abs(h) @ np.abs(w64).T))
            v = self.vecs[i]
            for s, (a, b) in enumerate(zip(src, dst)):
                r = slice(cu[s], cu[s + 1])
                f = glr(p[r, :D], p[r, D:2 * D], p[r, 2 * D:3 * D], p[r, 3 * D:4 * D] if self.gate else None, v["A_log"], v["a_bias"], v["b_bias"],
                        S0[a] if a >= 0 else np.zeros(D))
                near(run.o[r], f["out"], f["out_err"])
                near(self.S[i][b], f["S"], f["S_err"], 2.0 ** -24)
            self.product(np64(run.o[:n]), lw.w_o, run.y[:n])
            self.check_norm(i, x0, np64(run.y[:n]), out, n, last)
            x = out
        assert int(self.err.item()) == 0
        return x


@pytest.mark.parametrize("gate,fp8", [(True, False), (False, False), (True, True), (False, True)])
def test_stack(gate, fp8):
    k = Stack(gate, fp8, 300, seed=1 + 2 * gate + fp8)
    rng = torch.Generator("cuda").manual_seed(3)
    rows = lambda n: torch.randn(n, HIDDEN, device="cuda", generator=rng).to(torch.bfloat16)  # noqa: E731
    k.step(rows(217), [130, 0, 87], [-1, -1, -1], [0, 1, 2], False)
    k.step(rows(3), [1, 1, 1], [0, 1, 2], [0, 1, 2], True)
    k.step(rows(9), [3, 3, 3], [0, 1, 2], [3, 4, 5], True)
    k.step(rows(40), [40], [0], [0], False)


def test_a_captured_decode_step():
    k = Stack(True, True, 8, seed=9)
    gen = torch.Generator("cuda").manual_seed(4)
    x0 = torch.randn(4, HIDDEN, device="cuda", generator=gen).to(torch.bfloat16)
    x, out = x0.clone(), torch.empty_like(x0)
    k.S.normal_(generator=gen)
    S0 = k.S.clone()
    slots = torch.arange(4, dtype=torch.int32, device="cuda")

    def step():
        k.run.enter(k.layers[0].norm, x)
        k.run.decode(k.layers[0], k.S[0], slots, slots, 1, x, out, err=k.err)
        k.run.decode(k.layers[1], k.S[1], slots, slots, 1, out, out, last=True, err=k.err)

    step()
    torch.cuda.synchronize()
    want, S1 = out.clone(), k.S.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    k.S.copy_(S0)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(want, out) and torch.equal(S1, k.S)


def test_refusals():
    k = Stack(True, False, 8)
    x = torch.zeros(9, HIDDEN, device="cuda", dtype=torch.bfloat16)
    slot = torch.zeros(1, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        k.run.enter(k.layers[0].norm, x)
    with pytest.raises(ValueError):
        k.run.decode(k.layers[0], k.S[0], slot, slot, 9, x, x)
    with pytest.raises(TypeError):
        k.run.decode(Stack(True, True, 8).layers[0], k.S[0], slot, slot, 1, x[:1], x[:1])
    with pytest.raises(ValueError):
        L.GlrLayerRunner(K.kda_glr_config(D, K.KDA_F32), HIDDEN, 8, "cuda")
    graph = torch.cuda.CUDAGraph()
    cu = torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    with pytest.raises(RuntimeError, match="before one is captured"):
        with torch.cuda.graph(graph):
            k.run.prefill(k.layers[0], k.S[0], slot, slot, cu, [0, 8], x[:8], x[:8])
    k.run.enter(k.layers[0].norm, x[:8])  # the runner is as it was
    k.run.prefill(k.layers[0], k.S[0], slot, slot, cu, [0, 8], x[:8], x[:8])
    torch.cuda.synchronize()
