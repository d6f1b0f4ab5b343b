"""The norms around a block (kda_block_norm, kda_block_norm_backward) against FP64.

Tolerances are those that oracle/block_norm.py derives beside each result, and half a step of the rows' type for what
is rounded to it. E4M3 rows: half a step there is 2^-4 of a value (and half of 2^-9, its smallest number, times the scale).
"""
import numpy as np
import pytest
import torch

import kda_inputs as KI
import linear_attention_mixer_gb300 as K
from oracle import block_norm, fp8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from linear_attention_mixer_gb300 import build
    build.build()
    torch.cuda.set_device(0)


def near(got, ref, err, bf16=False):
    got = got.detach().cpu().double().numpy()
    bound = err + (2.0 ** -8 * (np.abs(ref) + err) + 2.0 ** -133 if bf16 else 2.0 ** -24 * np.abs(ref)) + 1e-37
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), (int(bad.sum()), float(np.nanmax(np.abs(got - ref) / bound)))


class Problem:
    def __init__(self, M, D, bf16=True, gate=False, seed=0, strided=False, edit=None):
        rng = np.random.default_rng([seed, M, D])
        self.M, self.D, self.bf16, self.gate = M, D, bf16, gate
        self.rows = ("x", "y", "dh", "dx1") + (("g",) if gate else ())
        h = {n: rng.standard_normal((M, D)).astype(np.float32) for n in self.rows}
        h["x"] *= np.exp(rng.standard_normal(D)).astype(np.float32)
        h["y"] *= 0.3
        h["post_w"], h["pre_w"] = (1 + 0.2 * rng.standard_normal((2, D))).astype(np.float32)
        h["scale"] = (0.1 + 0.05 * rng.standard_normal(D)).astype(np.float32)
        if edit:
            edit(h)
        self.h = {n: (KI.bf16_round(v) if bf16 and n in self.rows else v) for n, v in h.items()}
        self.h64 = {n: v.astype(np.float64) for n, v in self.h.items()} | ({} if gate else {"g": None})
        self.dt = torch.bfloat16 if bf16 else torch.float32
        self.dev = {n: torch.from_numpy(v).cuda().to(self.dt if n in self.rows else torch.float32) for n, v in self.h.items()}
        self.strided = strided
        for n in self.rows if strided else ():
            self.dev[n] = self.new(self.dev[n])
        self.dev.setdefault("g", None)
        self.cfg = K.kda_block_norm_config(D, K.KDA_BF16 if bf16 else K.KDA_F32)
        self.params = K.kda_block_norm_params_from(*(self.dev[n] for n in ("post_w", "scale", "pre_w")))

    def new(self, like=None):
        """Rows for an output (or as `like`), beside columns that belong to nobody, and a row behind the last."""
        t = torch.full((self.M + 1, self.D + (24 if self.strided else 0)), -7.0, dtype=self.dt, device="cuda")[:, :self.D]
        if like is not None:
            t[:self.M] = like
        return t[:self.M]

    def forward(self, y=True, h=True):
        d = self.dev
        x1, hh = self.new() if y else None, self.new() if h else None
        K.kda_block_norm(self.cfg, self.params, d["x"], y=d["y"] if y else None, g=d["g"] if y else None, x_out=x1, h=hh)
        torch.cuda.synchronize()
        return x1, hh

    def ref(self, y=True):
        v = self.h64
        return block_norm.forward(v["x"], v["y"] if y else None, v["g"], v["post_w"], v["scale"], v["pre_w"])

    def backward(self, y=True, dh=True, dx1=True, out=None):
        d = self.dev
        g = out or {n: self.new() for n in ("dx",) + (("dy",) if y else ()) + (("dg",) if y and self.gate else ())}
        s = {n: torch.full((self.D,), float("nan"), device="cuda") for n in ("dpost_w", "dscale", "dpre_w")}
        work = torch.empty(K.kda_block_norm_workspace_bytes(self.cfg, self.M), dtype=torch.uint8, device="cuda").fill_(0xFF)
        K.kda_block_norm_backward(self.cfg, self.params, d["x"], d["dh"] if dh else None, d["dx1"] if dx1 else None, g["dx"], work,
                                  y=d["y"] if y else None, g=d["g"] if y else None, dy=g.get("dy"), dg=g.get("dg"), **s)
        torch.cuda.synchronize()
        return g | s

    def check_back(self, got, y=True, dh=True, dx1=True):
        v = self.h64
        r = block_norm.backward(v["x"], v["y"] if y else None, v["g"] if y else None, v["post_w"], v["scale"], v["pre_w"],
                                v["dh"] if dh else None, v["dx1"] if dx1 else None)
        for n, t in got.items():
            if n in r:
                near(t, r[n], r[n + "_err"], self.bf16 and n in ("dx", "dy", "dg"))
            else:
                assert bool((t == 0).all())


SHAPES = [(1, 8, True, True, False), (1, 7168, True, False, False), (3, 4, False, True, True), (130, 64, True, True, True), (5, 256, True, False, False),
          (77, 264, False, True, False), (9, 512, True, True, True), (6, 520, True, False, False), (33, 1004, False, False, True),
          (700, 1024, True, True, False), (4, 1032, True, True, True), (12, 2048, False, True, False), (7, 2056, True, True, False), (5, 4096, True, True, True),
          (3, 4100, False, True, True), (310, 7168, True, True, False), (4, 8192, True, False, False), (2, 8200, True, True, True),
          (3, 16384, False, True, False), (320, 16384, True, False, False)]


@pytest.mark.parametrize("M,D,bf16,gate,strided", SHAPES)
def test_forward_and_backward(M, D, bf16, gate, strided):
    p = Problem(M, D, bf16, gate, strided=strided)
    x1, h = p.forward()
    r = p.ref()
    near(x1, r["x1"], r["x1_err"], bf16)
    near(h, r["h"], r["h_err"], bf16)
    for t in (x1, h):  # the row behind the last
        assert bool((torch.as_strided(t, (1, D), (1, 1), t.storage_offset() + M * t.stride(0)) == -7.0).all())
    p.check_back(p.backward())


def test_more_rows_than_partial_sums():
    for D in (64, 1000):
        p = Problem(3001, D, True, True, seed=1)
        x1, h = p.forward()
        r = p.ref()
        near(h, r["h"], r["h_err"], True)
        p.check_back(p.backward())


@pytest.mark.parametrize("D,bf16,gate,strided", [(520, True, True, False), (1024, False, False, True), (1032, True, False, True), (2048, False, True, False),
                                                (2056, True, True, True), (4096, False, False, False), (4100, False, True, True), (7168, True, True, False),
                                                (8192, True, False, False), (8188, False, True, False)])
def test_many_rows(D, bf16, gate, strided):
    """Blocks that stay and take one row after the other."""
    p = Problem(1301, D, bf16, gate, seed=8, strided=strided)
    x1, h = p.forward()
    r = p.ref()
    near(x1, r["x1"], r["x1_err"], bf16)
    near(h, r["h"], r["h_err"], bf16)
    got = p.backward()
    p.check_back(got)
    again = p.backward()
    assert all(torch.equal(got[n], again[n]) for n in got)
    for t in (x1, h, got["dx"], got["dy"]):  # the row behind the last
        assert bool((torch.as_strided(t, (1, D), (1, 1), t.storage_offset() + p.M * t.stride(0)) == -7.0).all())
    for kw in ({"y": False}, {"dh": False}, {"dx1": False}):
        p.check_back(p.backward(**kw), **kw)


@pytest.mark.parametrize("M,D,bf16,gate,strided", [(1, 264, True, True, False), (151, 16, True, False, True), (305, 4, False, True, False), (2433, 256, True, True, False),
                                                   (3001, 252, False, False, True), (3001, 512, True, True, True), (1217, 508, False, True, False)])
def test_many_short_rows(M, D, bf16, gate, strided):
    p = Problem(M, D, bf16, gate, seed=13, strided=strided)
    got = p.backward()
    p.check_back(got)
    again = p.backward()
    assert all(torch.equal(got[n], again[n]) for n in got)
    for n in ("dx", "dy"):  # the row behind the last
        t = got[n]
        assert bool((torch.as_strided(t, (1, D), (1, 1), t.storage_offset() + M * t.stride(0)) == -7.0).all())
    for kw in ({"y": False}, {"dh": False}, {"dx1": False}):
        p.check_back(p.backward(**kw), **kw)


def test_workspace_grows_with_the_rows():
    """Room for many rows serves fewer."""
    for D in (16, 512, 2048, 8200):
        cfg = K.kda_block_norm_config(D, K.KDA_BF16)
        need = [K.kda_block_norm_workspace_bytes(cfg, M) for M in (*range(1, 2000), 5000, 10000, 59000, 100000, 2 ** 31 - 1)]
        assert need == sorted(need)


@pytest.mark.parametrize("M,D,bf16,gate,strided", [(1, 8200, True, False, False), (76, 16384, False, True, True), (77, 12288, True, True, False),
                                                   (153, 8196, False, False, True), (701, 8200, True, True, True), (650, 16380, False, True, False),
                                                   (611, 16384, True, False, False)])
def test_wide_rows(M, D, bf16, gate, strided):
    """Rows of more than 8192 channels, which two blocks share."""
    p = Problem(M, D, bf16, gate, seed=11, strided=strided)
    x1, h = p.forward()
    r = p.ref()
    near(x1, r["x1"], r["x1_err"], bf16)
    near(h, r["h"], r["h_err"], bf16)
    got = p.backward()
    p.check_back(got)
    again = p.backward()
    assert all(torch.equal(got[n], again[n]) for n in got)
    for t in (x1, h, got["dx"], got["dy"]):  # the row behind the last
        assert bool((torch.as_strided(t, (1, D), (1, 1), t.storage_offset() + M * t.stride(0)) == -7.0).all())
    for kw in ({"y": False}, {"dh": False}, {"dx1": False}):
        p.check_back(p.backward(**kw), **kw)


@pytest.mark.parametrize("bf16", [True, False])
def test_only_one_of_the_norms(bf16):
    p = Problem(40, 200, bf16, True, seed=2)
    _, h = p.forward(y=False)
    r = p.ref(y=False)
    near(h, r["h"], r["h_err"], bf16)
    x1, none = p.forward(h=False)
    assert none is None
    near(x1, p.ref()["x1"], p.ref()["x1_err"], bf16)
    for kw in ({"y": False}, {"dh": False}, {"dx1": False}, {"y": False, "dx1": False}, {"dh": False, "dx1": True}):
        p.check_back(p.backward(**kw), **kw)


def test_in_place():
    p = Problem(50, 136, True, True, seed=3)
    x1, h = p.forward()
    x = p.dev["x"].clone()
    K.kda_block_norm(p.cfg, p.params, x, y=p.dev["y"], g=p.dev["g"], x_out=x, h=p.new())
    g = p.backward()
    first = g["dx"].clone()
    g2 = {n: p.new() for n in ("dy", "dg")} | {"dx": p.dev["dx1"]}
    p.backward(out=g2)
    assert torch.equal(x, x1) and torch.equal(first, p.dev["dx1"]) and torch.equal(g["dy"], g2["dy"])


@pytest.mark.parametrize("M,D,bf16", [(1, 16, True), (5, 128, False), (70, 400, True), (3, 1040, True), (17, 7168, True), (3, 16384, False), (1300, 528, True), (1250, 4096, False)])
def test_fp8(M, D, bf16):
    """The scale is the power of two for the group's largest value (or for one that FP32 could have in its place), and the
    codes are h / scale to half a step."""
    p = Problem(M, D, bf16, True, seed=4)
    q = torch.zeros(M, D, dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.zeros(M, -(-D // 128), device="cuda")
    x1 = p.new()
    K.kda_block_norm(p.cfg, p.params, p.dev["x"], y=p.dev["y"], g=p.dev["g"], x_out=x1, h=q, hs=s)
    r = p.ref()
    near(x1, r["x1"], r["x1_err"], bf16)
    s64 = s.cpu().double().numpy()
    for j in range(s64.shape[1]):
        c = slice(128 * j, 128 * j + 128)
        lo, hi = (np.abs(r["h"][:, c]) - r["h_err"][:, c]).max(1), (np.abs(r["h"][:, c]) + r["h_err"][:, c]).max(1)
        assert (s64[:, j] >= np.exp2(np.ceil(np.log2(lo / 448)))).all() and (s64[:, j] <= np.exp2(np.ceil(np.log2(hi / 448)))).all()
    whole = np.repeat(s64, 128, 1)[:, :D]
    got = q.float().cpu().double().numpy() * whole
    bound = r["h_err"] + np.maximum(2.0 ** -4 * (np.abs(r["h"]) + r["h_err"]), 2.0 ** -10 * whole)
    assert (np.abs(got - r["h"]) <= bound).all()


def test_fp8_rows_are_those_of_the_quantiser():
    """h in FP32, then kda_quant_fp8: the same codes and scales, to the bit."""
    p = Problem(130, 1040, False, True, seed=5)
    _, h = p.forward()
    q, q2 = (torch.zeros(130, 1040, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2))
    s, s2 = (torch.zeros(130, 9, device="cuda") for _ in range(2))
    K.kda_block_norm(p.cfg, p.params, p.dev["x"], y=p.dev["y"], g=p.dev["g"], x_out=p.new(), h=q, hs=s)
    K.kda_quant_fp8(h, q2, s2)
    assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s, s2)


def test_wide_fp8_rows_are_those_of_the_quantiser():
    p = Problem(640, 8208, False, True, seed=12)
    _, h = p.forward()
    q, q2 = (torch.zeros(640, 8208, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2))
    s, s2 = (torch.zeros(640, 65, device="cuda") for _ in range(2))
    K.kda_block_norm(p.cfg, p.params, p.dev["x"], y=p.dev["y"], g=p.dev["g"], x_out=p.new(), h=q, hs=s)
    K.kda_quant_fp8(h, q2, s2)
    assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s, s2)


def test_rows_of_zeros_and_far_gates():
    def edit(h):
        h["x"][3], h["y"][4], h["y"][5], h["x"][5] = 0, 0, 0, 0
        h["g"][6], h["g"][7] = -100, 100
        h["g"][8, ::2], h["g"][8, 1::2] = -np.inf, np.inf
    p = Problem(9, 136, False, True, seed=6, edit=edit)
    x1, h = p.forward()
    v = p.h64
    v["g"] = np.clip(v["g"], -700, 700)
    r = p.ref()
    near(x1, r["x1"], r["x1_err"])
    near(h, r["h"], r["h_err"])
    q = torch.zeros(9, 136, dtype=torch.bfloat16, device="cuda")
    assert bool((h[5] == 0).all()) and bool(x1[8].isfinite().all()) and q is not None


def test_stream_and_graph():
    p = Problem(300, 1000, True, True, seed=7)
    x1, h = p.forward()
    g = p.backward()
    s = torch.cuda.Stream()
    x2, h2 = p.new(), p.new()
    torch.cuda.synchronize()
    K.kda_block_norm(p.cfg, p.params, p.dev["x"], y=p.dev["y"], g=p.dev["g"], x_out=x2, h=h2, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(x1, x2) and torch.equal(h, h2)
    out = {n: torch.empty_like(t) for n, t in g.items()}
    work = torch.empty(K.kda_block_norm_workspace_bytes(p.cfg, p.M), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        K.kda_block_norm(p.cfg, p.params, p.dev["x"], y=p.dev["y"], g=p.dev["g"], x_out=x2, h=h2)
        K.kda_block_norm_backward(p.cfg, p.params, p.dev["x"], p.dev["dh"], p.dev["dx1"], work=work, y=p.dev["y"], g=p.dev["g"], **out)
    x2.zero_(), h2.zero_()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(x1, x2) and torch.equal(h, h2)
    for n in g:
        assert torch.equal(g[n], out[n]), n


def test_no_rows():
    p = Problem(0, 64, True, False)
    p.forward()
    g = p.backward()
    assert all(bool((g[n] == 0).all()) for n in ("dpost_w", "dscale", "dpre_w"))


def test_refusals_of_the_binding():
    p = Problem(20, 64, True, True, seed=9)
    d = p.dev

    def forward(**e):
        v = dict(x=d["x"], y=d["y"], g=d["g"], x_out=p.new(), h=p.new(), hs=None, prm=p.params) | e
        K.kda_block_norm(p.cfg, v["prm"], v["x"], y=v["y"], g=v["g"], x_out=v["x_out"], h=v["h"], hs=v["hs"])

    hs = torch.zeros(20, 1, device="cuda")
    q = torch.zeros(20, 64, device="cuda", dtype=torch.float8_e4m3fn)
    for e in ({"x": d["x"].float()}, {"y": d["y"][:3]}, {"g": d["g"].cpu()}, {"x_out": None}, {"h": q}, {"hs": hs}, {"h": q, "hs": hs[:, 0]}, {"h": q, "hs": hs.half()},
              {"h": None, "hs": hs}, {"y": None}, {"y": None, "g": None, "x_out": None, "h": None}, {"x": d["x"].t()},
              {"prm": K.kda_block_norm_params_from(*(torch.zeros(72, device="cuda") for _ in range(3)))},
              {"prm": K.kda_block_norm_params(p.params.post_w, p.params.scale, p.params.pre_w)}):
        with pytest.raises((TypeError, ValueError, K.KdaError)):
            forward(**e)
    forward(h=q, hs=hs)
    work = torch.empty(K.kda_block_norm_workspace_bytes(p.cfg, 20), dtype=torch.uint8, device="cuda")

    def backward(**e):
        v = dict(x_out=d["x"], dh=d["dh"], dx1=d["dx1"], dx=p.new(), work=work, y=d["y"], g=d["g"], dy=p.new(), dg=p.new(), dscale=None) | e
        K.kda_block_norm_backward(p.cfg, p.params, v["x_out"], v["dh"], v["dx1"], v["dx"], v["work"], y=v["y"], g=v["g"], dy=v["dy"], dg=v["dg"], dscale=v["dscale"])

    for e in ({"x_out": None}, {"dh": d["dh"][:2]}, {"dx1": d["dx1"].float()}, {"work": work[:100]}, {"dy": None}, {"dg": None}, {"g": None}, {"y": None},
              {"dscale": torch.zeros(63, device="cuda")}):
        with pytest.raises((TypeError, ValueError, K.KdaError)):
            backward(**e)
    backward()
    torch.cuda.synchronize()
