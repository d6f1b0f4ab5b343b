"""Host-side refusals of the gated linear recurrence's and the block norms' entry points: bad arguments are turned away
before anything touches a device (no GPU needed; the pointers below are never followed)."""
import ctypes

import numpy as np
import pytest

import linear_attention_mixer_gb300 as KG


@pytest.fixture(scope="module")
def K():
    from linear_attention_mixer_gb300 import build
    build.build()
    KG.lib()
    return KG


P = 1 << 20  # an aligned address
BIG = 1 << 40


def ints(v):
    return np.array(v, dtype=np.int32).ctypes.data_as(ctypes.POINTER(ctypes.c_int32))


def test_configs(K):
    c = K.kda_glr_config(4096)
    assert (c.dim, c.io_dtype) == (4096, K.KDA_BF16)
    assert K.kda_glr_config(4, K.KDA_F32).dim == 4 and K.kda_glr_config(1 << 20).dim == 1 << 20
    b = K.kda_block_norm_config(7168)
    assert (b.dim, b.io_dtype) == (7168, K.KDA_BF16) and b.eps == pytest.approx(1e-6)
    for make, bads in ((K.kda_glr_config, ((0,), (-8,), (4,), (12,), ((1 << 20) + 8,), (6, 0), (64, 2))),
                       (K.kda_block_norm_config, ((0,), (-8,), (4,), (16392,), (2, 0), (64, 7)))):
        for bad in bads:
            with pytest.raises(K.KdaError) as e:
                make(*bad)
            assert e.value.status == K.KDA_ERR_INVALID
    L = K.lib()
    assert L.kda_glr_config(None, 64, 1) == K.KDA_ERR_INVALID and L.kda_block_norm_config(None, 64, 1) == K.KDA_ERR_INVALID


def test_lengths(K):
    c = K.kda_glr_config(64)
    for cu in ([1, 2], [0, 5, 4], [0, -1], [0, 2 ** 31 - 2 ** 16 + 1], [0, 2 ** 31 - 1]):
        with pytest.raises(K.KdaError):
            K.kda_glr_workspace_bytes(c, cu)
        with pytest.raises(K.KdaError):
            K.kda_glr_chunks(cu)
    for cu in (np.array([0, 2 ** 32 + 64]), [0, 64.5]):
        with pytest.raises(ValueError):
            K.kda_glr_chunks(cu)
    # every sequence's chunks of 16 tokens have rows of their own
    rng = np.random.default_rng(0)
    for lens in ([0], [1], [16], [17], [15, 1, 16, 0, 0, 33], list(rng.integers(0, 40, 50)), [2 ** 31 - 2 ** 16]):
        cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        used = [cu[s] // 16 + s + k for s in range(len(lens)) for k in (range(-(-int(lens[s]) // 16)) if lens[s] < 10 ** 6 else [-(-int(lens[s]) // 16) - 1])]
        assert len(set(used)) == len(used) and (not used or max(used) < K.kda_glr_chunks(cu))
    assert K.kda_glr_chunks([0]) == 0
    L = K.lib()
    assert L.kda_glr_workspace_bytes(None, None, 0) == 0 and L.kda_glr_workspace_bytes(ctypes.byref(c), None, 2) == 0
    assert L.kda_glr_chunks(None, 1) == -1 and L.kda_glr_chunks(ints([0]), -1) == -1


GLR_BAD = [{"x": None}, {"a": P + 8}, {"b": P + 2}, {"g": P + 4}, {"out": None}, {"x_stride": 255}, {"a_stride": 260}, {"b_stride": -8},
           {"g_stride": 128}, {"out_stride": BIG}]


@pytest.mark.parametrize("edit", GLR_BAD)
def test_glr_rows(K, edit):
    c, prm, L, b = K.kda_glr_config(256), K.kda_glr_params(P, P, P), K.lib(), ctypes.byref
    r = K.kda_glr_rows(P, P, P, P, P, *[256] * 5)
    g = K.kda_glr_grad_rows(*[P] * 9, *[256] * 9)
    for n, v in edit.items():
        setattr(r, n, v)
        setattr(g, n.replace("out", "dout"), v)
    assert L.kda_glr_decode(b(c), b(prm), P, 4, P, P, 2, 1, b(r), None, None) == K.KDA_ERR_INVALID
    assert L.kda_glr_prefill(b(c), b(prm), P, 4, P, P, P, ints([0, 64, 70]), 2, b(r), None, P, BIG, None, None) == K.KDA_ERR_INVALID
    assert L.kda_glr_backward(b(c), b(prm), P, ints([0, 64, 70]), 2, P, b(g), None, None, None, None, None, P, BIG, None, None) == K.KDA_ERR_INVALID
    assert K.kda_last_error()


def test_glr_calls(K):
    c, prm, L, b = K.kda_glr_config(256), K.kda_glr_params(P, P, P), K.lib(), ctypes.byref
    r, g = K.kda_glr_rows(P, P, P, None, P, *[256] * 5), K.kda_glr_grad_rows(P, P, P, None, P, P, P, P, None, *[256] * 9)
    cu, need = ints([0, 64, 70]), K.kda_glr_workspace_bytes(c, [0, 64, 70])
    good = dict(c=b(c), prm=b(prm), S=P, slots=4, src=P, dst=P, B=2, n=1, r=b(r), cu=P, cuh=cu, starts=P, ws=P, bytes=need)

    def decode(**e):
        x = good | e
        return L.kda_glr_decode(x["c"], x["prm"], x["S"], x["slots"], x["src"], x["dst"], x["B"], x["n"], x["r"], None, None)

    def prefill(**e):
        x = good | e
        return L.kda_glr_prefill(x["c"], x["prm"], x["S"], x["slots"], x["src"], x["dst"], x["cu"], x["cuh"], x["B"], x["r"], x["starts"],
                                 x["ws"], x["bytes"], None, None)

    broken, no_A = K.kda_glr_config(256), K.kda_glr_params(None, P, P)
    broken.dim = 12
    shared = [{"c": None}, {"c": b(broken)}, {"prm": None}, {"prm": b(no_A)}, {"prm": b(K.kda_glr_params(P, P + 4, P))}, {"S": None}, {"S": P + 8},
              {"slots": 0}, {"src": None}, {"dst": None}, {"B": -1}, {"r": None}]
    for e in shared + [{"n": 0}, {"n": 9}, {"B": 2 ** 31 - 1}]:
        assert decode(**e) == K.KDA_ERR_INVALID, e
    for e in shared + [{"cu": None}, {"cuh": None}, {"cuh": ints([0, 5, 4])}, {"starts": P + 4}, {"ws": None}, {"ws": P + 8}, {"bytes": need - 1}]:
        assert prefill(**e) == K.KDA_ERR_INVALID, e
    assert decode(B=0) == K.KDA_OK and prefill(B=0) == K.KDA_OK

    def back(rows=g, **e):
        x = good | dict(dS=None, dS0=None, sums=(None,) * 3) | e
        return L.kda_glr_backward(x["c"], x["prm"], x["cu"], x["cuh"], x["B"], x["starts"], None if rows is None else b(rows), x["dS"], x["dS0"], *x["sums"],
                                  x["ws"], x["bytes"], None, None)

    for e in ({"c": None}, {"prm": None}, {"prm": b(no_A)}, {"cu": None}, {"cuh": None}, {"B": -1}, {"starts": None}, {"starts": P + 4}, {"rows": None},
              {"dS": P + 4}, {"dS0": P + 8}, {"sums": (P + 4, None, None)}, {"sums": (None, None, P + 2)}, {"ws": None}, {"bytes": need - 1}):
        assert back(**e) == K.KDA_ERR_INVALID, e
    for edit in ({"dx": None}, {"da": P + 8}, {"db": None}, {"dg": P}, {"g": P}, {"dx_stride": 8}, {"dout": None}):
        bad = K.kda_glr_grad_rows(P, P, P, None, P, P, P, P, None, *[256] * 9)
        for n, v in edit.items():
            setattr(bad, n, v)
        assert back(rows=bad) == K.KDA_ERR_INVALID, edit


def norm_rows(K, **e):
    r = K.kda_block_norm_rows(P, P, P, P, P, None, *[256] * 5)
    for n, v in e.items():
        setattr(r, n, v)
    return r


def test_block_norm_calls(K):
    c, prm, L, b = K.kda_block_norm_config(256), K.kda_block_norm_params(P, P, P), K.lib(), ctypes.byref
    assert L.kda_block_norm(b(c), b(prm), 0, b(norm_rows(K)), None) == K.KDA_OK
    for e in ({"x": None}, {"x": P + 8}, {"y": P + 4}, {"y": None}, {"g": P + 8}, {"x_out": None}, {"h": P + 8}, {"h": None, "hs": P}, {"hs": P + 2},
              {"x_stride": 255}, {"y_stride": 252}, {"g_stride": -8}, {"x_out_stride": 128}, {"h_stride": BIG},
              {"y": None, "g": None, "x_out": None, "h": None}, {"y": None, "x_out": None}, {"h": P + 4, "hs": P}, {"h_stride": 260, "hs": P}):
        assert L.kda_block_norm(b(c), b(prm), 3, b(norm_rows(K, **e)), None) == K.KDA_ERR_INVALID, e
    odd = K.kda_block_norm_config(264)
    r = norm_rows(K, hs=P, **{n + "_stride": 264 for n in ("x", "y", "g", "x_out", "h")})
    assert L.kda_block_norm(b(odd), b(prm), 3, b(r), None) == K.KDA_ERR_INVALID and "multiple of 16" in K.kda_last_error()
    for args in ((None, b(prm), 3, b(norm_rows(K))), (b(c), None, 3, b(norm_rows(K))), (b(c), b(prm), -1, b(norm_rows(K))), (b(c), b(prm), 1 << 31, b(norm_rows(K))),
                 (b(c), b(prm), 3, None), (b(c), b(K.kda_block_norm_params(None, P, P)), 3, b(norm_rows(K))),
                 (b(c), b(K.kda_block_norm_params(P, P, P + 4)), 3, b(norm_rows(K)))):
        assert L.kda_block_norm(*args, None) == K.KDA_ERR_INVALID
    bad = K.kda_block_norm_config(256)
    bad.eps = 0.0
    assert L.kda_block_norm(b(bad), b(prm), 3, b(norm_rows(K)), None) == K.KDA_ERR_INVALID
    assert L.kda_block_norm_workspace_bytes(b(bad), 3) == 0 and L.kda_block_norm_workspace_bytes(b(c), -1) == 0
    with pytest.raises(K.KdaError):
        K.kda_block_norm_workspace_bytes(c, 1 << 31)

    need = K.kda_block_norm_workspace_bytes(c, 3)

    def back(rows=None, sums=(P, P, P), M=3, ws=P, nbytes=need, **e):
        r = K.kda_block_norm_grad_rows(*[P] * 8, *[256] * 8)
        for n, v in e.items():
            setattr(r, n, v)
        return L.kda_block_norm_backward(b(c), b(prm), M, b(r), *sums, ws, nbytes, None)

    for e in ({"x_out": None}, {"dh": P + 8}, {"dx1": P + 4}, {"y": P + 8}, {"y": None}, {"g": None}, {"dg": None}, {"dy": None}, {"dx": None}, {"dx_stride": 8},
              {"dh_stride": 260}, {"y": None, "g": None, "dg": None}, {"y": None, "g": None, "dg": None, "dy": None, "dh": None}, {"sums": (P + 4, P, P)}, {"ws": None},
              {"ws": P + 8}, {"nbytes": need - 1}, {"M": -1}, {"M": 1 << 31}):
        assert back(**e) == K.KDA_ERR_INVALID, e


def test_binding_checks(K):
    import torch
    z = torch.zeros(64)
    with pytest.raises(TypeError):
        K.kda_glr_params_from(z, z, z)
    with pytest.raises(TypeError):
        K.kda_block_norm_params_from(z, z, z)
