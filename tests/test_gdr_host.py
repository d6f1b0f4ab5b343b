"""Host-side refusals of the gated delta rule's entry points: bad arguments are turned away before
anything touches a device (no GPU needed; the pointers below are never followed)."""
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


def test_config(K):
    c = K.kda_gdr_config(32, 16)
    assert (c.num_heads, c.num_qk_heads, c.head_dim, c.io_dtype, c.qk_l2norm) == (32, 16, 128, K.KDA_BF16, 1)
    assert c.l2_eps == pytest.approx(1e-6) and c.q_scale == pytest.approx(128 ** -0.5)
    assert K.kda_gdr_config(3).num_qk_heads == 3
    for bad in ((0, 1), (4, 0), (4, 3), (2, 4), (-4, -2), (1 << 17, 1), (4, 2, 64), (4, 2, 128, 5)):
        with pytest.raises(K.KdaError) as e:
            K.kda_gdr_config(*bad)
        assert e.value.status == K.KDA_ERR_INVALID


def test_workspace(K):
    c = K.kda_gdr_config(4, 2)
    one = K.kda_gdr_workspace_bytes(c, [0, 64]) - K.kda_gdr_workspace_bytes(c, [0, 0])
    assert one == 4 * 25856
    for cu, chunks in (([0, 1], 1), ([0, 65], 2), ([0, 0, 64, 64, 129], 3), ([0, 2 ** 31 - 1], 2 ** 25)):
        assert K.kda_gdr_workspace_bytes(c, cu) == K.kda_gdr_workspace_bytes(c, [0, 0]) + chunks * one
    for cu in ([1, 2], [0, 5, 4], [0, -1]):
        with pytest.raises(K.KdaError):
            K.kda_gdr_workspace_bytes(c, cu)
    assert K.lib().kda_gdr_workspace_bytes(None, None, 0) == 0


@pytest.mark.parametrize("cu", [np.array([0, 2 ** 32 + 64]), np.array([2 ** 32, 64]), np.array([0, 2 ** 63], dtype=np.uint64), [0, 64.5],
                                np.array([0.0, np.inf])])
def test_lengths_that_are_no_32_bit_numbers(K, cu):
    """Refused, and not taken modulo 2^32 or cut: their queries would answer for other lengths."""
    c = K.kda_gdr_config(4, 2)
    with pytest.raises(ValueError):
        K.kda_gdr_workspace_bytes(c, cu)
    for same in (np.array([0, 64]), np.array([0, 64], dtype=np.uint8), [0, 64], (0, 64.0), np.array([0, 1, 64], dtype=np.int32)[::2]):
        assert K.kda_gdr_workspace_bytes(c, same) == K.kda_gdr_workspace_bytes(c, np.array([0, 64], dtype=np.int32))


P = 1 << 20  # an aligned address


def rows(K, **edit):
    r = K.kda_gdr_rows(P, P, P, P, P, P, 256, 256, 512, 4, 4, 512)
    for n, x in edit.items():
        setattr(r, n, x)
    return r


BAD_ROWS = [{"q": None}, {"k": P + 2}, {"v": P + 8}, {"a": P + 1}, {"b": None}, {"out": P + 4}, {"q_stride": 255},
            {"q_stride": 260}, {"k_stride": 128}, {"v_stride": 504}, {"a_stride": 3}, {"b_stride": -4},
            {"out_stride": 516}, {"v_stride": 1 << 40}]


@pytest.mark.parametrize("edit", BAD_ROWS)
def test_bad_rows(K, edit):
    c, prm = K.kda_gdr_config(4, 2), K.kda_gdr_params(P, P)
    r = rows(K, **edit)
    L, b = K.lib(), ctypes.byref
    assert L.kda_gdr_decode(b(c), b(prm), P, 4, P, P, 2, 1, b(r), None, None) == K.KDA_ERR_INVALID
    cu = np.array([0, 64, 70], dtype=np.int32)
    cp = cu.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))
    assert L.kda_gdr_prefill(b(c), b(prm), P, 4, P, P, P, cp, 2, b(r), P, 1 << 30, None, None) == K.KDA_ERR_INVALID
    assert K.kda_last_error()


def test_bad_calls(K):
    c, prm, r = K.kda_gdr_config(4, 2), K.kda_gdr_params(P, P), rows(K)
    L, b = K.lib(), ctypes.byref
    good = dict(c=b(c), prm=b(prm), S=P, slots=4, src=P, dst=P, B=2, n=1, r=b(r))

    def decode(**e):
        x = {**good, **e}
        return L.kda_gdr_decode(x["c"], x["prm"], x["S"], x["slots"], x["src"], x["dst"], x["B"], x["n"], x["r"], None, None)

    broken = K.kda_gdr_config(4, 2)
    broken.head_dim = 64
    no_eps = K.kda_gdr_config(4, 2)
    no_eps.l2_eps = 0.0
    inf_scale = K.kda_gdr_config(4, 2)
    inf_scale.q_scale = float("inf")
    for e in ({"c": None}, {"c": b(broken)}, {"c": b(no_eps)}, {"c": b(inf_scale)}, {"prm": None},
              {"prm": b(K.kda_gdr_params(P, None))}, {"S": None}, {"S": P + 4}, {"slots": 0}, {"src": None}, {"dst": None},
              {"B": -1}, {"B": 1 << 30}, {"n": 0}, {"n": 9}, {"r": None}):
        assert decode(**e) == K.KDA_ERR_INVALID, e
    assert decode(B=0) == K.KDA_OK
    cu = np.array([0, 64, 70], dtype=np.int32)
    ptr = lambda a: a.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))

    def prefill(cu_dev=P, host=cu, N=2, ws=P, size=1 << 30):
        return L.kda_gdr_prefill(b(c), b(prm), P, 4, P, P, cu_dev, None if host is None else ptr(host), N, b(r), ws, size, None, None)

    need = K.kda_gdr_workspace_bytes(c, cu)
    for e in ({"cu_dev": None}, {"host": None}, {"N": -1}, {"ws": None}, {"ws": P + 8}, {"size": need - 1},
              {"host": np.array([0, 70, 64], dtype=np.int32)}, {"host": np.array([3, 64, 70], dtype=np.int32)}):
        assert prefill(**e) == K.KDA_ERR_INVALID, e
    assert prefill(N=0) == K.KDA_OK
