"""The FP8 oracle's own arithmetic, and the host-side refusals of the FP8 entry points (no GPU needed; the
pointers below are never followed)."""
import numpy as np
import pytest
import torch

import linear_attention_mixer_gb300 as KG
from oracle import fp8 as O8

P = 1 << 20


@pytest.fixture(scope="module")
def K():
    from linear_attention_mixer_gb300 import build
    build.build()
    KG.lib()
    return KG


def test_oracle_e4m3_is_the_nearest_code():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy().astype(np.float64)
    codes = np.unique(codes[np.isfinite(codes)])
    assert np.array_equal(O8.e4m3(codes), codes) and codes.max() == 448.0
    x = np.concatenate([np.linspace(-448, 448, 20011), np.ldexp(np.linspace(1, 2, 501), -9), -np.ldexp(np.linspace(0, 1, 301), -8)])
    got = O8.e4m3(x)
    best = np.abs(x[:, None] - codes[None]).min(1)
    assert np.array_equal(np.abs(x - got), best)
    mid = (codes[1:] + codes[:-1]) / 2  # a tie goes to the code whose last bit is 0, as FP32 -> E4M3 in torch does
    assert np.array_equal(O8.e4m3(mid), torch.from_numpy(mid).float().to(torch.float8_e4m3fn).double().numpy())


def test_quantiser_refusals(K):
    good = dict(M=4, K=256, x=P, st=256, dt=K.KDA_BF16, rows=1, q=P, s=P)

    def call(**e):
        x = {**good, **e}
        return K.lib().kda_quant_fp8(x["M"], x["K"], x["x"], x["st"], x["dt"], x["rows"], x["q"], x["s"], None)

    for e in ({"M": -1}, {"K": 0}, {"K": 24}, {"x": None}, {"x": P + 8}, {"st": 255}, {"st": 260}, {"dt": 2}, {"rows": 64},
              {"q": None}, {"q": P + 4}, {"s": None}, {"s": P + 2}, {"M": 1 << 40}, {"M": 1 << 62}, {"M": (1 << 63) - 1}, {"st": 1 << 62}, {"dt": K.KDA_F32, "st": 258}):
        assert call(**e) == K.KDA_ERR_INVALID, e
        assert K.kda_last_error()
    assert call(M=0) == K.KDA_OK


def test_product_refusals(K):
    good = dict(M=4, N=256, K=256, xq=P, xs=P, wq=P, ws=P, r=None, y=P, split=0, w=P, size=1 << 30)

    def call(**e):
        x = {**good, **e}
        return K.lib().kda_linear_fp8(x["M"], x["N"], x["K"], x["xq"], x["xs"], x["wq"], x["ws"], x["r"], x["y"], x["split"],
                                      x["w"], x["size"], None)

    for e in ({"M": -1}, {"N": 0}, {"N": 12}, {"K": 8}, {"K": 0}, {"M": 1 << 20, "N": 1 << 12}, {"xq": None}, {"xs": None},
              {"wq": P + 8}, {"ws": P + 1}, {"y": None}, {"y": P + 2}, {"w": None}, {"r": P + 4}, {"split": 64}, {"split": 384},
              {"split": -128}, {"split": 128, "r": P}):
        assert call(**e) == K.KDA_ERR_INVALID, e
        assert K.kda_last_error()
    assert call(M=0) == K.KDA_OK
    for bad in ((4, 12, 256), (4, 256, 8), (-1, 256, 256)):
        with pytest.raises(K.KdaError):
            K.kda_linear_fp8_workspace_bytes(*bad)
    assert K.kda_linear_fp8_workspace_bytes(0, 256, 256) == 256


def test_a_k_whose_blocks_are_not_counted_in_32_bits(K):
    """K + 127 passes 2^31: refused by name, by the product, its query and the quantiser; the largest K is taken."""
    top = 2 ** 31 - 128
    assert K.kda_linear_fp8_workspace_bytes(2, 8, top) > 256  # k splits: partial sums
    for k in (top + 16, 2 ** 31 - 16):
        with pytest.raises(K.KdaError) as e:
            K.kda_linear_fp8_workspace_bytes(2, 8, k)
        assert str(top) in e.value.message
        for M in (0, 2):
            assert K.lib().kda_linear_fp8(M, 8, k, P, P, P, P, None, P, 0, P, 1 << 30, None) == K.KDA_ERR_INVALID
            assert str(top) in K.kda_last_error()
            for rows in (1, 128):
                assert K.lib().kda_quant_fp8(M, k, P, k, K.KDA_BF16, rows, P, P, None) == K.KDA_ERR_INVALID
                assert str(top) in K.kda_last_error()
