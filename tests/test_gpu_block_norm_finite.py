"""The norms around a block where values are not finite, or nothing but zeros: a row keeps to itself, and E4M3 rows are those that
kda_quant_fp8 makes of h in FP32, to the bit."""
import pytest
import torch

import linear_attention_mixer_gb300 as K
from tests.test_gpu_block_norm import Problem

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from linear_attention_mixer_gb300 import build
    build.build()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("M,D,bf16,gate", [(9, 136, True, True), (9, 136, False, False), (40, 1040, True, True), (1301, 1032, True, True), (1250, 4100, False, True),
                                           (77, 8200, True, True), (700, 8208, False, False)])
@pytest.mark.parametrize("value", [NAN, INF])
def test_a_row_keeps_to_itself(M, D, bf16, gate, value):
    """Rows beside the one that has it are the same to the bit."""
    for name in ("x", "y", "dh", "dx1") + (("g",) if gate else ()):
        p, q = (Problem(M, D, bf16, gate, seed=20) for _ in range(2))
        row = M // 2
        q.dev[name][row, D - 3] = value
        same = torch.arange(M, device="cuda") != row
        for a, b in zip(p.forward(), q.forward()):
            assert torch.equal(a[same], b[same]), name
            if name in ("x", "y") and value != value:
                assert bool(b[row, D - 3].isnan())
        g, h = p.backward(), q.backward()
        for n in ("dx", "dy") + (("dg",) if gate else ()):
            assert torch.equal(g[n][same], h[n][same]), (name, n)
        if value != value:  # x' is an input here: dx knows neither y nor g
            assert bool(h["dy" if name in "yg" else "dx"][row, D - 3].isnan()), name


def fp8_of(p):
    """E4M3 rows and scales from the norms, and from the quantiser of their FP32 h."""
    _, h = p.forward()
    q, q2 = (torch.zeros(p.M, p.D, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2))
    s, s2 = (torch.full((p.M, -(-p.D // 128)), -7.0, device="cuda") for _ in range(2))
    K.kda_block_norm(p.cfg, p.params, p.dev["x"], y=p.dev["y"], g=p.dev["g"], x_out=p.new(), h=q, hs=s)
    K.kda_quant_fp8(h, q2, s2)
    torch.cuda.synchronize()
    return h, q.view(torch.uint8), s, q2.view(torch.uint8), s2


@pytest.mark.parametrize("M,D,gate", [(6, 144, True), (5, 400, False), (1300, 528, True), (7, 1040, True), (1250, 4112, False), (4, 8208, True), (640, 8208, False)])
def test_fp8_rows_of_zeros_and_of_what_is_not_finite(M, D, gate):
    def edit(h):
        h["x"][1], h["y"][1] = 0, 0  # a row of zeros
        h["pre_w"][:128] = 0.0       # a group of zeros in every row

    p = Problem(M, D, False, gate, seed=21, edit=edit)
    h, q, s, q2, s2 = fp8_of(p)
    assert torch.equal(q, q2) and torch.equal(s, s2)
    assert bool((q[1] & 0x7F == 0).all()) and bool((s[1] == 1).all()) and bool((q[:, :128] & 0x7F == 0).all()) and bool((s[:, 0] == 1).all())

    def edit(h):  # noqa: F811
        h["pre_w"][5], h["pre_w"][D - 1] = INF, -INF  # in the first group and in the last, shorter than 128 columns
        h["pre_w"][130:134] = NAN
        h["x"][2, 7] = NAN          # a whole row
        h["x"][3, 9] = INF          # rms infinite: zeros, and a NaN where it was
    p = Problem(M, D, False, gate, seed=22, edit=edit)
    h, q, s, q2, s2 = fp8_of(p)
    assert torch.equal(q, q2) and torch.equal(s, s2)
    assert bool(s.isfinite().all()) and bool((s > 0).all())
    bad = ~h.isfinite()
    assert bool(((q & 0x7F == 0x7F) == bad).all()) and bool(bad[2].all()) and bool(bad[0, 5]) and bool(bad[0, D - 1]) and not bool(bad[0, 6:128].any())


def test_fp8_rows_before_a_first_block():
    """h of x alone, with BF16 rows: as in FP32, whose values these are."""
    p = Problem(33, 400, True, False, seed=23)
    p.dev["x"][4, 3] = NAN
    p.dev["x"][5] = 0
    out = {}
    for bf16 in (True, False):
        cfg = K.kda_block_norm_config(400, K.KDA_BF16 if bf16 else K.KDA_F32)
        q, s = torch.zeros(33, 400, dtype=torch.float8_e4m3fn, device="cuda"), torch.zeros(33, 4, device="cuda")
        K.kda_block_norm(cfg, p.params, p.dev["x"] if bf16 else p.dev["x"].float(), h=q, hs=s)
        out[bf16] = q.view(torch.uint8), s
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out[True], out[False]))
