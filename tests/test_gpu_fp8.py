"""The FP8 quantiser bit for bit, and the FP8 product, against oracle/fp8.py.

The quantiser divides by a power of two and rounds once, so its codes and scales equal the oracle's. The
product: E4M3 times E4M3 is exact in FP32; a sum of K <= 16384 terms takes at most 128 roundings in a block
and one a block outside, fewer than 256 of 2^-24 of the sum of absolute terms, 2^-16 with the scale; then
the result is rounded to BF16, half a step of which is 2^-8."""
import numpy as np
import pytest
import torch

import kda_inputs as KI
import linear_attention_mixer_gb300 as K
from oracle import fp8 as O8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from linear_attention_mixer_gb300 import build
    build.build()
    torch.cuda.set_device(0)


def quant(x, rows, dtype, pad=0):
    """x (numpy) through kda_quant_fp8, from rows `pad` elements apart: values of q, s."""
    M, Kd = x.shape
    wide = torch.full((M, Kd + pad), float("nan"), dtype=dtype, device="cuda")
    wide[:, :Kd] = torch.from_numpy(x).to(dtype)
    q = torch.zeros(M + 1, Kd, dtype=torch.uint8, device="cuda").fill_(0x55).view(torch.float8_e4m3fn)
    s = torch.full((-(-M // rows) + 1, -(-Kd // 128)), -3.0, device="cuda")
    K.kda_quant_fp8(wide[:, :Kd], q[:M], s[:-1], block_rows=rows)
    torch.cuda.synchronize()
    assert bool((q[M:].view(torch.uint8) == 0x55).all()) and bool((s[-1] == -3.0).all())
    return q[:M].float().cpu().numpy(), s[:-1].cpu().numpy()


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,Kd,pad", [(1, 16, 0), (1, 128, 0), (3, 144, 8), (128, 128, 0), (129, 272, 16), (257, 1040, 0)])
def test_quantiser(M, Kd, pad, dtype, rows):
    rng = np.random.default_rng([M, Kd])
    x = rng.standard_normal((M, Kd)) * np.exp(3 * rng.standard_normal((M, 1)))
    x = KI.bf16_round(x.astype(np.float32)) if dtype == torch.bfloat16 else x.astype(np.float32)
    q, s = quant(x, rows, dtype, pad)
    qr, sr = O8.quantise(x, rows)
    assert np.array_equal(s, sr) and np.array_equal(q, qr)


@pytest.mark.parametrize("rows", [1, 128])
def test_quantiser_edges(rows):
    """Zero groups, a group whose largest value is exactly 448 * 2^e or just above, ties between two codes,
    denormals, the largest FP32 numbers, and values that are not finite."""
    x = np.zeros((11, 256), dtype=np.float32)
    x[1, :4] = 448.0, 1.0, -17.0, 0.001
    x[2, :4] = np.nextafter(np.float32(448.0), np.float32(1e9)), 17.0, -19.0, 2.0 ** -10
    x[3, :] = np.arange(256) / 16.0
    x[4, :3] = 1e-44, -3e-45, 1.2e-38
    x[5, :3] = 3.4e38, -1e38, 1.0
    x[6, :] = 448.0 * 2.0 ** -126
    x[7, 128:] = -2.0 ** -9
    x[8, :4] = np.nan, 5.0, -448.0, 2.0 ** -9
    x[9, :5] = np.inf, -np.inf, 1.0, -2.5, 3.0
    x[10, :] = np.nan
    blocks = [x] if rows == 1 else [x[i:i + 1] for i in range(11)] + [x[:8]]
    for b in blocks:
        q, s = quant(np.ascontiguousarray(b), rows, torch.float32)
        qr, sr = O8.quantise(b, rows)
        assert np.array_equal(s, sr) and np.array_equal(q, qr, equal_nan=True)


def operands(M, N, Kd, seed=0):
    rng = np.random.default_rng([seed, M, N, Kd])
    xq, xs = O8.quantise(rng.standard_normal((M, Kd)) * np.exp(rng.standard_normal((M, 1))), 1)
    wq, ws = O8.quantise(rng.standard_normal((N, Kd)) * Kd ** -0.5, 128)
    xs = (xs * rng.uniform(0.5, 2.0, xs.shape)).astype(np.float32)  # any FP32 scales
    ws = (ws * rng.uniform(0.5, 2.0, ws.shape)).astype(np.float32)
    return xq, xs, wq, ws


def dev8(q):
    return torch.from_numpy(q.astype(np.float32)).cuda().to(torch.float8_e4m3fn)


def product(ops, r=None, ysplit=0, **kw):
    xq, xs, wq, ws = ops
    (M, Kd), N = xq.shape, wq.shape[0]
    work = torch.empty(K.kda_linear_fp8_workspace_bytes(M, N, Kd), dtype=torch.uint8, device="cuda").fill_(0xFF)
    work[:4] = 0
    y = torch.full((M * N + 64,), -7.0, dtype=torch.bfloat16, device="cuda")
    rd = None if r is None else torch.from_numpy(r).cuda().to(torch.bfloat16)
    K.kda_linear_fp8(dev8(xq), torch.from_numpy(xs).cuda(), dev8(wq), torch.from_numpy(ws).cuda(), y[:M * N], work, r=rd,
                     ysplit=ysplit, **kw)
    torch.cuda.synchronize()
    assert int(work[:4].view(torch.int32).item()) == 0
    assert bool((y[M * N:] == -7.0).all())
    out = y[:M * N].float().cpu().numpy().astype(np.float64)
    return np.concatenate(list(out.reshape(N // ysplit, M, ysplit)), axis=1) if ysplit else out.reshape(M, N)


def near(got, ref, mag):
    bound = 2.0 ** -8 * np.abs(ref) + 2.0 ** -16 * mag
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), (int(bad.sum()), float(np.nanmax(np.abs(got - ref) / bound)))


SIZES = [(1, 8, 16), (1, 128, 128), (5, 136, 144), (16, 1024, 4096), (37, 256, 272), (128, 384, 128), (129, 264, 400),
         (200, 1000, 2064), (300, 72, 8192), (513, 2056, 640), (1200, 4104, 1040), (2500, 640, 96), (70, 640, 16384)]


@pytest.mark.parametrize("M,N,Kd", SIZES)
@pytest.mark.parametrize("res", [False, True])
def test_product(M, N, Kd, res):
    ops = operands(M, N, Kd)
    r = KI.bf16_round(np.random.default_rng(5).standard_normal((M, N)).astype(np.float32)) if res else None
    got = product(ops, r)
    near(got, *O8.linear(*ops, r))
    assert np.array_equal(got, product(ops, r))  # repeats bit for bit


@pytest.mark.parametrize("M,N,Kd,ysplit", [(1, 512, 1024, 128), (150, 768, 384, 256), (40, 1536, 4096, 384)])
def test_product_split_outputs(M, N, Kd, ysplit):
    ops = operands(M, N, Kd, 1)
    near(product(ops, None, ysplit), *O8.linear(*ops))


@pytest.mark.parametrize("M,N,Kd", [(5, 136, 400), (150, 264, 4096), (1200, 4104, 272)])
@pytest.mark.parametrize("ex,ew", [(70, 60), (-76, -76), (-70, -70), (-126, 20), (100, -126), (120, -20), (-10, 127)])
def test_scales_at_both_ends(M, N, Kd, ex, ew):
    """Scales whose product overflows or underflows where the result does not, in some rows and blocks, among
    ordinary ones; the blocks with a product past 2^127 hold zeros and the smallest codes alone. Beyond the bound
    of `near`: half a step of BF16's smallest numbers, 2^-134."""
    xq, xs, wq, ws = operands(M, N, Kd, 6)
    rng = np.random.default_rng([M, N, Kd, 7])
    rows, blocks = rng.random(M) < 0.4, rng.random(xs.shape[1]) < 0.6
    rows[0] = blocks[0] = True
    if ex + ew > 100:  # E4M3's smallest code is 2^-9, so that a sum is k 2^-18: results of up to 2^126
        small = 2.0 ** -9 * (rng.random((M, Kd)) < 0.02)
        xq = np.where(np.repeat(blocks, 128)[None, :Kd], np.where(rng.random((M, 1)) < 0.5, small, 0), xq)
        wq = np.where(np.repeat(blocks, 128)[None, :Kd], 2.0 ** -9 * rng.integers(-1, 2, (N, Kd)), wq)
    xs = np.where(rows[:, None] & blocks[None], np.ldexp(rng.uniform(1, 2, xs.shape), ex), xs).astype(np.float32)
    ws = np.where(blocks[None], np.ldexp(rng.uniform(1, 2, ws.shape), ew), ws).astype(np.float32)
    if ex + ew < -120:  # rows of scales of that size alone, so that ordinary ones do not hide them
        xs[0], ws[0] = np.ldexp(1.5, ex), np.ldexp(1.25, ew)
    got = product((xq, xs, wq, ws))
    ref, mag = O8.linear(xq, xs, wq, ws)
    assert np.isfinite(ref).all() and np.abs(ref).max() < 3e38
    bad = ~(np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -16 * mag + 2.0 ** -134)
    assert not bad.any(), (int(bad.sum()), got[bad][:4], ref[bad][:4])
    if ex + ew < -120:
        assert (got[0, :128] != 0).any() == (np.abs(ref[0, :128]) > 2.0 ** -134).any()


def test_scales_far_apart_in_neighbouring_rows():
    """Rows whose product of scales is ordinary, though one of the two is huge, beside rows whose product underflows."""
    M, N, Kd = 64, 136, 272
    xq, xs, wq, ws = operands(M, N, Kd, 8)
    xs = np.ldexp(xs, np.where(np.arange(M) % 2, 115, -115)[:, None]).astype(np.float32)
    ws = np.ldexp(ws, -20).astype(np.float32)
    got = product((xq, xs, wq, ws))
    ref, mag = O8.linear(xq, xs, wq, ws)
    assert np.isfinite(ref).all()
    bad = ~(np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -16 * mag + 2.0 ** -134)
    assert not bad.any(), (int(bad.sum()), got[bad][:4], ref[bad][:4])


def test_not_finite_codes_stay_in_their_rows():
    ops = operands(140, 264, 272, 2)
    ops[0][3, 5] = np.nan
    ops[2][200, 9] = np.nan
    got = product(ops)
    ref, mag = O8.linear(*ops)
    hit = np.zeros_like(ref, dtype=bool)
    hit[3], hit[:, 200] = True, True
    assert np.isnan(got[hit]).all()
    near(np.where(hit, 0, got), np.where(hit, 0, ref), np.where(hit, 0, mag))


def test_stream_and_graph():
    ops = operands(33, 384, 4096, 3)
    want = product(ops)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    xq, xs, wq, ws = dev8(ops[0]), torch.from_numpy(ops[1]).cuda(), dev8(ops[2]), torch.from_numpy(ops[3]).cuda()
    x = torch.from_numpy(O8.whole(ops[0], np.ones_like(ops[1]), 1).astype(np.float32)).cuda()
    work = torch.zeros(K.kda_linear_fp8_workspace_bytes(33, 384, 4096), dtype=torch.uint8, device="cuda")
    y = torch.empty(33, 384, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    K.kda_linear_fp8(xq, xs, wq, ws, y, work, stream=st)
    st.synchronize()
    assert np.array_equal(y.float().cpu().numpy(), want)
    q, s = torch.empty_like(xq), torch.empty_like(xs)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        K.kda_quant_fp8(x, q, s)
        K.kda_linear_fp8(q, s, wq, ws, y, work)
    for k in (1.0, -3.0):
        x2 = (O8.whole(ops[0], np.ones_like(ops[1]), 1) * k).astype(np.float32)
        x.copy_(torch.from_numpy(x2))
        g.replay()
        torch.cuda.synchronize()
        qr, sr = O8.quantise(x2, 1)
        near(y.float().cpu().numpy(), *O8.linear(qr, sr, ops[2], ops[3]))


def test_no_rows():
    e = lambda *s, dt=torch.float8_e4m3fn: torch.empty(*s, dtype=dt, device="cuda")
    K.kda_quant_fp8(e(0, 256, dt=torch.bfloat16), e(0, 256), e(0, 2, dt=torch.float32))
    K.kda_linear_fp8(e(0, 256), e(0, 2, dt=torch.float32), e(8, 256), e(1, 2, dt=torch.float32), e(0, 8, dt=torch.bfloat16),
                     e(256, dt=torch.uint8))
    torch.cuda.synchronize()


def test_binding_refusals():
    z = lambda *s, dt=torch.float8_e4m3fn, d="cuda": torch.zeros(*s, dtype=dt, device=d)
    f32, bf, u8 = torch.float32, torch.bfloat16, torch.uint8
    good = dict(xq=z(4, 256), xs=z(4, 2, dt=f32), wq=z(8, 256), ws=z(1, 2, dt=f32), y=z(4, 8, dt=bf), workspace=z(4096, dt=u8))
    K.kda_linear_fp8(**good)
    for bad in ({"xq": z(4, 240)}, {"xs": z(4, 1, dt=f32)}, {"ws": z(2, 2, dt=f32)}, {"y": z(4, 7, dt=bf)}, {"r": z(3, 8, dt=bf)}):
        with pytest.raises(ValueError):
            K.kda_linear_fp8(**{**good, **bad})
    for bad in ({"xq": z(4, 256, dt=u8)}, {"wq": z(8, 256, d="cpu")}, {"y": z(4, 8, dt=f32)}):
        with pytest.raises(TypeError):
            K.kda_linear_fp8(**{**good, **bad})
    for bad in ({"wq": z(12, 256), "y": z(4, 12, dt=bf)}, {"workspace": z(128, dt=u8)}, {"xq": z(4, 264), "wq": z(8, 264), "xs": z(4, 3, dt=f32), "ws": z(1, 3, dt=f32)},
                {"workspace": z(4100, dt=u8)[4:]}):
        with pytest.raises(K.KdaError) as e:
            K.kda_linear_fp8(**{**good, **bad})
        assert e.value.status == K.KDA_ERR_INVALID
    x = z(4, 256, dt=bf)
    K.kda_quant_fp8(x, z(4, 256), z(4, 2, dt=f32))
    for a, kw in (((x, z(4, 255), z(4, 2, dt=f32)), {}), ((x, z(4, 256), z(1, 2, dt=f32)), {}), ((x, z(4, 256), z(4, 2, dt=f32)), {"block_rows": 0}),
                  ((x.t().contiguous().t(), z(4, 256), z(4, 2, dt=f32)), {})):
        with pytest.raises(ValueError):
            K.kda_quant_fp8(*a, **kw)
    for a in ((x.half(), z(4, 256), z(4, 2, dt=f32)), (x, z(4, 256, dt=u8), z(4, 2, dt=f32))):
        with pytest.raises(TypeError):
            K.kda_quant_fp8(*a)
    for a, kw in (((x, z(4, 256), z(2, 2, dt=f32)), {"block_rows": 2}), ((z(4, 40, dt=bf), z(4, 40), z(4, 1, dt=f32)), {}),
                  ((z(4, 257, dt=bf)[:, :256], z(4, 256), z(4, 2, dt=f32)), {}), ((z(4, 264, dt=bf)[:, 1:257], z(4, 256), z(4, 2, dt=f32)), {})):
        with pytest.raises(K.KdaError) as e:
            K.kda_quant_fp8(*a, **kw)
        assert e.value.status == K.KDA_ERR_INVALID
