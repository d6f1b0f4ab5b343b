"""The gated linear recurrence's and the block norms' gradients in FP64 against differences of their results."""
import numpy as np
import pytest

from oracle import block_norm, glr


def _differences(f, v, step=1e-6):
    """The gradient of f() by the array v, by central differences in place."""
    d = np.zeros_like(v)
    for i in np.ndindex(v.shape):
        old = v[i]
        v[i] = old + step
        hi = f()
        v[i] = old - step
        d[i] = (hi - f()) / (2 * step)
        v[i] = old
    return d


@pytest.mark.parametrize("gate", [False, True])
def test_recurrence(gate):
    rng = np.random.default_rng(3)
    T, D = 6, 3
    v = {n: rng.standard_normal((T, D)) for n in ("x", "a", "b", "g", "dout")} | {n: rng.standard_normal(D) for n in ("a_bias", "b_bias", "h0", "dS")}
    v["A_log"] = rng.uniform(-4, 1, D)
    if not gate:
        v["g"] = None
    args = ("x", "a", "b", "g", "A_log", "a_bias", "b_bias", "h0")

    def loss():
        f = glr.glr(*(v[n] for n in args))
        return (f["out"] * v["dout"]).sum() + (f["S"] * v["dS"]).sum()

    r = glr.grad(*(v[n] for n in args), v["dout"], v["dS"])
    for n, got in (("x", "dx"), ("a", "da"), ("b", "db"), ("g", "dg"), ("A_log", "dA_log"), ("a_bias", "da_bias"), ("b_bias", "db_bias"), ("h0", "dS")):
        if v[n] is not None:
            np.testing.assert_allclose(r[got], _differences(loss, v[n]), rtol=1e-7, atol=1e-8)


def test_recurrence_by_hand():
    """One channel, two tokens, alpha = exp(-log(2) / 2 x ...): A_log = log(2 log 2), a = 0 gives alpha = 1/2."""
    A_log = np.array([np.log(2 * np.log(2.0))])
    z = np.zeros(1)
    f = glr.glr(np.array([[4.0], [0.0]]), np.zeros((2, 1)), np.zeros((2, 1)), None, A_log, z, z, np.array([2.0]))
    u = np.sqrt(0.75) * 0.5 * 4.0
    np.testing.assert_allclose(f["out"][:, 0], [1.0 + u, (1.0 + u) / 2], rtol=1e-14)


@pytest.mark.parametrize("gate", [False, True])
def test_norms(gate):
    rng = np.random.default_rng(4)
    M, D = 2, 5
    v = {n: rng.standard_normal((M, D)) for n in ("x", "y", "g", "dh", "dx1")} | {n: rng.standard_normal(D) for n in ("post_w", "scale", "pre_w")}
    if not gate:
        v["g"] = None

    def loss():
        f = block_norm.forward(*(v[n] for n in ("x", "y", "g", "post_w", "scale", "pre_w")))
        return (f["x1"] * v["dx1"]).sum() + (f["h"] * v["dh"]).sum()

    x1 = block_norm.forward(*(v[n] for n in ("x", "y", "g", "post_w", "scale", "pre_w")))["x1"]
    r = block_norm.backward(x1, *(v[n] for n in ("y", "g", "post_w", "scale", "pre_w", "dh", "dx1")))
    for n in ("x", "y", "g", "post_w", "scale", "pre_w"):
        if v[n] is not None:
            np.testing.assert_allclose(r["d" + n], _differences(loss, v[n]), rtol=1e-7, atol=1e-8)
