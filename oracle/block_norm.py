"""The norms around a block, fused with its residual, in FP64 (numpy): x' = x + scale sigmoid(g) post_w y / rms(y),
h = pre_w x' / rms(x'), their gradients, and bounds of what FP32 may miss.

Bounds, with r = 2^-24: a mean of D squares or products is added up in at most D / 32 + 10 steps a lane and log steps more,
off by n r of its absolute terms, n = D / 32 + 20; 1 / rms is off by half of that and 2^-22. sigmoid(g) is off by
2^-20 (1 + |g| / 4).
"""
from __future__ import annotations

import numpy as np

R = 2.0 ** -24


def _rr(z, eps):
    return 1.0 / np.sqrt((z * z).mean(-1, keepdims=True) + eps)


def _sig(g):
    return (1.0, 0.0) if g is None else (1.0 / (1.0 + np.exp(-g)), 2.0 ** -20 * (1 + np.abs(g) / 4))


def forward(x, y, g, post_w, scale, pre_w, eps=1e-6):
    """x' and h [M, D] with x1_err and h_err; y None: x' = x."""
    n = (x.shape[1] / 32 + 20) * R + 2.0 ** -21
    x1, e1 = x, np.zeros_like(x)
    if y is not None:
        s, ds = _sig(g)
        t = scale * s * post_w * y * _rr(y, eps)
        x1 = x + t
        e1 = np.abs(t) * (n + ds) + R * np.abs(x1)
    rx = _rr(x1, eps)
    h = pre_w * x1 * rx
    # x1's own errors move its norm by no more than their root mean square
    return dict(x1=x1, x1_err=e1, h=h, h_err=np.abs(pre_w) * rx * (e1 + np.abs(x1) * rx * np.sqrt((e1 * e1).mean(-1, keepdims=True))) + np.abs(h) * n)


def backward(x1, y, g, post_w, scale, pre_w, dh, dx1, eps=1e-6):
    """Gradients of sum(x' dx1) + sum(h dh), x1 the rows of x' as given, each with its bound."""
    M, D = x1.shape
    n = (D / 32 + 20) * R + 2.0 ** -21
    dx, ex, r = np.zeros((M, D)) if dx1 is None else dx1.copy(), np.zeros((M, D)), {}
    ex += R * np.abs(dx)
    dpre, epre = np.zeros(D), np.zeros(D)
    if dh is not None:
        rx = _rr(x1, eps)
        nx, w = x1 * rx, dh * pre_w
        dx = dx + rx * (w - nx * (w * nx).mean(-1, keepdims=True))
        ex = R * np.abs(dx) + rx * (np.abs(w) * n + 4 * n * np.abs(nx) * np.abs(w * nx).mean(-1, keepdims=True)) + ex
        dpre, epre = (dh * nx).sum(0), np.abs(dh * nx).sum(0) * (n + M * R)
    r |= dict(dx=dx, dx_err=ex, dpre_w=dpre, dpre_w_err=epre)
    if y is not None:
        s, ds = _sig(g)
        ry = _rr(y, eps)
        ny, k = y * ry, scale * post_w * s
        w = dx * k
        ew = np.abs(k) * ex + np.abs(w) * (ds + 4 * R)
        mean, am = (w * ny).mean(-1, keepdims=True), np.abs(w * ny).mean(-1, keepdims=True)
        r["dy"] = ry * (w - ny * mean)
        r["dy_err"] = ry * (ew + np.abs(w) * n + np.abs(ny) * ((ew * np.abs(ny)).mean(-1, keepdims=True) + 4 * n * am))
        if g is not None:
            r["dg"] = w * ny * (1 - s)
            r["dg_err"] = (np.abs(ny) * ew + np.abs(w * ny) * (n + 2 * ds)) * (1 - s)
        q = dx * s * ny
        eq = (np.abs(s * ny) * ex + np.abs(q) * (n + ds)).sum(0) + M * R * np.abs(q).sum(0)
        q = q.sum(0)
        r |= dict(dpost_w=q * scale, dpost_w_err=eq * np.abs(scale), dscale=q * post_w, dscale_err=eq * np.abs(post_w))
    return r
