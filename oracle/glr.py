"""The gated linear recurrence, one token at a time in FP64 (numpy), its gradients, and bounds of what FP32 may miss.

Per channel: gk = -exp(A_log) sigmoid(a + a_bias), alpha = exp(gk), beta = sigmoid(b + b_bias), m = sqrt(1 - alpha^2),
    h = alpha h + u, u = m beta x,   out = h or h silu(g)

Bounds, with r = 2^-24 (half a step of FP32). A gate's argument is off by 3 r of |a| + |a_bias| (two products with log2 e and
a sum), the exponential by 2^-22, sum, reciprocal, product and exp(A_log) by 2^-21 together: gk and beta by
    d = 2^-20 (1 + (|a| + |a_bias| + |b| + |b_bias|) / 4)   relative,
alpha - 1 = e by no more than that (exp(x) - 1 has a condition number <= 1 for x <= 0) and its own evaluation: a polynomial to 2^-22
above x = -1/4, below it an exponential, off by 2^-22 of itself, less 1, a difference of at least 0.22: 2^-22 0.78 / 0.22 + 2^-24
< 2^-20. m = sqrt(-e (2 + e)) is off by as much and 2^-21, u by 3 (d + 2^-20) with beta and the products.
A step h + (e h + u) rounds twice, and splitting the tokens into parts and joining the parts (h = A h + H, A a product of
alphas) rounds A and the sum, each at most as often as there are tokens: 8 r of M = alpha M + |u|, M of absolute values, is
more than all of it. So
    E = alpha E + q |e| M_before + 3 q |u| + 8 r (M_before + |u|),  q = d + 2^-20.
A sigmoid below 2^-126, FP32's smallest normal number, counts as 0. Where that of a does, gk is off by up to exp(A_log) 2^-126,
and m = sqrt(1 - exp(2 gk)) <= sqrt(2 |gk|) by up to f = sqrt(2 exp(A_log)) 2^-63, u by f beta |x|, and gk / m = sqrt(|gk| / 2) in
the gradients by no more than f; where beta does, u is off by m |x| 2^-126, dx by as much for each lam.
"""
from __future__ import annotations

import numpy as np

R = 2.0 ** -24


def sigmoid(x):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-x))


def gates(x, a, b, A_log, a_bias, b_bias):
    sa, beta = sigmoid(a + a_bias), sigmoid(b + b_bias)
    gk = -np.exp(A_log) * sa
    e = np.expm1(gk)
    m = np.sqrt(-e * (2.0 + e))
    d = 2.0 ** -20 * (1 + (np.abs(a) + np.abs(a_bias) + np.abs(b) + np.abs(b_bias)) / 4)
    f = np.where(sa < 2.0 ** -126, np.sqrt(2 * np.exp(A_log)) * 2.0 ** -63, 0.0)
    return sa, beta, gk, e, m, np.where(np.isfinite(d), d, 2.0 ** -20), f * beta + np.where(beta < 2.0 ** -126, m * 2.0 ** -126, 0.0)


def glr(x, a, b, g, A_log, a_bias, b_bias, h0):
    """One sequence: rows [T, D] (g None: no gate), h0 [D] -> dict of out, S, their bounds out_err, S_err, and what grad needs."""
    x, a, b, A_log, a_bias, b_bias, h0 = (np.asarray(v, dtype=np.float64) for v in (x, a, b, A_log, a_bias, b_bias, h0))
    T, D = x.shape
    sa, beta, gk, e, m, d, lost = gates(x, a, b, A_log, a_bias, b_bias)
    with np.errstate(invalid="ignore"):
        u = m * beta * x
    h, M, E, q = h0.copy(), np.abs(h0), np.zeros(D), d + 2.0 ** -20
    before, hs, Es = np.empty((T, D)), np.empty((T, D)), np.empty((T + 1, D))
    Es[0] = 0
    for t in range(T):
        before[t] = h
        E = (1 + e[t]) * E + q[t] * np.abs(e[t]) * M + 3 * q[t] * np.abs(u[t]) + 8 * R * (M + np.abs(u[t])) + lost[t] * np.abs(x[t])
        M = (1 + e[t]) * M + np.abs(u[t])
        h = (1 + e[t]) * h + u[t]
        hs[t], Es[t + 1] = h, E
    out, out_err = hs, Es[1:]
    if g is not None:
        g = np.asarray(g, dtype=np.float64)
        s = sigmoid(g) * g
        out, out_err = hs * s, Es[1:] * np.abs(s) + np.abs(hs * s) * 2.0 ** -20 * (1 + np.abs(g) / 4)
    return dict(out=out, out_err=out_err, S=h, S_err=E, h=hs, before=before, E=Es)


def grad(x, a, b, g, A_log, a_bias, b_bias, h0, dout, dS):
    """Gradients of sum(out dout) + sum(S dS), each with its bound (name + "_err"); the bounds follow the formulas with the
    absolute values of their terms. alpha = 1 + e is off by p = alpha (|gk| d + 2^-21) + 2 r, which where alpha is small is no small part of it: d gk
has alpha (h gk - alpha w0), off by p |h gk| + (2 alpha p + p^2) |w0|. A sum over T tokens is off by T r of its absolute terms."""
    x, a, b, A_log, a_bias, b_bias, h0, dout, dS = (np.asarray(v, dtype=np.float64) for v in (x, a, b, A_log, a_bias, b_bias, h0, dout, dS))
    f = glr(x, a, b, g, A_log, a_bias, b_bias, h0)
    T, D = x.shape
    sa, beta, gk, e, m, d, lost = gates(x, a, b, A_log, a_bias, b_bias)
    al, na, nb = 1 + e, sigmoid(-(a + a_bias)), sigmoid(-(b + b_bias))  # nb = 1 - beta without the difference
    dh, dh_err, r = dout, np.zeros((T, D)), {}
    if g is not None:
        g = np.asarray(g, dtype=np.float64)
        s, ns, dg_ = sigmoid(g), sigmoid(-g), 2.0 ** -19 * (1 + np.abs(g) / 4)
        slope = s * (1 + g * ns)
        r["dg"] = dout * f["h"] * slope
        r["dg_err"] = np.abs(dout) * (np.abs(slope) * f["E"][1:] + np.abs(f["h"]) * s * (1 + np.abs(g) * ns) * dg_)
        dh = dout * g * s
        dh_err = np.abs(dh) * dg_
    c, L, E = dS.copy(), np.abs(dS), np.zeros(D)
    lam, lamM, lamE = np.empty((T, D)), np.empty((T, D)), np.empty((T, D))
    for t in range(T - 1, -1, -1):
        lam[t], lamM[t] = dh[t] + c, np.abs(dh[t]) + L
        lamE[t] = E + dh_err[t] + 8 * R * lamM[t]
        c, L = al[t] * lam[t], al[t] * lamM[t]
        E = al[t] * lamE[t] + (d[t] + 2.0 ** -20) * np.abs(e[t]) * lamM[t] + 8 * R * lamM[t]
    r["dS"], r["dS_err"] = c, E
    r["dx"] = lam * m * beta
    r["dx_err"] = lamE * m * beta + (4 * (d + 2.0 ** -20) * m * beta + lost) * lamM
    r["db"] = lam * m * beta * x * nb
    r["db_err"] = np.abs(x) * nb * r["dx_err"] + 3 * d * np.abs(x * nb * lamM * m * beta)
    with np.errstate(divide="ignore", invalid="ignore"):
        w0 = beta * x * np.where(gk < 0, gk / m, 0.0)
    w = w0 * al
    mag = np.abs(f["before"] * gk) + np.abs(w)
    dA = lam * al * (f["before"] * gk - w)
    al_err = al * (np.abs(gk) * d + 2.0 ** -21) + 2 * R
    gk_lost = np.where(sa < 2.0 ** -126, np.exp(A_log) * 2.0 ** -126, 0.0)
    dA_err = lamE * al * mag + lamM * (al * (f["E"][:-1] * np.abs(gk) + 6 * (d + 2.0 ** -20) * mag + lost * np.abs(x) + gk_lost * np.abs(f["before"])) + 2 * al_err * mag + al_err ** 2 * np.abs(w0))
    r["da"], r["da_err"] = dA * na, (dA_err + 2 * d * np.abs(lamM * al * mag)) * na
    for name, v, err, mags in (("dA_log", dA, dA_err, lamM * al * mag), ("da_bias", r["da"], r["da_err"], lamM * al * mag * na),
                               ("db_bias", r["db"], r["db_err"], np.abs(x * nb * lamM * m * beta))):
        r[name], r[name + "_err"] = v.sum(0), err.sum(0) + T * R * mags.sum(0)
    return f | r
