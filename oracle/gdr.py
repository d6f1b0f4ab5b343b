"""The gated delta rule, one token at a time in FP64 (numpy).

Per value head h with key head h // (H / Hk) and state S[key][value]:
    alpha = exp(-exp(A_log) softplus(a + dt_bias)),  beta = sigmoid(b)
    S = alpha S;  u = beta (v - S^T k^);  S = S + k^ u^T;  o = S^T q^
with k^, q^ normalised (q^ scaled) or as given. Beside the results it returns
    mag = |q^| . M,   M = alpha M + |k^| |u|   (the same sums with every term's absolute value)
    E = alpha E + beta (|v| + |k^| . alpha M)  (per value column; E starts at 0)
which error bounds are stated in: mag for the output. For the state: an error eps (|v| + |k^| . M) made in
one u enters S along k^, |k^| <= 1, and the later steps alpha (I - beta k^ k^T) never lengthen it, so column
v of S is off by at most eps (E_v + |M_v|) in the 2-norm.
"""
from __future__ import annotations

import numpy as np


def softplus(x):
    return np.maximum(x, 0.0) + np.log1p(np.exp(-np.abs(x)))


def gdr(q, k, v, a, b, A_log, dt_bias, S0, l2norm=True, l2_eps=1e-6, q_scale=128 ** -0.5):
    """One sequence: q, k [T, Hk, d], v [T, H, d], a, b [T, H], S0 [H, d, d] -> o [T, H, d], S, mag, E + |M| [H, d]."""
    q, k, v, a, b, A_log, dt_bias, S0 = (np.asarray(x, dtype=np.float64) for x in (q, k, v, a, b, A_log, dt_bias, S0))
    T, H, d = v.shape
    G = H // q.shape[1]
    if l2norm:
        q = q / np.sqrt((q * q).sum(-1, keepdims=True) + l2_eps)
        k = k / np.sqrt((k * k).sum(-1, keepdims=True) + l2_eps)
    q = np.repeat(q * q_scale, G, axis=1)
    k = np.repeat(k, G, axis=1)
    with np.errstate(over="ignore"):
        alpha = np.exp(-np.exp(A_log) * softplus(a + dt_bias))
        beta = 1.0 / (1.0 + np.exp(-b))
    S, M, E = S0.copy(), np.abs(S0), np.zeros((H, d))
    o, mag = np.empty((T, H, d)), np.empty((T, H, d))
    for t in range(T):
        S = S * alpha[t][:, None, None]
        u = beta[t][:, None] * (v[t] - np.einsum("hk,hkv->hv", k[t], S))
        S = S + k[t][:, :, None] * u[:, None, :]
        E = E * alpha[t][:, None] + beta[t][:, None] * (
            np.abs(v[t]) + np.einsum("hk,hkv->hv", np.abs(k[t]), M) * alpha[t][:, None])
        M = M * alpha[t][:, None, None] + np.abs(k[t])[:, :, None] * np.abs(u)[:, None, :]
        o[t] = np.einsum("hk,hkv->hv", q[t], S)
        mag[t] = np.einsum("hk,hkv->hv", np.abs(q[t]), M)
    return o, S, mag, E + np.sqrt((M * M).sum(1))
