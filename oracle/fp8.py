"""E4M3 operands with a power-of-two scale per block of 128 columns, and their product, in FP64 (numpy)."""
from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0


def e4m3(x):
    """x (FP64) rounded to the nearest E4M3 number, ties to even, |x| <= 448; NaN and infinity give NaN."""
    x = np.asarray(x, dtype=np.float64)
    ok = np.isfinite(x)
    z = np.where(ok, x, 0.0)
    _, p = np.frexp(z)                       # |z| in [2^(p-1), 2^p)
    step = np.ldexp(1.0, np.maximum(p - 4, -9))  # 4 significant bits, the smallest step 2^-9
    return np.where(ok, np.rint(z / step) * step, np.nan)


def quantise(x, rows):
    """(values of q, s) of x [M, K]: one scale for each rows x 128 block."""
    x = np.asarray(x, dtype=np.float64)
    M, K = x.shape
    nm, nk = -(-M // rows), -(-K // 128)
    q, s = np.empty((M, K)), np.ones((nm, nk))
    for i in range(nm):
        for j in range(nk):
            b = x[i * rows:(i + 1) * rows, j * 128:(j + 1) * 128]
            f = np.abs(b[np.isfinite(b)])
            if f.size and f.max() > 0:
                e = -126
                while f.max() > E4M3_MAX * 2.0 ** e:
                    e += 1
                s[i, j] = 2.0 ** e
            q[i * rows:(i + 1) * rows, j * 128:(j + 1) * 128] = e4m3(b / s[i, j])
    return q, s


def whole(q, s, rows):
    """The matrix that q and s stand for."""
    M, K = q.shape
    return np.asarray(q, np.float64) * np.repeat(np.repeat(np.asarray(s, np.float64), rows, 0)[:M], 128, 1)[:, :K]


def linear(xq, xs, wq, ws, r=None):
    """y and the sums of absolute terms."""
    x, w = whole(xq, xs, 1), whole(wq, ws, 128)
    y = x @ w.T
    return (y if r is None else y + np.asarray(r, np.float64)), np.abs(x) @ np.abs(w).T + (0 if r is None else np.abs(r))
