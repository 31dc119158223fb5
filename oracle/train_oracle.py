"""The training-step operators in plain numpy float64, written from their formulas: RMS norm with the residual's addition
and its gradient, 8-bit codes of rows, the 8-bit product, and the distillation loss on a teacher's top logits with its
gradient.  Used by the tests only.
"""
from __future__ import annotations

import numpy as np


def rmsnorm(s, w, eps):
    """y and rstd of the rows of s (the sum of the input and its residual)."""
    s, w = np.asarray(s, np.float64), np.asarray(w, np.float64)
    rstd = 1.0 / np.sqrt((s * s).mean(1) + eps)
    return s * rstd[:, None] * w, rstd


def rmsnorm_backward(dy, h, w, eps, dh=None):
    """Gradients of sum(y * dy) + sum(h * dh) with respect to h and w."""
    dy, h, w = (np.asarray(v, np.float64) for v in (dy, h, w))
    rstd = 1.0 / np.sqrt((h * h).mean(1, keepdims=True) + eps)
    g = dy * w
    dx = rstd * g - h * rstd ** 3 * (g * h).mean(1, keepdims=True)
    if dh is not None:
        dx = dx + np.asarray(dh, np.float64)
    return dx, (dy * h * rstd).sum(0)


def int8_linear(a, sa, b, sb, bias=None):
    """The product with its scales; the integer sum is exact in float64."""
    y = np.asarray(a, np.float64) @ np.asarray(b, np.float64).T
    y = y * np.asarray(sa, np.float64)[:, None] * np.asarray(sb, np.float64)
    return y if bias is None else y + np.asarray(bias, np.float64)


def distill(z, t, idx, temp):
    """loss, dloss/dz (for a gradient of one) and the live rows, row by row."""
    z, t = np.asarray(z, np.float64), np.asarray(t, np.float64)
    rows, vocab = z.shape
    loss, dz, live = np.zeros(rows), np.zeros((rows, vocab)), np.zeros(rows, bool)
    for r in range(rows):
        here = [(int(i), v) for i, v in zip(idx[r], t[r]) if 0 <= i < vocab and v != -np.inf]
        if not here:
            continue
        live[r] = True
        ii = np.array([i for i, _ in here])
        tt = np.array([v for _, v in here])
        p = np.exp((tt - tt.max()) / temp)
        p /= p.sum()
        u = (z[r] - z[r].max()) / temp
        logq = u - np.log(np.exp(u).sum())
        some = p > 0
        loss[r] = temp ** 2 * (p[some] * (np.log(p[some]) - logq[ii][some])).sum()
        dz[r] = temp * np.exp(logq)
        np.subtract.at(dz[r], ii, temp * p)
    return loss, dz, live
