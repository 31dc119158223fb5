"""Layer norm with the residual's addition and its gradient, microscaled 4-bit floating point, and log probabilities with
entropy, top alternatives and gradient, in plain numpy float64, written from their formulas.  Used by the tests only.
"""
from __future__ import annotations

import numpy as np

GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])   # the values of codes 0 .. 7


def layernorm(s, w, b, eps):
    """y, mean and rstd of the rows of s (the sum of the input and its residual)."""
    s, w = np.asarray(s, np.float64), np.asarray(w, np.float64)
    mean = s.mean(1)
    d = s - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).mean(1) + eps)
    y = d * rstd[:, None] * w
    return (y if b is None else y + np.asarray(b, np.float64)), mean, rstd


def layernorm_backward(dy, h, w, mean, rstd, dh=None):
    """Gradients of sum(y * dy) + sum(h * dh) with respect to h, w and b, at the given mean and rstd."""
    dy, h, w = (np.asarray(v, np.float64) for v in (dy, h, w))
    u = (h - np.asarray(mean, np.float64)[:, None]) * np.asarray(rstd, np.float64)[:, None]
    g = dy * w
    dx = (g - g.mean(1, keepdims=True) - u * (g * u).mean(1, keepdims=True)) * np.asarray(rstd, np.float64)[:, None]
    if dh is not None:
        dx = dx + np.asarray(dh, np.float64)
    return dx, (dy * u).sum(0), dy.sum(0)


def mx_codes(x):
    """Codes (one an element) and scale bytes of the rows of x, block by block."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    x = np.concatenate([x, np.zeros((rows, -cols % 32))], 1).reshape(rows, (cols + 31) // 32, 32)
    top = np.abs(x).max(2)
    bad = ~np.isfinite(top)
    e = np.full(top.shape, -127)
    for k in range(-126, 127):   # the least exponent whose 7 2^e lies above
        e = np.where((e == k - 1) & ~(top < 7 * 2.0 ** (k - 1)), k, e)
    a = np.abs(np.where(bad[:, :, None], 0, x)) / 2.0 ** e.astype(np.float64)[:, :, None]
    code = np.zeros(a.shape, np.uint8)
    far = a.copy()
    for i in range(1, 8):   # the nearest; of two equally near ones the even code
        d = np.abs(a - GRID[i])
        nearer = d < far if i % 2 else d <= far
        code, far = np.where(nearer, i, code), np.where(nearer, d, far)
    code = code + 8 * (np.signbit(x) & ~bad[:, :, None])
    return code.astype(np.uint8).reshape(rows, (cols + 31) // 32 * 32)[:, :cols], np.where(bad, 255, e + 127).astype(np.uint8)


def mx_pack(code):
    """Two codes a byte, the even element in the low half."""
    if code.shape[1] % 2:
        code = np.concatenate([code, np.zeros((code.shape[0], 1), np.uint8)], 1)
    return code[:, ::2] | (code[:, 1::2] << 4)


def mx_values(q, scale, cols):
    """The values that packed codes stand for."""
    code = np.stack([q & 15, q >> 4], 2).reshape(q.shape[0], 2 * q.shape[1])[:, :cols]
    v = GRID[code & 7] * np.where(code & 8, -1.0, 1.0)
    s = np.where(scale == 255, np.nan, 2.0 ** (scale.astype(np.float64) - 127))
    return v * np.repeat(s, 32, 1)[:, :cols]


def logprobs(z, tokens, temp):
    """logprob (0 for tokens outside), entropy, and the row's log q and q."""
    z = np.asarray(z, np.float64)
    rows, vocab = z.shape
    with np.errstate(all="ignore"):
        m = z.max(1, keepdims=True)
        u = (z - m) / temp
        e = np.exp(u)
        s = e.sum(1, keepdims=True)
        q, logq = e / s, u - np.log(s)
        none = np.isneginf(m)
        q, logq = np.where(none, 0, q), np.where(none, -np.inf, logq)
        entropy = -np.where(q == 0, 0, q * logq).sum(1)
    inside = (tokens >= 0) & (tokens < vocab)
    lp = np.where(inside, logq[np.arange(rows), np.where(inside, tokens, 0)], 0)
    return lp, entropy, logq, q


def top(z, k):
    """Indices of the k largest logits of each row, equal ones by their index; -1 where no logit above -inf is left."""
    z = np.asarray(z, np.float64)
    out = np.full((z.shape[0], k), -1, np.int64)
    for r, row in enumerate(z):
        here = np.flatnonzero(row > -np.inf)
        here = here[np.argsort(-row[here], kind="stable")][:k]
        out[r, :len(here)] = here
    return out


def logprobs_backward(gl, ge, z, tokens, temp):
    """Gradient of sum(gl logprob) + sum(ge entropy)."""
    _, entropy, logq, q = logprobs(z, tokens, temp)
    rows, vocab = q.shape
    inside = (tokens >= 0) & (tokens < vocab)
    g = np.where(inside, gl, 0)[:, None]
    with np.errstate(all="ignore"):
        d = -q * g - np.where(q == 0, 0, q * (logq + entropy[:, None])) * np.asarray(ge)[:, None]
    r = np.flatnonzero(inside & ~np.isneginf(np.asarray(z, np.float64).max(1)))
    d[r, tokens[r]] += np.asarray(gl)[r]
    return d / temp
