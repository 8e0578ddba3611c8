"""fp64 oracle of the operators around the expert layer: the router's balance loss, layer norm,
gradient clipping and the block-128 FP8 formats and product.

TEST INFRASTRUCTURE ONLY (see the package docstring). Plain definitions, one line of mathematics
a line of code; nothing here is shared with the CUDA path.
"""
from __future__ import annotations

import math

import numpy as np

FP8_MAX = np.float32(448.0)
FP8_TINY = np.float32(2.0 ** -100)
CLIP_EPS = 1e-6


# ------------------------------------------------------------------ router
def softmax(logits: np.ndarray) -> np.ndarray:
    """Row softmax; NaN reads as -inf, a value equal to the row's maximum weighs 1."""
    x = np.where(np.isnan(logits), -np.inf, logits.astype(np.float64))
    m = x.max(axis=1, keepdims=True)
    with np.errstate(invalid="ignore"):
        w = np.where(x == m, 1.0, np.exp(x - m))
    return w / w.sum(axis=1, keepdims=True)


def router_loss(logits, ids, coef, mask=None):
    """(loss, counts, mean_prob, f, n) of logits [T, E] and ids [T, k]."""
    T, E = logits.shape
    k = ids.shape[1]
    m = np.ones(T, bool) if mask is None else mask.astype(bool)
    n = int(m.sum())
    counts = np.zeros(E, np.int64)
    for t in np.flatnonzero(m):
        for e in ids[t]:
            if 0 <= e < E:
                counts[e] += 1
    if n == 0:
        return 0.0, counts, np.zeros(E), np.zeros(E), 0
    mean_prob = softmax(logits)[m].sum(axis=0) / n
    f = counts * E / (k * n)
    return coef * float(f @ mean_prob), counts, mean_prob, f, n


def router_grad(logits, ids, coef, mask=None, d_loss=1.0, probs=None, d_probs=None):
    """d_logits and, elementwise, the magnitude of the terms it is a sum of."""
    T, E = logits.shape
    _, _, _, f, n = router_loss(logits, ids, coef, mask)
    p = softmax(logits)
    m = np.ones(T) if mask is None else mask.astype(np.float64)
    c = (d_loss * coef / n if n else 0.0) * m[:, None]
    s = p @ f
    d = c * p * (f[None, :] - s[:, None])
    size = np.abs(c) * p * (np.abs(f)[None, :] + np.abs(s)[:, None])
    if probs is not None:
        w, g = probs.astype(np.float64), d_probs.astype(np.float64)
        live = (ids >= 0) & (ids < E)
        dot = (w * g * live).sum(axis=1)
        adot = (np.abs(w * g) * live).sum(axis=1)
        for t in range(T):
            for j, e in enumerate(ids[t]):
                if live[t, j]:
                    d[t, e] += w[t, j] * (g[t, j] - dot[t])
                    size[t, e] += abs(w[t, j]) * (abs(g[t, j]) + adot[t])
    return d, size


# ------------------------------------------------------------------ layer norm
def layernorm(x, gamma, beta, eps):
    x = x.astype(np.float64)
    mean = x.mean(axis=1)
    rstd = 1.0 / np.sqrt(((x - mean[:, None]) ** 2).mean(axis=1) + eps)
    h = (x - mean[:, None]) * rstd[:, None]
    return h * (1.0 if gamma is None else gamma) + (0.0 if beta is None else beta), mean, rstd


def layernorm_grad(dy, x, gamma, mean, rstd):
    """(dx, dgamma, dbeta, sum |dy h|, sum |dy|) from the given statistics."""
    dy = dy.astype(np.float64)
    h = (x.astype(np.float64) - mean[:, None]) * rstd[:, None]
    u = dy * (1.0 if gamma is None else gamma)
    dx = rstd[:, None] * (u - u.mean(axis=1, keepdims=True)
                          - h * (u * h).mean(axis=1, keepdims=True))
    return (dx, (dy * h).sum(axis=0), dy.sum(axis=0), np.abs(dy * h).sum(axis=0),
            np.abs(dy).sum(axis=0))


# ------------------------------------------------------------------ clipping
def clip(grads, max_norm):
    """(norm, factor) of a list of arrays."""
    norm = math.sqrt(sum(float((g.astype(np.float64) ** 2).sum()) for g in grads))
    return norm, min(1.0, max_norm / (norm + CLIP_EPS))


# ------------------------------------------------------------------ block-128 E4M3
def e4m3_nearest(v: np.ndarray) -> np.ndarray:
    """Nearest E4M3 value (ties to even mantissas), at most 448 in magnitude."""
    a = np.abs(np.asarray(v, np.float64))
    _, e = np.frexp(a)
    step = np.ldexp(1.0, np.maximum(e, -5) - 4)
    return np.sign(v) * np.minimum(np.round(a / step) * step, 448.0)


def e4m3_values(codes: np.ndarray) -> np.ndarray:
    """Values of E4M3 bytes (sign, 4 exponent bits with bias 7, 3 mantissa bits; 0x7F is NaN)."""
    c = codes.astype(np.int64)
    ex, man = (c >> 3) & 15, c & 7
    v = np.where(ex == 0, man * 2.0 ** -9, (8 + man) * 2.0 ** (ex - 10.0))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c & 128, -v, v)


def _factors(amax):
    a = np.maximum(amax.astype(np.float32), FP8_TINY)
    return a / FP8_MAX, FP8_MAX / a


def quantize_rows(x: np.ndarray):
    """Blocks of 1 x 128 of fp32 x [M, N]: (E4M3 values [M, N], scales [ceil(N/128), M])."""
    M, N = x.shape
    q = np.empty((M, N))
    s = np.empty((-(-N // 128), M), np.float32)
    for b in range(s.shape[0]):
        blk = x[:, 128 * b:128 * b + 128].astype(np.float32)
        s[b], f = _factors(np.abs(blk).max(axis=1))
        q[:, 128 * b:128 * b + 128] = e4m3_nearest(blk * f[:, None])
    return q, s


def quantize_weight(w: np.ndarray):
    """Blocks of 128 x 128 of fp32 w [N, K]: (values [N, K], scales [ceil(N/128), ceil(K/128)])."""
    N, K = w.shape
    q = np.empty((N, K))
    s = np.empty((-(-N // 128), -(-K // 128)), np.float32)
    for i in range(s.shape[0]):
        for j in range(s.shape[1]):
            at = (slice(128 * i, 128 * i + 128), slice(128 * j, 128 * j + 128))
            blk = w[at].astype(np.float32)
            s[i, j], f = _factors(np.abs(blk).max(keepdims=True).reshape(()))
            q[at] = e4m3_nearest(blk * f)
    return q, s


def rows_scaled(q, s):
    """Values of 1 x 128 blocks: q [M, K], s [ceil(K/128), M]."""
    return q * np.repeat(s.astype(np.float64), 128, axis=0)[:q.shape[1]].T


def blocks_scaled(q, s):
    """Values of 128 x 128 blocks: q [N, K], s [ceil(N/128), ceil(K/128)]."""
    full = np.repeat(np.repeat(s.astype(np.float64), 128, axis=0), 128, axis=1)
    return q * full[:q.shape[0], :q.shape[1]]
