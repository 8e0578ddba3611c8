"""fp64 oracle of the operators of a block's step: the choice of experts, the norms around the
residual stream, and AdamW with 32- and 8-bit states.

TEST INFRASTRUCTURE ONLY (see the package docstring). Plain definitions, one line of mathematics
a line of code; nothing here is shared with the CUDA path.
"""
from __future__ import annotations

import math

import numpy as np

WEIGHT_EPS = 1e-20
CLIP_EPS = 1e-6
BLOCK = 256
f32 = np.float32


# ------------------------------------------------------------------ choice of experts
def sigmoid(x):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-x))


def softmax(x):
    """Row softmax; a value equal to the row's maximum weighs 1 before normalisation."""
    m = x.max(axis=-1, keepdims=True)
    with np.errstate(invalid="ignore"):
        w = np.where(x == m, 1.0, np.exp(x - m))
    return w / w.sum(axis=-1, keepdims=True)


def order(values, first, last):
    """Indices by descending value, ties to the lower index; the smallest difference, equal values
    aside, of the neighbours in that order at places first, first + 1 to last, last + 1: those whose
    comparison decides which are taken (and, from place 0 on, in which order)."""
    at = np.argsort(-values, kind="stable")
    with np.errstate(invalid="ignore"):
        d = -np.diff(values[at])[first:last + 1]
    d = d[d > 0]
    return at, d.min() if d.size else math.inf


def route(logits, k, score, bias=None, mask=None, groups=1, of_groups=1, group_top=1, renorm=True,
          scale=1.0):
    """(ids [T, k], weights [T, k], margin [T]): margin is how near the closest two values that
    decided a choice were (equal ones aside), in fp64."""
    x = np.where(np.isnan(logits), -np.inf, logits.astype(np.float64))
    T, E = x.shape
    s = sigmoid(x) if score == "sigmoid" else softmax(x)
    value = s
    if bias is not None:
        value = s + bias.astype(np.float64)
        value = np.where(np.isnan(value), -np.inf, value)
    choice = x if bias is None else value
    ids, w, margin = np.full((T, k), -1), np.zeros((T, k)), np.full(T, math.inf)
    for t in range(T):
        if mask is not None and not mask[t]:
            continue
        open_ = np.arange(E)
        if groups > 1:
            size = E // groups
            if group_top == 1:
                g = choice[t].reshape(groups, size).max(axis=1)
            else:
                g = np.sort(value[t].reshape(groups, size), axis=1)[:, -2:].sum(axis=1)
            at, margin[t] = order(g, of_groups - 1, of_groups - 1)
            open_ = np.flatnonzero(np.isin(np.arange(E) // size, at[:of_groups]))
        at, near = order(choice[t][open_], 0, k - 1)
        margin[t] = min(margin[t], near)
        ids[t] = open_[at[:k]]
        w[t] = s[t, ids[t]]
        if renorm and score == "sigmoid":
            w[t] /= w[t].sum() + WEIGHT_EPS
        elif renorm:
            w[t] = softmax(x[t, ids[t]])
    return ids, w * scale, margin


def route_weights(logits, ids, score, renorm, scale):
    """The weights as a function of the logits, for given ids (outside [0, E): 0)."""
    x = logits.astype(np.float64)
    T, E = x.shape
    on = (ids >= 0) & (ids < E)
    at = np.where(on, ids, 0)
    w = np.zeros(ids.shape)
    for t in range(T):
        c = np.flatnonzero(on[t])
        if score == "sigmoid":
            w[t, c] = sigmoid(x[t, at[t, c]])
            if renorm:
                w[t] /= w[t].sum() + WEIGHT_EPS
        elif not renorm:
            w[t, c] = softmax(x[t])[at[t, c]]
        elif c.size:
            w[t, c] = softmax(x[t, at[t, c]])
    return w * scale


def route_grad(logits, ids, d_weights, score, renorm, scale):
    """d_logits and, elementwise, the magnitude of the terms it is a sum of."""
    x = logits.astype(np.float64)
    T, E = x.shape
    d, mag = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        c = np.flatnonzero((ids[t] >= 0) & (ids[t] < E))
        e = ids[t, c]
        u = scale * d_weights[t, c].astype(np.float64)
        if score == "sigmoid":
            s = sigmoid(x[t, e])
            slope = s * sigmoid(-x[t, e])
            if renorm:
                S = s.sum() + WEIGHT_EPS
                part, size = (u - (u * s).sum() / S) / S, (abs(u) + (abs(u) * s).sum() / S) / S
            else:
                part, size = u, abs(u)
            np.add.at(d[t], e, part * slope)
            np.add.at(mag[t], e, size * slope)
        elif renorm:
            if c.size:
                w = softmax(x[t, e])
                np.add.at(d[t], e, w * (u - (w * u).sum()))
                np.add.at(mag[t], e, w * (abs(u) + (w * abs(u)).sum()))
        else:
            p, ue, ua = softmax(x[t]), np.zeros(E), np.zeros(E)
            np.add.at(ue, e, u)
            np.add.at(ua, e, abs(u))
            d[t] = p * (ue - (p * ue).sum())
            mag[t] = p * (ua + (p * ua).sum())
    return d, mag


# ------------------------------------------------------------------ residual norm
def rms(a, eps):
    return 1.0 / np.sqrt((a * a).mean(axis=1, keepdims=True) + eps)


def residual(x, o, wp, gate, scale, post, eps):
    """x_new in fp64."""
    z = o * rms(o, eps) if post else o
    q = scale * (np.ones(len(x)) if gate is None else gate)
    return x + q[:, None] * z * (1.0 if wp is None else wp)


def normed(x_new, w, eps):
    return x_new * rms(x_new, eps) * (1.0 if w is None else w)


def residual_grad(dh, dx_new, x_new, o, wp, gate, w, scale, post, eps):
    """{name: (gradient, magnitude of its terms)} for dx, do, d_weight, d_post_weight, d_gate."""
    M, N = (dx_new if dh is None else dh).shape
    dx = np.zeros((M, N)) if dx_new is None else dx_new.copy()
    size = abs(dx)
    out = {}
    if dh is not None:
        r = rms(x_new, eps)
        y, u = x_new * r, dh * (1.0 if w is None else w)
        dx += r * (u - y * (u * y).mean(axis=1, keepdims=True))
        size += r * (abs(u) + abs(y) * abs(u * y).mean(axis=1, keepdims=True))
        out["d_weight"] = (dh * y).sum(axis=0), abs(dh * y).sum(axis=0)
    out["dx"] = dx, size
    if o is not None:
        rp = rms(o, eps) if post else np.ones((M, 1))
        z, v = o * rp, 1.0 if wp is None else wp
        q = scale * (np.ones((M, 1)) if gate is None else gate[:, None])
        e, es = dx * v, size * abs(v)
        dot, ds = (e * z).sum(axis=1, keepdims=True), (es * abs(z)).sum(axis=1, keepdims=True)
        out["d_gate"] = scale * dot[:, 0], abs(scale) * ds[:, 0]
        out["d_post_weight"] = (q * dx * z).sum(axis=0), (abs(q) * size * abs(z)).sum(axis=0)
        if post:
            out["do"] = q * rp * (e - z * dot / N), abs(q) * rp * (es + abs(z) * ds / N)
        else:
            out["do"] = q * e, abs(q) * es
    return out


# ------------------------------------------------------------------ AdamW
def mix(x):
    x = np.asarray(x, np.uint64) & np.uint64(0xFFFFFFFF)
    x = ((x ^ (x >> np.uint64(16))) * np.uint64(0xF75341D5)) & np.uint64(0xFFFFFFFF)
    x = ((x ^ (x >> np.uint64(15))) * np.uint64(0x99D5D0A1)) & np.uint64(0xFFFFFFFF)
    return x ^ (x >> np.uint64(16))


def words(seed, t, tensor, n, first=0):
    """The random words of a tensor's elements first .. first + n - 1 in step t."""
    key = mix(np.uint64(t) ^ mix(np.uint64(seed & 0xFFFFFFFF) ^ mix(seed >> 32)))
    key = mix(np.uint64(tensor) + key)
    e = np.arange(first, first + n, dtype=np.uint64)
    return mix(e ^ mix(key ^ (e >> np.uint64(32))))


def ladder(scale, signed):
    """The fp64 values of codes 0 .. 127 or 0 .. 255 under a scale byte."""
    top = 127 if signed else 255
    if scale == 255:
        return np.full(top + 1, np.nan)
    down = top - np.arange(top + 1)
    x = (1 + (7 - down % 8) / 8.0) * 2.0 ** (int(scale) - 127 - down // 8)
    x[0] = 0.0
    return x


def decode(codes, scales, signed):
    x = np.empty(len(codes))
    for b in range(len(scales)):
        part = slice(b * BLOCK, (b + 1) * BLOCK)
        c = codes[part].astype(int)
        v = ladder(scales[b], signed)[c & (127 if signed else 255)]
        x[part] = np.where(c > 127, -v, v) if signed else v
    return x


def encode(x, bits, signed):
    """(codes, scales) of fp32 values; bits: 16 random ones each. By the ladder of a scale's values
    and comparison: the scale is the smallest (from 32 on) whose largest value is not below a block's
    largest one rounded up."""
    codes, scales = np.zeros(len(x), np.uint8), np.zeros(-(-len(x) // BLOCK), np.uint8)
    for b in range(len(scales)):
        part = slice(b * BLOCK, (b + 1) * BLOCK)
        a, u = abs(x[part].astype(np.float64)), bits[part].astype(np.float64)
        if not np.isfinite(a).all():
            scales[b] = 255
            continue
        s = 32
        while s < 255 and a.max() > ladder(s, signed)[-1]:
            s += 1
        scales[b] = s
        if s == 255:
            continue
        v = ladder(s, signed)
        low = np.searchsorted(v, a, side="right") - 1       # v[low] <= a
        high = np.minimum(low + 1, len(v) - 1)
        frac = np.where(high > low, (a - v[low]) / np.where(high > low, v[high] - v[low], 1), 0)
        # the last 4 of the 20 bits below a code are not compared; between 0 and the least value
        # the distance is compared whole
        up = np.where(low > 0, np.floor(frac * 2.0 ** 20) + 16 * u >= 2.0 ** 20, frac * 65536 > u)
        c = np.where(up, high, low)
        if signed:
            c = c | np.where((x[part] < 0) & (c > 0), 128, 0)
        codes[part] = c
    return codes, scales


def moments(g, m, v, beta1, beta2):
    """m, v and sqrt(v) by single rounded fp32 operations."""
    g = g.astype(f32)
    m = m.astype(f32) * f32(beta1) + g * f32(1 - beta1)
    v = v.astype(f32) * f32(beta2) + (g * f32(1 - beta2)) * g
    return m, v, np.sqrt(v)


def clip_factor(norm, max_norm):
    """fp32 factor of the gradients."""
    return f32(1.0) if norm is None else min(f32(1.0), f32(max_norm) / (f32(norm) + f32(CLIP_EPS)))


def adamw(p, g, m, v, t, lr, beta1, beta2, eps, decay, factor=1.0):
    """(p, m, v) in fp64."""
    g = g * float(factor)
    m, v = beta1 * m + (1 - beta1) * g, beta2 * v + (1 - beta2) * g * g
    step = lr / (1 - beta1 ** t) * m / (np.sqrt(v / (1 - beta2 ** t)) + eps)
    return p * (1 - lr * decay) - step, m, v
