"""Plain 64-bit references of the router and expert calls, and the bounds their
results are held to."""

from __future__ import annotations

import math

import numpy as np

U32 = 2.0 ** -24   # half a step of fp32, relative
UBF16 = 2.0 ** -8  # of bf16


def scores(x, score):
    """(values v, probabilities p) of logits x [T,E] in 64 bits; a row of -inf
    has p = 0."""
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "softmax":
            m = x.max(axis=1, keepdims=True)
            v = np.exp(x - np.where(np.isneginf(m), 0.0, m))
        else:
            v = 1.0 / (1.0 + np.exp(-x))
        s = v.sum(axis=1, keepdims=True)
        return v, np.where(s == 0, 0.0, v / np.where(s == 0, 1.0, s))


def top(order, k):
    """Columns of the k largest of each row, ties to the lower, NaN last."""
    key = np.where(np.isnan(order), -np.inf, order)
    rank = np.lexsort((np.broadcast_to(np.arange(order.shape[1]), order.shape), -key,
                       np.isnan(order)), axis=1)
    return rank[:, :k].astype(np.int32)


def gate_weights(x, idx, score, normalize, scale):
    v, p = scores(x, score)
    w = np.take_along_axis(v if score == "sigmoid" or normalize else p, idx, axis=1)
    if normalize:
        s = w.sum(axis=1, keepdims=True)
        w = np.where(s == 0, 0.0, w / np.where(s == 0, 1.0, s))
    return w * scale


def gate(x, bias, k, score, normalize, scale):
    x = np.asarray(x, dtype=np.float64)
    if score == "sigmoid" and bias is not None:
        order = scores(x, score)[0] + np.asarray(bias, dtype=np.float64)
    else:
        order = x  # the sigmoid is increasing
    idx = top(order, k)
    return idx, gate_weights(x, idx, score, normalize, scale)


def balance(x, idx, mask, score, coef):
    T, E = x.shape
    keep = np.ones(T, bool) if mask is None else np.asarray(mask) != 0
    n, k = int(keep.sum()), idx.shape[1]
    ids = idx[keep].reshape(-1)
    counts = np.bincount(ids[(ids >= 0) & (ids < E)], minlength=E)
    if n == 0:
        return np.zeros(E + 1, np.int64), np.zeros(E), 0.0
    mean = scores(x[keep], score)[1].sum(axis=0) / n
    return np.append(counts, n), mean, coef * E / (k * n) * float((counts * mean).sum())


def gate_grad(x, idx, mask, score, normalize, scale, coef, gw, counts, gl):
    """(gradient, bound of its fp32 evaluation): the bound adds up the magnitudes
    of the terms the formula subtracts."""
    x = np.asarray(x, dtype=np.float64)
    T, E = x.shape
    k = idx.shape[1]
    v, p = scores(x, score)
    g, mag = np.zeros((T, E)), np.zeros((T, E))
    s = v.sum(axis=1, keepdims=True)
    inv = np.where(s == 0, 0.0, 1.0 / np.where(s == 0, 1.0, s))
    slope = v * (1.0 - v)
    if counts is not None and counts[E] > 0:
        n = float(counts[E])
        u = gl * coef * E / (k * n * n) * np.asarray(counts[:E], dtype=np.float64)[None]
        dot = (u * p).sum(axis=1, keepdims=True)
        f = p if score == "softmax" else slope * inv
        g += f * (u - dot)
        mag += f * (np.abs(u) + np.abs(dot))
    if gw is not None:
        ok = (idx >= 0) & (idx < E)
        safe = np.where(ok, idx, 0)
        vk = np.where(ok, np.take_along_axis(v, safe, axis=1), 0.0)
        dk = np.where(ok, np.take_along_axis(slope, safe, axis=1), 0.0)
        w = np.where(ok, scale * np.asarray(gw, dtype=np.float64), 0.0)
        tot = vk.sum(axis=1, keepdims=True)
        tinv = np.where(tot == 0, 0.0, 1.0 / np.where(tot == 0, 1.0, tot))
        mean, amean = (w * vk).sum(axis=1, keepdims=True), (np.abs(w) * vk).sum(axis=1, keepdims=True)
        if normalize:
            f = vk if score == "softmax" else dk
            add, amag = f * tinv * (w - mean * tinv), f * tinv * (np.abs(w) + amean * tinv)
        elif score == "softmax":
            add, amag = vk * inv * w, np.abs(vk * inv * w)
            g -= p * mean * inv
            mag += p * amean * inv
        else:
            add, amag = dk * w, np.abs(dk * w)
        rows = np.repeat(np.arange(T), k)
        np.add.at(g, (rows, safe.reshape(-1)), np.where(ok, add, 0.0).reshape(-1))
        np.add.at(mag, (rows, safe.reshape(-1)), np.where(ok, amag, 0.0).reshape(-1))
    if mask is not None:
        g[np.asarray(mask) == 0] = 0.0
        mag[np.asarray(mask) == 0] = 0.0
    return g, mag


# Roundings of a probability: the exponential within 2 units of its last place
# (4 half-steps) and the argument's rounding, which the exponent's size turns
# into |x - max| half-steps (logits here lie within 2 * 12 of each other); the
# sum of at most 64 values in a lane and 6 more over lanes; division or
# reciprocal and product, 3.
def prob_steps(spread=24.0):
    return 4 + spread + 70 + 3


_erf = np.vectorize(math.erf, otypes=[np.float64])


def act(z, name, N):
    sg = lambda a: 1.0 / (1.0 + np.exp(-a))  # noqa: E731
    if name == "gelu":
        return 0.5 * z * (1.0 + _erf(z / math.sqrt(2.0)))
    if name == "silu":
        return z * sg(z)
    if name == "silu_glu":
        return z[:, :N] * sg(z[:, :N]) * z[:, N:]
    return z


def act_grad(gy, z, name, N):
    sg = lambda a: 1.0 / (1.0 + np.exp(-a))  # noqa: E731
    if name == "none":
        return gy
    if name == "gelu":
        return gy * (0.5 * (1.0 + _erf(z / math.sqrt(2.0)))
                     + z * np.exp(-z * z / 2.0) / math.sqrt(2.0 * math.pi))
    g = z[:, :N]
    s = sg(g)
    slope = s * (1.0 + g * (1.0 - s))
    if name == "silu":
        return gy * slope
    return np.concatenate([gy * z[:, N:] * slope, gy * g * s], axis=1)
