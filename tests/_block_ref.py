"""Plain 64-bit references of the grouped router and of the norms around a block, and the
bounds their fp32 evaluation is held to.

Each ``e`` below is a bound of a value's absolute error.  U32 is half a step of fp32,
relative; sums of a row take at most 16 values in turn in a lane, 6 steps over a wave, 4
over a block's waves and one product with 1/H (itself rounded): below 32 half-steps of
the magnitudes they add."""

from __future__ import annotations

import numpy as np

import _experts_ref as R

U32, UBF16 = R.U32, R.UBF16
SUM = 32 * U32


def grouped(x, bias, k, score, normalize, scale, groups, top_groups, by):
    """(indices, weights) of the router over groups."""
    x = np.asarray(x, dtype=np.float64)
    T, E = x.shape
    S = E // groups
    if score == "sigmoid" and bias is not None:
        order = R.scores(x, score)[0] + np.asarray(bias, dtype=np.float64)
        of = order
    else:
        order = of = x
        if by == "top2" and score == "sigmoid":
            of = R.scores(x, score)[0]
        elif by == "top2":  # p up to a factor of the row: relative to the largest if finite
            m = np.where(np.isnan(x), -np.inf, x).max(axis=1, keepdims=True)
            of = np.exp(x - np.where(np.isfinite(m), m, 0.0))
    with np.errstate(invalid="ignore"):
        inside = -np.sort(-np.where(np.isnan(of), -np.inf, of).reshape(T, groups, S), axis=2)
        best = inside[:, :, 0]
        if by == "top2":
            best = np.where(best == np.inf, best, best + inside[:, :, 1])
    chosen = R.top(best, top_groups)
    # experts of groups left out come after NaN: they are never among the first k
    keep = np.zeros((T, groups), bool)
    np.put_along_axis(keep, chosen.astype(np.int64), True, axis=1)
    keep = np.repeat(keep, S, axis=1)
    idx = np.empty((T, k), np.int32)
    for t in range(T):
        at = np.flatnonzero(keep[t])
        idx[t] = at[R.top(order[t, at][None], k)[0]]
    return idx, R.gate_weights(x, idx, score, normalize, scale)


def hat(kind, u, eu, eps):
    """(normed rows, their error, factor)."""
    if kind == "none":
        return u, eu, np.ones((u.shape[0], 1))
    if kind == "layer":
        m = u.mean(axis=1, keepdims=True)
        em = eu.mean(axis=1, keepdims=True) + SUM * np.abs(u).mean(axis=1, keepdims=True)
        u = u - m
        eu = eu + em + U32 * np.abs(u)
    r = 1.0 / np.sqrt((u * u).mean(axis=1, keepdims=True) + eps)
    h = u * r
    # half the sum's error, the root, the quotient, the product
    rel = r * np.sqrt((eu * eu).mean(axis=1, keepdims=True)) + SUM / 2 + 3 * U32
    return h, r * eu + np.abs(h) * rel, r


def factor(w, offset, H):
    return np.ones(H) if w is None else offset + np.asarray(w, dtype=np.float64)


def gate_of(gate, sigmoid):
    """(factor, slope) as columns of rows; the sigmoid within 8 half-steps."""
    if gate is None:
        return np.ones((1, 1)), np.ones((1, 1))
    g = np.asarray(gate, dtype=np.float64)
    g = g[:, None] if g.ndim == 1 else g
    if not sigmoid:
        return g, np.ones_like(g)
    f = 1.0 / (1.0 + np.exp(-g))
    return f, f * (1.0 - f)


def block_norm(c, x, y, gate, wp, bp, wn, bn):
    """c: dict of post, pre, sigmoid, eps, offset, a, c.  ((s, es), (n, en)) before any
    rounding to the rows' type."""
    shape = (x if x is not None else y).shape
    s, es = np.zeros(shape), np.zeros(shape)
    if y is not None:
        h, eh, _ = hat(c["post"], y, np.zeros(shape), c["eps"])
        W = factor(wp, c["offset"], shape[1])
        v = h * W + (0 if bp is None else bp)
        ev = eh * np.abs(W) + U32 * (np.abs(h * W) + np.abs(v))
        g, _ = gate_of(gate, c["sigmoid"])
        s = c["c"] * g * v
        es = np.abs(c["c"] * g) * ev + 12 * U32 * np.abs(s)
    if x is not None:
        s = s + c["a"] * x
        es = es + 2 * U32 * np.abs(s)
    h, eh, _ = hat(c["pre"], s, es, c["eps"])
    W = factor(wn, c["offset"], shape[1])
    n = h * W + (0 if bn is None else bn)
    return (s, es), (n, eh * np.abs(W) + 2 * U32 * (np.abs(h * W) + np.abs(n)))


def hat_backward(kind, h, eh, r, g, eg):
    """(what the norm hands back of g, error)."""
    if kind == "none":
        return g, eg
    mean = lambda a: a.mean(axis=1, keepdims=True)  # noqa: E731
    along, ealong = mean(g * h), mean(eg * np.abs(h) + np.abs(g) * eh) + SUM * mean(np.abs(g * h))
    base, ebase = 0.0, 0.0
    if kind == "layer":
        base, ebase = mean(g), mean(eg) + SUM * mean(np.abs(g))
    out = r * (g - base - h * along)
    mag = r * (np.abs(g) + np.abs(base) + np.abs(h * along))
    err = r * (eg + ebase + eh * np.abs(along) + np.abs(h) * ealong) + (SUM / 2 + 8 * U32) * mag
    return out, err


def block_norm_backward(c, gs, gn, s, y, gate, wp, bp, wn, rows):
    """{name: (gradient, error)} before any rounding to the rows' type; rows: the most that
    one partial sum of a column holds."""
    shape = (gs if gs is not None else gn).shape
    H, zero = shape[1], np.zeros(shape)
    out = {}

    def column(terms, errs):
        return terms.sum(axis=0), errs.sum(axis=0) + (rows + 2) * U32 * np.abs(terms).sum(axis=0)

    grad, egrad = (zero, zero) if gs is None else (gs, zero)
    if gn is not None:
        h, eh, r = hat(c["pre"], s, zero, c["eps"])
        W = factor(wn, c["offset"], H)
        g = gn * W
        back, eback = hat_backward(c["pre"], h, eh, r, g, 2 * U32 * np.abs(g))
        egrad = eback + U32 * (np.abs(back) + np.abs(grad))
        grad = grad + back
        out["pre_weight"] = column(gn * h, np.abs(gn) * eh + U32 * np.abs(gn * h))
        out["pre_bias"] = column(gn, zero)
    out["x"] = c["a"] * grad, np.abs(c["a"]) * egrad + U32 * np.abs(c["a"] * grad)
    if y is None:
        return out
    h, eh, r = hat(c["post"], y, zero, c["eps"])
    W = factor(wp, c["offset"], H)
    v = h * W + (0 if bp is None else bp)
    ev = eh * np.abs(W) + 2 * U32 * (np.abs(h * W) + np.abs(v))
    f, slope = gate_of(gate, c["sigmoid"])
    f = c["c"] * f
    gv = f * grad
    egv = np.abs(f) * egrad + 12 * U32 * np.abs(gv)
    g, eg = gv * W, egv * np.abs(W) + 2 * U32 * np.abs(gv * W)
    out["y"] = hat_backward(c["post"], h, eh, r, g, eg)
    out["post_weight"] = column(gv * h, egv * np.abs(h) + np.abs(gv) * eh + U32 * np.abs(gv * h))
    out["post_bias"] = column(gv, egv)
    if gate is not None:
        t = c["c"] * grad * v * slope
        et = np.abs(c["c"] * slope) * (egrad * np.abs(v) + np.abs(grad) * ev) + 16 * U32 * np.abs(t)
        if np.ndim(gate) == 1:
            out["gate"] = t.sum(axis=1), et.sum(axis=1) + SUM * np.abs(t).sum(axis=1)
        else:
            out["gate"] = t, et
    return out


def rounded(value, error, dtype):
    """The bound of a value in the rows' type."""
    return error + (UBF16 if dtype == "bf16" else U32) * (np.abs(value) + error) + 1e-37
