"""The expert layers' operators from their definitions, in numpy and float64: gated blocks and their gradients, 8-bit
integer quantisation and products, gathered and combined rows.  Imports nothing of the package.
"""
from __future__ import annotations

from math import erfc, pi, sqrt

import numpy as np

_cdf = np.vectorize(lambda v: 0.5 * erfc(-v / sqrt(2.0)), otypes=[float])


def _sigmoid(v):
    e = np.exp(-np.abs(v))
    return np.where(v < 0, e, 1.0) / (1.0 + e)


def activation(v, kind):
    """(value, slope)"""
    v = np.asarray(v, dtype=float)
    if kind == "silu":
        s = _sigmoid(v)
        return v * s, s * (1.0 + v * _sigmoid(-v))
    if kind == "gelu":
        p = _cdf(v)
        return v * p, p + v * np.exp(-0.5 * v * v) / sqrt(2 * pi)
    return np.where(v > 0, v, 0.0), np.where(v > 0, 1.0, 0.0)


def segments(offsets, m):
    """[(group, first row, end)] with bounds clamped to the m rows."""
    if offsets is None:
        return [(None, 0, m)]
    o = np.clip(np.asarray(offsets, dtype=int), 0, m)
    return [(g, o[g], o[g + 1]) for g in range(len(o) - 1) if o[g + 1] > o[g]]


def rows_product(x, w, offsets=None):
    """Each row of x by the transpose of its segment's matrix; (product, the same of magnitudes, rows covered)."""
    n = w.shape[-2]
    y, size, hit = np.zeros((len(x), n)), np.zeros((len(x), n)), np.zeros(len(x), dtype=bool)
    for g, lo, hi in segments(offsets, len(x)):
        m = w if g is None else w[g]
        y[lo:hi], size[lo:hi], hit[lo:hi] = x[lo:hi] @ m.T, np.abs(x[lo:hi]) @ np.abs(m).T, True
    return y, size, hit


def gated(x, gate, up, kind, offsets=None):
    g, u = rows_product(x, gate, offsets)[0], rows_product(x, up, offsets)[0]
    return activation(g, kind)[0] * u


def gated_pre_grads(d, g, u, kind):
    value, slope = activation(g, kind)
    return d * u * slope, d * value


def gated_grad_x(dg, du, gate, up, offsets=None):
    """(gradient, the same of magnitudes)"""
    out, size = np.zeros((len(dg), gate.shape[-1])), np.zeros((len(dg), gate.shape[-1]))
    for g, lo, hi in segments(offsets, len(dg)):
        G, U = (gate, up) if g is None else (gate[g], up[g])
        out[lo:hi] = dg[lo:hi] @ G + du[lo:hi] @ U
        size[lo:hi] = np.abs(dg[lo:hi]) @ np.abs(G) + np.abs(du[lo:hi]) @ np.abs(U)
    return out, size


def gated_grad_w(d, x, offsets=None):
    """(gradient per group, the same of magnitudes) of a projection whose output has the gradient d."""
    groups = 1 if offsets is None else len(offsets) - 1
    out = np.zeros((groups, d.shape[1], x.shape[1]))
    size = np.zeros_like(out)
    for g, lo, hi in segments(offsets, len(d)):
        out[g or 0], size[g or 0] = d[lo:hi].T @ x[lo:hi], np.abs(d[lo:hi]).T @ np.abs(x[lo:hi])
    return (out[0], size[0]) if offsets is None else (out, size)


def quantize_int8(x):
    """(codes, scales): whole rows of x."""
    x = np.asarray(x, dtype=float)
    finite = np.isfinite(x).all(-1)
    with np.errstate(all="ignore"):
        s = (np.abs(np.where(finite[..., None], x, 0.0)).max(-1) / 127).astype(np.float32)
        q = np.where(s[..., None] > 0, x / s[..., None].astype(float), 0.0)
    codes = np.where(finite[..., None], np.clip(np.rint(np.where(np.isfinite(q), q, 0.0)), -127, 127), 0.0)
    return codes.astype(np.int8), np.where(finite, s, np.float32(np.nan))


def gather(src, rows, per=1):
    rows = np.asarray(rows)
    there = (rows >= 0) & (rows < len(src) * per)
    return np.where(there[:, None], src[np.where(there, rows, 0) // per], 0.0)


def combine(src, position, weights=None, residual=None):
    """(sum, the same of magnitudes)"""
    t, k = position.shape
    out = np.zeros((t, src.shape[1])) if residual is None else residual.astype(float).copy()
    size = np.abs(out)
    for j in range(k):
        p = position[:, j]
        there = (p >= 0) & (p < len(src))
        w = np.ones(t) if weights is None else weights[:, j]
        part = np.where(there[:, None], np.where(there, w, 0.0)[:, None] * src[np.where(there, p, 0)], 0.0)
        out, size = out + part, size + np.abs(part)
    return out, size


def combine_backward(grad, src, rows, position, weights):
    """(gradient of src, gradient of the weights, the latter of magnitudes)"""
    t, k = position.shape
    g = gather(grad, rows, k)
    ok = (rows >= 0) & (rows < t * k)
    d_src = g * np.where(ok, weights.reshape(-1)[np.where(ok, rows, 0)], 0.0)[:, None]
    there = (position >= 0) & (position < len(src))
    at = src[np.where(there, position, 0)]
    dots = (grad[:, None] * at).sum(-1)
    sizes = np.abs(grad[:, None] * at).sum(-1)
    return d_src, np.where(there, dots, 0.0), np.where(there, sizes, 0.0)
