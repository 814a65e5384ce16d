"""Plain float64 definitions of the routed-expert operators on the CPU (numpy), for the tests.

Written from the formulas, one value at a time where that is clearest; shares no code with the
library or with the benchmark's plain forms.
"""
from __future__ import annotations

import numpy as np

F32_MAX = float(np.finfo(np.float32).max)
MAX = {"e4m3": 448.0, "e5m2": 57344.0}
MANTISSA = {"e4m3": 3, "e5m2": 2}
LOWEST = {"e4m3": -6, "e5m2": -14}          # exponent of the smallest normal value


def scores(x, score):
    """(scores, which experts are there) of logits (tokens, experts)."""
    x = np.minimum(np.asarray(x, dtype=np.float64), F32_MAX)
    there = x > -np.inf
    s = np.zeros_like(x)
    for t in range(x.shape[0]):
        ok = there[t]
        if not ok.any():
            continue
        if score == "sigmoid":
            with np.errstate(over="ignore"):
                s[t, ok] = 1.0 / (1.0 + np.exp(-x[t, ok]))
        else:
            e = np.exp(x[t, ok] - x[t, ok].max())
            s[t, ok] = e / e.sum()
    return s, there


def ratios(x, score):
    """Scores of the chosen logits x over their sum, from the scores' logarithms: also where the scores underflow."""
    x = np.asarray(x, dtype=np.float64)
    log_s = -np.logaddexp(0.0, -x) if score == "sigmoid" else x
    e = np.exp(log_s - log_s.max())
    return e / e.sum()


def route(x, top_k, bias=None, score="softmax", groups=1, top_groups=1, renormalize=True, scale=1.0):
    s, there = scores(x, score)
    x = np.minimum(np.asarray(x, dtype=np.float64), F32_MAX)
    T, E = s.shape
    experts = np.full((T, top_k), -1, dtype=np.int64)
    weights = np.zeros((T, top_k))
    for t in range(T):
        biased = s[t] + (0.0 if bias is None else np.asarray(bias, dtype=np.float64))
        left = [e for e in range(E) if there[t, e] and not (bias is not None and not biased[e] > -np.inf)]
        if groups > 1:
            per = E // groups
            worth = []
            for g in range(groups):
                best = sorted((biased[e] for e in left if e // per == g), reverse=True)[:2]
                worth.append((-sum(best) if best else np.inf, g))
            kept = {g for _, g in sorted(worth)[:top_groups]}
            left = [e for e in left if e // per in kept]
        order = sorted(left, key=lambda e: (-(x[t, e] if bias is None else biased[e]), e))[:top_k]
        experts[t, :len(order)] = order
        w = s[t, order]
        if renormalize and len(order):
            w = ratios(x[t, order], score)
        weights[t, :len(order)] = w * scale
    return experts, weights


def route_backward(x, experts, grad, score="softmax", renormalize=True, scale=1.0):
    s, there = scores(x, score)
    T, E = s.shape
    dx = np.zeros((T, E))
    for t in range(T):
        slots = [j for j in range(experts.shape[1]) if 0 <= experts[t, j] < E and there[t, experts[t, j]]]
        chosen = [int(experts[t, j]) for j in slots]
        g = np.asarray([float(grad[t, j]) * scale for j in slots])
        if not chosen:
            continue
        if renormalize:
            # with w = s / sum s: ds = (g - sum g w) / sum s, and the softmax's inner sum is zero
            w = ratios([min(float(x[t, e]), F32_MAX) for e in chosen], score)
            for e, d in zip(chosen, w * (g - (g * w).sum())):
                dx[t, e] += d * (1.0 - s[t, e] if score == "sigmoid" else 1.0)
            continue
        ds = g
        full = np.zeros(E)
        for e, d in zip(chosen, ds):
            full[e] += d
        if score == "sigmoid":
            dx[t] = full * s[t] * (1.0 - s[t])
        else:
            dx[t] = s[t] * (full - (full * s[t]).sum())
    return dx


def capacity(n, n_experts, align):
    return -(-(n + min(n, n_experts) * (align - 1)) // align) * align


def group_rows(experts, n_experts, align):
    """counts, offsets, rows, position of a flat list of choices."""
    members = [[] for _ in range(n_experts)]
    for i, e in enumerate(experts):
        if 0 <= e < n_experts:
            members[e].append(i)
    counts = np.asarray([len(m) for m in members])
    offsets = np.concatenate([[0], np.cumsum(-(-counts // align) * align)])
    rows = np.full(capacity(len(experts), n_experts, align), -1)
    position = np.full(len(experts), -1)
    for e, m in enumerate(members):
        for i, r in enumerate(m):
            rows[offsets[e] + i] = r
            position[r] = offsets[e] + i
    return counts, offsets, rows, position


def round_fp8(v, fmt):
    """v (float64, at most the format's largest value) rounded to the format, nearest even."""
    v = np.asarray(v, dtype=np.float64)
    _, e = np.frexp(v)
    step = np.exp2(np.maximum(e - 1, LOWEST[fmt]) - MANTISSA[fmt])
    return np.round(v / step) * step                       # numpy rounds halves to even


def block_exponents(amax, fmt):
    """The least e in [-127, 127] with amax <= MAX * 2^e."""
    e = np.full(amax.shape, 127)
    for cand in range(126, -128, -1):
        e = np.where(amax <= MAX[fmt] * 2.0 ** cand, cand, e)
    return np.where(amax > 0, e, -127)


def quantize(x, fmt, square):
    """(code values, scale exponents) of x (rows, cols); infinities and NaN give NaN codes."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    kb, rb = -(-cols // 128), -(-rows // 128)
    codes = np.zeros((rows, kb * 128))
    exps = np.full((rb if square else rows, -(-kb // 4) * 4), -127)
    tall = 128 if square else 1
    for i in range(0, rows, tall):
        for b in range(kb):
            blk = x[i:i + tall, b * 128:(b + 1) * 128]
            fin = np.where(np.isfinite(blk), np.abs(blk), 0.0)
            e = int(block_exponents(np.asarray(fin.max()), fmt))
            exps[i // tall, b] = e
            v = np.where(np.isfinite(blk), blk, 0.0) * 2.0 ** -e
            codes[i:i + tall, b * 128:b * 128 + blk.shape[1]] = np.where(np.isfinite(blk), round_fp8(v, fmt), np.nan)
    return codes, exps
