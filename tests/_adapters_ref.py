"""64-bit NumPy forms of the expert selection and the low-rank adapters, written
from their definitions for the tests, with bounds on what rounding may do."""
import numpy as np

U = 2.0 ** -24     # half a step of fp32, relative


def scores(l, score):
    """p [M][E] of logits float64; -infinity and NaN count nothing, +infinity is the largest fp32 value."""
    l = np.where(np.isnan(l), -np.inf, np.minimum(l, np.finfo(np.float32).max))
    if score == 1:
        with np.errstate(over="ignore"):
            return l, 1 / (1 + np.exp(-l))
    top = l.max(1, keepdims=True)
    e = np.where(np.isinf(l), 0.0, np.exp(l - np.where(np.isinf(top), 0.0, top)))
    s = e.sum(1, keepdims=True)
    return l, np.where(s > 0, e / np.where(s > 0, s, 1), 0.0)


def select(logits, top_k, bias=None, score=0, groups=1, top_groups=1, group_picks=1, renormalise=True, scale=1.0):
    """(ids int32, weights float64), token by token with Python sorts."""
    l, p = scores(logits, score)
    M, E = l.shape
    each = E // groups
    ids, w = np.full((M, top_k), -1, np.int32), np.zeros((M, top_k))
    for t in range(M):
        c = l[t] if bias is None and groups == 1 else p[t] + (0.0 if bias is None else bias)
        there = [e for e in range(E) if l[t, e] > -np.inf and (bias is None or bias[e] > -np.inf)]
        if groups > 1:
            value = {}
            for g in {e // each for e in there}:
                best = sorted((c[e] for e in there if e // each == g), reverse=True)
                value[g] = sum(best[:group_picks])
            kept = sorted(value, key=lambda g: (-value[g], g))[:top_groups]
            there = [e for e in there if e // each in kept]
        picks = sorted(there, key=lambda e: (-c[e], e))[:top_k]
        ids[t, :len(picks)] = picks
        s = p[t, picks]
        total = s.sum() if renormalise else 1.0
        w[t, :len(picks)] = scale * s / total if total > 0 else 0.0
    return ids, w


def select_backward(d_w, logits, ids, score=0, renormalise=True, scale=1.0):
    """(d_logits float64, bound on its error before the last rounding)."""
    l, p = scores(logits, score)
    M, E = l.shape
    d, bound = np.zeros((M, E)), np.zeros((M, E))
    span = np.minimum(128, np.where(np.isinf(l), 0, np.abs(l)).max(1)) if score == 0 else np.zeros(M)
    for t in range(M):
        slots = [j for j, e in enumerate(ids[t]) if 0 <= e < E]
        e, g = ids[t][slots], d_w[t][slots]
        S = p[t, e].sum() if renormalise else 1.0
        if S == 0:
            continue
        ds, big = np.zeros(E), np.zeros(E)
        mean = (p[t, e] * g).sum() / S if renormalise else 0.0
        amean = (p[t, e] * np.abs(g)).sum() / S if renormalise else 0.0
        np.add.at(ds, e, scale * (g - mean) / S)
        np.add.at(big, e, abs(scale) * (np.abs(g) + amean) / S)
        if score == 1:
            with np.errstate(over="ignore"):
                q = p[t] / (1 + np.exp(l[t]))
            d[t], bound[t] = ds * q, big * q
        else:
            d[t], bound[t] = p[t] * (ds - (p[t] * ds).sum()), p[t] * (big + (p[t] * big).sum())
        # each score and sum is a few roundings off, exp by as many as its argument has
        bound[t] *= (40 + len(slots) + 4 * span[t]) * U
    return d, bound


def pieces(dtype, n):
    """Relative error of a value held as n 16-bit pieces."""
    return {"float16": {2: 2.0 ** -21, 3: 2.0 ** -21}, "bfloat16": {2: 2.0 ** -16, 3: 2.0 ** -23}}[dtype][n]


def forward(x, a, b, scales, ids, base, dtype):
    """(y, h, bound of y before its rounding, bound of h), all float64: a sum of n terms in 32 bits is off by at most
    n roundings of the terms' absolute sum; h enters the second product as two 16-bit pieces."""
    M, N, r, K = x.shape[0], b.shape[1], a.shape[1], x.shape[1]
    y = np.zeros((M, N)) if base is None else base.copy()
    by = np.abs(y) * 4 * U
    h, bh = np.zeros((M, r)), np.zeros((M, r))
    for i in range(a.shape[0]):
        t = np.nonzero(ids == i)[0]
        if len(t) == 0:
            continue
        h[t] = x[t] @ a[i].T
        bh[t] = (K + 8) * U * (np.abs(x[t]) @ np.abs(a[i]).T)
        y[t] += scales[i] * (h[t] @ b[i].T)
        eh = bh[t] + np.abs(h[t]) * (pieces(dtype, 2) + (2 * r + 8) * U)
        by[t] += abs(scales[i]) * (eh @ np.abs(b[i]).T)
    return y, h, by, bh


def backward(dy, x, h, a, b, scales, ids, base, dtype):
    """(dx, d_a, d_b) and their bounds (dx's before its rounding)."""
    M, K = x.shape
    N = dy.shape[1]
    dx = np.zeros((M, K)) if base is None else base.copy()
    bx = np.abs(dx) * 4 * U
    da, db = np.zeros(a.shape), np.zeros(b.shape)
    ba, bb = np.zeros(a.shape), np.zeros(b.shape)
    for i in range(a.shape[0]):
        t = np.nonzero(ids == i)[0]
        if len(t) == 0:
            continue
        r = a.shape[1]
        u = scales[i] * (dy[t] @ b[i])
        bu = (N + 8) * U * abs(scales[i]) * (np.abs(dy[t]) @ np.abs(b[i]))
        dx[t] += u @ a[i]
        bx[t] += (bu + np.abs(u) * (pieces(dtype, 2) + (2 * r + 8) * U)) @ np.abs(a[i])
        n = (3 * len(t) + 16) * U + pieces(dtype, 3)
        da[i] = u.T @ x[t]
        ba[i] = (bu + n * np.abs(u)).T @ np.abs(x[t])
        db[i] = scales[i] * (dy[t].T @ h[t])
        bb[i] = abs(scales[i]) * n * (np.abs(dy[t]).T @ np.abs(h[t]))
    return (dx, da, db), (bx, ba, bb)
