"""Plain 64-bit definitions of the operators around the expert GEMMs: routing,
its gradient, the dispatch plan, the combine of the experts' rows and its
gradient, and clipping by the global norm.  numpy, one row at a time, written
from the formulas in include/mx.h; test infrastructure only.
"""
from __future__ import annotations

import math

import numpy as np

SOFTMAX, SIGMOID = 0, 1


def scores(l, score):
    """Scores of one row of logits in 64 bits; a row of -inf alone has none."""
    l = np.asarray(l, dtype=np.float64)
    with np.errstate(all="ignore"):
        if score == SIGMOID:
            return np.exp(_log_sigmoid(l))
        if np.isneginf(l).all():
            return np.zeros_like(l)
        x = np.exp(l - np.nanmax(l))
        return x / x.sum()


def keys(l, bias, score, groups, group_best):
    """What the choice goes by (-inf: not available)."""
    l = np.asarray(l, dtype=np.float64)
    if bias is None and (groups == 1 or group_best == 1):
        return l.copy()
    s = scores(l, score)
    if bias is None:
        return np.where(np.isneginf(l), -np.inf, s)
    b = np.asarray(bias, dtype=np.float64)
    return np.where(np.isneginf(l) | np.isneginf(b), -np.inf, s + b)


def _order(v):
    """Indices best first: NaN behind every number, -inf last, ties lowest."""
    rank = np.where(np.isneginf(v), 2, np.where(np.isnan(v), 1, 0))
    return sorted(range(len(v)), key=lambda i: (rank[i], -v[i] if rank[i] == 0 else 0.0, i))


def group_scores(key, groups, group_best):
    out = np.full(groups, -np.inf)
    size = len(key) // groups
    for g in range(groups):
        low = -float(np.finfo(np.float32).max)
        k = [x for x in key[g * size:(g + 1) * size] if not np.isneginf(x) and not np.isnan(x)]
        if k:
            out[g] = max(sum(sorted(k)[-group_best:]), low)
    return out


def route_row(l, top_k, score=SOFTMAX, bias=None, groups=1, top_groups=1, group_best=1, renorm=True, scale=1.0):
    """ids, weights of one row, and the smallest distance between two different
    keys (or group scores) that the choice turns on."""
    key = keys(l, bias, score, groups, group_best)
    margin = np.inf

    def gap(v, n):
        near = [v[i] for i in _order(v)[:n + 1] if np.isfinite(v[i])]
        return min([a - b for a, b in zip(near, near[1:]) if a > b], default=np.inf)

    if groups > 1 and top_groups < groups:
        of = group_scores(key, groups, group_best)
        margin = gap(of, top_groups)
        keep = set(_order(of)[:top_groups])
        size = len(key) // groups
        key = np.array([k if e // size in keep else -np.inf for e, k in enumerate(key)])
    margin = min(margin, gap(key, top_k))
    at = [e for e in _order(key)[:top_k] if not np.isneginf(key[e])]
    ids = np.array(at + [-1] * (top_k - len(at)), dtype=np.int32)
    return ids, weights_of(l, ids, score, renorm, scale), margin


def weights_of(l, ids, score, renorm, scale):
    """The weights of the chosen experts (the choice held fixed)."""
    l = np.asarray(l, dtype=np.float64)
    there = [int(e) for e in ids if 0 <= e < len(l)]
    w = np.zeros(len(ids))
    if not there:
        return w
    if renorm:
        # s / sum s with every score scaled alike, so that none underflows
        c = l[there]
        with np.errstate(all="ignore"):
            top = np.nanmax(c) if not np.isnan(c).all() else 0.0
            p = np.exp(c - top)
            if score == SIGMOID:
                p = np.exp(_log_sigmoid(c) - _log_sigmoid(np.array([top]))[0])
            p = p / p.sum()
    else:
        p = scores(l, score)[there]
    w[[j for j, e in enumerate(ids) if 0 <= e < len(l)]] = scale * p
    return w


def _log_sigmoid(x):
    return np.minimum(x, 0.0) - np.log1p(np.exp(-np.abs(x)))


def route_bwd_row(l, ids, dw, score=SOFTMAX, renorm=True, scale=1.0):
    """d(sum_j dw_j w_j) / dl, from the chain rule through the scores."""
    l = np.asarray(l, dtype=np.float64)
    n = len(l)
    j = [i for i, e in enumerate(ids) if 0 <= e < n]
    at = [int(ids[i]) for i in j]
    d = np.zeros(n)
    if not at:
        return d
    g = scale * np.asarray(dw, dtype=np.float64)[j]
    if renorm:
        p = weights_of(l, np.array(at), score, True, 1.0)
        for m, e in enumerate(at):
            d[e] = p[m] * (g[m] - (g * p).sum()) * (1.0 if score == SOFTMAX else scores(-l[[e]], SIGMOID)[0])
        return d
    s = scores(l, score)
    if score == SIGMOID:
        for m, e in enumerate(at):
            d[e] = g[m] * s[e] * scores(-l[[e]], SIGMOID)[0]
        return d
    ds = np.zeros(n)
    ds[at] = g
    return s * (ds - (ds * s).sum())


def route_plan(ids, experts):
    flat = np.asarray(ids).reshape(-1)
    bins = [[] for _ in range(experts + 1)]
    for i, e in enumerate(flat):
        bins[e if 0 <= e < experts else experts].append(i)
    order = np.array([i for b in bins for i in b], dtype=np.int64)
    slot = np.full(flat.size, -1, dtype=np.int32)
    for p, i in enumerate(order):
        if 0 <= flat[i] < experts:
            slot[i] = p
    offsets = np.cumsum([0] + [len(b) for b in bins[:-1]]).astype(np.int32)
    k = ids.shape[1]
    return offsets, (order // k).astype(np.int32), slot.reshape(ids.shape)


def combine(y, slot, weights=None, residual=None):
    y = np.asarray(y, dtype=np.float64)
    t, k = slot.shape
    out = np.zeros((t, y.shape[1])) if residual is None else np.array(residual, dtype=np.float64)
    for i in range(t):
        for j in range(k):
            if 0 <= slot[i, j] < len(y):
                out[i] += (1.0 if weights is None else float(weights[i, j])) * y[slot[i, j]]
    return out


def combine_bwd(dout, y, slot, weights=None):
    """dy (rows that no slot names stay NaN) and dweights."""
    y, dout = np.asarray(y, dtype=np.float64), np.asarray(dout, dtype=np.float64)
    dy, dw = np.full(y.shape, np.nan), np.zeros(slot.shape)
    for i in range(slot.shape[0]):
        for j in range(slot.shape[1]):
            s = slot[i, j]
            if 0 <= s < len(y):
                dy[s] = (1.0 if weights is None else float(weights[i, j])) * dout[i]
                dw[i, j] = (dout[i] * y[s]).sum()
    return dy, dw


def grad_norm(grads):
    return math.sqrt(math.fsum(float(v) * float(v) for g in grads for v in np.asarray(g).reshape(-1)))


def clip_coef(norm, max_norm):
    return min(1.0, max_norm / (norm + 1e-6)) if math.isfinite(norm) else 1.0
