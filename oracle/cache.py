"""Plain 64-bit definitions of the key/value cache and of the attention over
it.  numpy, written from the formulas in include/mx.h; test infrastructure
only.  (The cache's codes and scales are oracle.quantize_1d's, bit for bit.)
"""
from __future__ import annotations

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def decode(codes, scales):
    """Values of codes [..., n / 2] with one scale byte for 32: [..., n / 32]."""
    codes = np.asarray(codes)
    nibble = np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[:-1] + (2 * codes.shape[-1],))
    value = np.where(nibble & 8, -1.0, 1.0) * GRID[nibble & 7]
    unit = np.where(scales == 255, np.nan, np.exp2(np.asarray(scales, dtype=np.float64) - 127))
    return value * np.repeat(unit, 32, axis=-1)


def rht(x, mask, inverse=False):
    """The transform of every 32-block of the last axis (a block that is not
    finite leaves the others alone)."""
    h = np.array([[1.0]])
    for _ in range(5):
        h = np.block([[h, h], [h, -h]])
    m = h * np.array([-1.0 if (mask >> j) & 1 else 1.0 for j in range(32)]) / np.sqrt(32.0)
    x = np.asarray(x, dtype=np.float64)
    return (x.reshape(-1, 32) @ (m if inverse else m.T)).reshape(x.shape)


def token_slots(table, length, page_size, pages):
    """The slot of each key of a sequence, -1 where its page does not exist."""
    at = np.asarray([int(table[j // page_size]) * page_size + j % page_size
                     if 0 <= table[j // page_size] < pages else -1 for j in range(length)], dtype=np.int64)
    return at


def held(codes, scales, slots, head):
    """Values [len(slots), dim] of one head in these slots."""
    page_size = codes.shape[2]
    p, o = slots // page_size, slots % page_size
    return decode(codes[p, head, o], scales[p, head, :, o])


def attention(cache, q, table, lengths, q_offsets=None, scale=None, causal=True, window=0, sinks=None, mask=None):
    """cache: (k_codes, k_scales, v_codes, v_scales); q [tokens, q_heads, dim]
    in 64 bits; mask: the RHT's signs, None without.
    Returns out, lse, and what errors are measured by, for each row: the sum of
    p |v| (transformed back as magnitudes: every element of a block gets the
    block's norm), and the largest scale * sum |q k|.  Rows in no sequence are
    NaN in all."""
    k_codes, k_scales, v_codes, v_scales = cache
    pages, heads, page_size, half = k_codes.shape
    tokens, q_heads, dim = q.shape
    scale = dim ** -0.5 if scale is None else scale
    off = np.arange(len(lengths) + 1) if q_offsets is None else np.asarray(q_offsets)
    out, size = np.full(q.shape, np.nan), np.full(q.shape, np.nan)
    lse, reach = np.full((tokens, q_heads), np.nan), np.full((tokens, q_heads), np.nan)
    for s in range(len(lengths)):
        n = off[s + 1] - off[s]
        length = max(0, min(int(lengths[s]), table.shape[1] * page_size))
        slots = token_slots(table[s], length, page_size, pages)
        for h in range(q_heads if n > 0 else 0):
            kv = h // (q_heads // heads)
            keys, values = (held(c, sc, np.maximum(slots, 0), kv) for c, sc in ((k_codes, k_scales), (v_codes, v_scales)))
            for i in range(n):
                pos = length - n + i
                last = pos if causal else length - 1
                first = max(0, pos - window + 1) if window else 0
                seen = np.flatnonzero((np.arange(length) <= last) & (np.arange(length) >= first) & (slots >= 0))
                row = off[s] + i
                x = q[row, h] if mask is None else rht(q[row, h], mask)
                with np.errstate(all="ignore"):
                    z = scale * (keys[seen] @ x)
                    all_z = z if sinks is None else np.append(z, float(sinks[h]))
                    if np.isneginf(all_z).all():           # (also: there are none)
                        out[row, h], size[row, h], lse[row, h], reach[row, h] = 0.0, 0.0, -np.inf, 0.0
                        continue
                    top = np.max(all_z)
                    total = np.exp(all_z - top).sum()
                    p = np.exp(z - top) / total
                    y, a = p @ values[seen] if len(seen) else np.zeros(dim), p @ np.abs(values[seen])
                if mask is not None:
                    y = rht(y, mask, inverse=True)
                    a = np.repeat(np.sqrt((a.reshape(-1, 32) ** 2).sum(1)), 32)
                out[row, h], size[row, h] = y, a
                lse[row, h] = top + np.log(total)
                reach[row, h] = scale * np.max(np.abs(keys[seen]) @ np.abs(x), initial=0.0)
    return out, lse, size, reach


def scores_of(l, score):
    """Scores of a row: softmax, or sigmoids over their sum, and 1 - sigmoid."""
    l = np.asarray(l, dtype=np.float64)
    with np.errstate(all="ignore"):
        if np.isneginf(l).all():
            return np.zeros_like(l), np.ones_like(l)
        if score == 0:
            e = np.exp(l - np.max(l))
            return e / e.sum(), np.ones_like(l)
        log_sig = np.minimum(l, 0.0) - np.log1p(np.exp(-np.abs(l)))
        e = np.exp(log_sig - np.max(log_sig))
        return e / e.sum(), np.exp(np.minimum(-l, 0.0) - np.log1p(np.exp(-np.abs(l))))


def balance(logits, ids, score=0):
    """loss, counts, slope."""
    tokens, experts = logits.shape
    counts = np.zeros(experts, dtype=np.int64)
    for e in np.asarray(ids).reshape(-1):
        if 0 <= e < experts:
            counts[e] += 1
    used = int((~np.isneginf(logits)).any(1).sum())
    slope = experts * counts / (counts.sum() * used) if counts.sum() * used else np.zeros(experts)
    s = np.zeros(experts)
    for row in logits:
        s += scores_of(row, score)[0]
    return float((slope * s).sum()) if counts.sum() * used else 0.0, counts.astype(np.int32), slope


def balance_bwd(logits, slope, score=0, factor=1.0):
    out = np.zeros(logits.shape)
    for t, row in enumerate(logits):
        s, rest = scores_of(row, score)
        with np.errstate(all="ignore"):
            out[t] = np.where(s == 0, 0.0, factor * s * rest * (slope - (s * slope).sum()))
    return out
