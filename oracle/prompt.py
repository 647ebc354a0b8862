"""Attention of several query tokens per sequence, groups behind a shared prefix, and the rotated cache write,
in float64.

Test infrastructure (see the package docstring). Ordinary softmax attention over the rows that a query sees:
`attention` for ragged queries (causal with an optional window, or all rows), `prefix_tables` for the tables
that a decode of sharing groups is defined by, `rotate` for the rotation of pairs by position.
"""

import numpy as np

from .int4 import weight_error
from .numerics import to_f64

BLOCK_SIZE = 16


def visible(context_len, num_queries, i, causal, window):
    """[first, end) of the positions that query token i sees."""
    if not causal:
        return 0, context_len
    end = max(0, context_len - num_queries + i + 1)
    return (max(0, end - window) if window > 0 else 0), end


def attention(q, k_pool, v_pool, block_tables, context_lens, query_starts, scale, dtype, causal=True, window=0,
              heads=None, wanted=None):
    """float64 [T, H, D] and the error bound of each element before the output's own rounding: one rounding of
    every softmax weight to the 16-bit type, and the scores' fp32 arithmetic. ``heads`` picks query heads (all),
    ``wanted`` query tokens (all); other rows stay NaN, as do rows of no sequence."""
    qf, kf, vf = (to_f64(x, dtype) for x in (q, k_pool, v_pool))
    T, Hq, D = qf.shape
    group = Hq // kf.shape[1]
    heads = list(range(Hq)) if heads is None else heads
    out = np.full((T, len(heads), D), np.nan)
    bound = np.zeros((T, len(heads), D))
    rounding = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}[dtype]
    for s in range(len(context_lens)):
        n = int(query_starts[s + 1]) - int(query_starts[s])
        L = int(context_lens[s])
        for i in range(n):
            t = int(query_starts[s]) + i
            if wanted is not None and t not in wanted:
                continue
            first, end = visible(L, n, i, causal, window)
            if end <= first:
                out[t] = 0.0
                continue
            at = np.arange(first, end)
            ids = np.asarray(block_tables[s])[at // BLOCK_SIZE]
            if (ids < 0).any():
                raise ValueError("a visible position maps to no block")
            for j, h in enumerate(heads):
                K, V = kf[ids, h // group, at % BLOCK_SIZE], vf[ids, h // group, at % BLOCK_SIZE]
                x = scale * (K @ qf[t, h])
                p = np.exp(x - x.max())
                p /= p.sum()
                out[t, j] = p @ V
                spread = float((np.abs(K) @ np.abs(qf[t, h])).max()) * abs(scale)
                bound[t, j] = weight_error(spread, D, rounding) * (p @ np.abs(V))
    return out, bound


def prefix_tables(block_tables, group_starts, prefix_blocks):
    """The tables of a decode of groups: each member's first blocks are those of its group's first sequence."""
    out = np.array(block_tables, copy=True)
    for i in range(len(prefix_blocks)):
        first, n = int(group_starts[i]), int(prefix_blocks[i])
        out[first:int(group_starts[i + 1]), :n] = out[first, :n]
    return out


def rotate(x, positions, cos_sin, interleaved):
    """float64 rows [T, H, D] with their first R = cos_sin.shape[1] elements rotated as pairs."""
    y = np.array(x, np.float64)
    R = cos_sin.shape[1]
    for t, p in enumerate(np.asarray(positions).tolist()):
        for i in range(R // 2):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
            c, s = float(cos_sin[p, i]), float(cos_sin[p, R // 2 + i])
            y[t, :, a], y[t, :, b] = x[t, :, a] * c - x[t, :, b] * s, x[t, :, b] * c + x[t, :, a] * s
    return y
