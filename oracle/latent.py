"""Latent attention over paged rows [latent 512, rotary 64], absorbed form, in float64.

Test infrastructure (see the package docstring): out[s, h] = softmax_p(scale *
<q[s, h], row_p>) . latent_p over the sequence's rows. `expanded` computes the
same attention from per-head keys and values, which pins the absorbed form to
the definition of latent attention.
"""

import numpy as np

from .int4 import weight_error
from .numerics import to_f64

LATENT, ROPE, BLOCK_SIZE = 512, 64, 16


def rows_of(cache, table, L):
    """float64 [L, 576] rows of one sequence from a float64 cache [num_blocks, 16, 576]."""
    return np.array([cache[table[p // BLOCK_SIZE], p % BLOCK_SIZE] for p in range(L)]).reshape(L, LATENT + ROPE)


def cache_write(latent, rope, cache, slots):
    """A copy of `cache` (any storage) with each token's row at its slot; slots < 0 are skipped."""
    out = np.array(cache, copy=True)
    for t, slot in enumerate(np.asarray(slots).tolist()):
        if slot >= 0:
            out[slot // BLOCK_SIZE, slot % BLOCK_SIZE] = np.concatenate((latent[t], rope[t]))
    return out


def decode(q, cache, block_tables, context_lens, scale, dtype):
    """float64 [S, H, 512] and the error bound of each element (weights rounded to the 16-bit type)."""
    qf, cf = to_f64(q, dtype), to_f64(cache, dtype)
    S, H, _ = qf.shape
    out, bound = np.zeros((S, H, LATENT)), np.zeros((S, H, LATENT))
    rounding = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}[dtype]
    for s in range(S):
        L = int(context_lens[s])
        if L == 0:
            continue
        rows = rows_of(cf, block_tables[s], L)
        for h in range(H):
            x = scale * (rows @ qf[s, h])
            p = np.exp(x - x.max())
            p /= p.sum()
            out[s, h] = p @ rows[:, :LATENT]
            spread = float((np.abs(rows) @ np.abs(qf[s, h])).max()) * abs(scale)
            bound[s, h] = weight_error(spread, LATENT + ROPE, rounding) * (p @ np.abs(rows[:, :LATENT]))
    return out, bound


def expanded(qn, qr, latent, rope, U, W, scale):
    """Latent attention of one sequence from expanded keys and values: qn [H, N], qr [H, 64], latent
    [L, 512], rope [L, 64], U [H, N, 512] (keys), W [H, V, 512] (values) -> [H, V]."""
    outs = []
    for h in range(len(qn)):
        K, V = latent @ U[h].T, latent @ W[h].T
        x = scale * (K @ qn[h] + rope @ qr[h])
        p = np.exp(x - x.max())
        outs.append((p / p.sum()) @ V)
    return np.array(outs)
