"""4-bit KV cache: per-group asymmetric quantisation and decode over it.

Test infrastructure (see the package docstring). Rows are kept here as plain
arrays -- codes [num_blocks, num_kv_heads, 16, head_dim] (0..15) and {scale,
offset} pairs [num_blocks, num_kv_heads, 16, head_dim / 64, 2] as float64 values
of the cache's 16-bit type -- and `tile_bytes` lays them out as the library
stores them.

The glossary entry "PagedAttention（ページドアテンション）" (section
"他のKVキャッシュ最適化との組み合わせ") names quantised KV caches as a companion
of paging without a scheme. Reading taken: per group of 64 head dims, z = min x,
s = (max x - z) / 15 rounded to the row's type, c = rint((x - z) / s) clamped to
0..15; a group holding an infinity or NaN reads as NaN.
"""

import numpy as np

from .attention import gather_kv
from .numerics import to_f64

GROUP = 64
BLOCK_SIZE = 16


def round_to(x, dtype):
    """float32 values rounded to fp16 or bf16 (nearest even), as float64."""
    x = np.asarray(x, np.float32)
    if dtype == "f16":
        with np.errstate(over="ignore"):
            return x.astype(np.float16).astype(np.float64)
    bits = x.view(np.uint32).astype(np.uint64)
    up = (bits + 0x7FFF + ((bits >> 16) & 1)) & 0xFFFF0000
    out = up.astype(np.uint32).view(np.float32).astype(np.float64)
    return np.where(np.isnan(x), np.nan, out)


def quantize(x, dtype):
    """float rows [..., D] -> codes uint8 [..., D], pairs float64 [..., D / 64, 2]; fp32 steps as defined."""
    g = np.asarray(x, np.float32).reshape(*np.shape(x)[:-1], -1, GROUP)
    half = np.float32(0.5)
    with np.errstate(all="ignore"):
        lo, hi = g.min(-1), g.max(-1)
        s = round_to((half * hi - half * lo) / np.float32(7.5), dtype)
        hs = half * s.astype(np.float32)
        c = np.rint((half * g - (half * lo)[..., None]) / hs[..., None])
        c = np.where(hs[..., None] > 0, np.clip(c, 0, 15), 0)
        bad = ~np.isfinite(g).all(-1)
    c = np.where(bad[..., None], 0, c).astype(np.uint8)
    s = np.where(bad, np.nan, s)
    z = np.where(bad, np.nan, lo.astype(np.float64))
    return c.reshape(np.shape(x)), np.stack((s, z), -1)


def dequantize(codes, pairs):
    """float64 rows z + c s."""
    c = np.asarray(codes, np.float64).reshape(*np.shape(codes)[:-1], -1, GROUP)
    return (c * pairs[..., 0:1] + pairs[..., 1:2]).reshape(np.shape(codes))


def bits_of(x, dtype):
    """uint16 storage of values that the 16-bit type holds exactly."""
    if dtype == "f16":
        return np.asarray(x, np.float16).view(np.uint16)
    return (np.asarray(x, np.float32).view(np.uint32) >> 16).astype(np.uint16)


def _row(slot):
    return 8 * (slot // 8) + 2 * (slot % 4) + (slot // 4) % 2


def tile_bytes(k_codes, k_pairs, v_codes, v_pairs, dtype):
    """The library's tiles uint8 [..., 18 D] of codes [..., 16, D] and pairs [..., 16, D / 64, 2]."""
    D = k_codes.shape[-1]
    lead = k_codes.shape[:-2]
    tile = np.zeros((*lead, 18 * D), np.uint8)
    for slot in range(16):
        row = _row(slot)
        for w in range(D // 8):
            t, i = (w % 8) // 2, 2 * (w // 8) + w % 2
            if D == 256:
                k_at = row * 128 + 16 * ((4 * (i // 4) + t) ^ (4 * (row % 2))) + 4 * (i % 4)
            else:
                k_at = row * (D // 2) + (D // 8) * t + 4 * i
            turn = {64: 0, 128: 4 * ((slot // 2) % 2), 256: 2 * (slot % 4)}[D]
            v_at = 8 * D + slot * (D // 2) + (D // 16) * ((w % 8) ^ turn) + 4 * (w // 8)
            for b in range(4):
                d = 8 * w + 2 * b
                tile[..., k_at + b] = k_codes[..., slot, d] | (k_codes[..., slot, d + 1] << 4)
                tile[..., v_at + b] = v_codes[..., slot, d] | (v_codes[..., slot, d + 1] << 4)
        for base, pairs in ((16 * D, k_pairs), (17 * D, v_pairs)):
            raw = bits_of(pairs[..., slot, :, :], dtype)
            for g in range(D // GROUP):
                for e in range(2):
                    at = base + row * (D // 16) + 4 * g + 2 * e
                    tile[..., at] = raw[..., g, e] & 0xFF
                    tile[..., at + 1] = raw[..., g, e] >> 8
    return tile


def decode(q, k_codes, k_pairs, v_codes, v_pairs, block_tables, context_lens, scale, dtype, window=0):
    """Decode attention over the dequantised cache, float64 [S, Hq, D], and per output element the bound of
    `error_bound`."""
    qf = to_f64(q, dtype)
    S, hq, D = qf.shape
    hkv = k_codes.shape[1]
    group = hq // hkv
    kf, vf = dequantize(k_codes, k_pairs), dequantize(v_codes, v_pairs)
    vc = np.asarray(v_codes, np.float64).reshape(*v_codes.shape[:-1], -1, GROUP) * np.abs(v_pairs[..., 0:1])
    va = (vc + np.abs(v_pairs[..., 1:2])).reshape(v_codes.shape)
    ka = np.abs(np.asarray(k_codes, np.float64).reshape(*k_codes.shape[:-1], -1, GROUP) * k_pairs[..., 0:1]) \
        + np.abs(k_pairs[..., 1:2])
    ka = ka.reshape(k_codes.shape)
    out, bound = np.zeros((S, hq, D)), np.zeros((S, hq, D))
    for s in range(S):
        L = int(context_lens[s])
        first = max(0, L - window) if window > 0 else 0
        if L == 0:
            continue
        for g in range(hkv):
            K, V, KA, VA = (gather_kv(x, block_tables[s], L, g, BLOCK_SIZE)[first:] for x in (kf, vf, ka, va))
            for h in range(g * group, (g + 1) * group):
                x = scale * (K @ qf[s, h])
                p = np.exp(x - x.max())
                p /= p.sum()
                out[s, h] = p @ V
                spread = float((KA @ np.abs(qf[s, h])).max()) * abs(scale)
                bound[s, h] = weight_error(spread, D, 2.0 ** -11) * (p @ VA)
    return out, bound


def weight_error(spread, terms, rounding):
    """Relative error of a softmax-weighted sum's weights: `rounding` of each weight to its 16-bit type, a
    score that is a fp32 sum of `terms` products whose magnitudes sum to `spread` (an error of terms * 2^-23
    of it, once in the weight and once in the sum of the weights), and 2^-20 for the exponential, the
    rescalings and the final division."""
    return rounding + 2.0 * terms * 2.0 ** -23 * spread + 2.0 ** -20
