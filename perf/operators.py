"""Cases of the operators over compressed KV caches and of the device-side block tables.

Four kinds of case, each one pass as a serving loop makes it:

* ``int4_write``   -- new tokens' K/V rows are quantised into their slots of the 4-bit cache and read
  back as 16-bit rows (what a prompt step does with a cached prefix).
* ``int4_decode``  -- one query token per sequence attends over the 4-bit cache.
* ``latent_step``  -- each sequence's new latent row is written to its slot, then every query head
  attends over the shared latent rows (the absorbed form of latent attention).
* ``tables``       -- block tables, slot map and lengths of a step are made from the requests' lengths.

``own`` chooses between this file's plain forms (elementary torch operations in 32 bits, rounded once
at the end) and the library's calls.
"""

import math

import numpy as np
import torch

own = False

BLOCK = 16          # tokens per block
GROUP = 64          # head dims that share one scale and one offset in the 4-bit cache
LATENT, ROPE = 512, 64
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def _library():
    import paged_kv_cache_217_gb300 as pkv
    return pkv


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # a decode step's cache write of a 40-head layer, 64 sequences: launch latency counts
        {"name": "int4_write_step", "op": "int4_write", "dtype": "bf16", "tokens": 64, "kv_heads": 40, "head_dim": 128,
         "skipped": 0},
        # a prompt step of several requests packed together, padded at the end, 8 KV heads
        {"name": "int4_write_prompt", "op": "int4_write", "dtype": "f16", "tokens": 12301, "kv_heads": 8,
         "head_dim": 128, "skipped": 211},
        # one user, a short context, 32 query heads on 8 KV heads: the smallest decode call
        {"name": "int4_decode_one", "op": "int4_decode", "dtype": "bf16", "seqs": 1, "median": 411, "spread": 0.0,
         "max_len": 2048, "q_heads": 32, "kv_heads": 8, "head_dim": 128, "window": 0},
        # 40 heads with their own K/V, 64 requests with log-normal lengths
        {"name": "int4_decode_mha", "op": "int4_decode", "dtype": "bf16", "seqs": 64, "median": 512, "spread": 0.8,
         "max_len": 2048, "q_heads": 40, "kv_heads": 40, "head_dim": 128, "window": 0},
        # 32 query heads on 8 KV heads, a wide batch of short chats
        {"name": "int4_decode_gqa", "op": "int4_decode", "dtype": "bf16", "seqs": 256, "median": 150, "spread": 0.6,
         "max_len": 1024, "q_heads": 32, "kv_heads": 8, "head_dim": 128, "window": 0},
        # 96 heads, a few long documents: the largest call
        {"name": "int4_decode_long", "op": "int4_decode", "dtype": "f16", "seqs": 3, "median": 21845, "spread": 0.35,
         "max_len": 32768, "q_heads": 96, "kv_heads": 96, "head_dim": 128, "window": 0},
        # one user on a slice of 16 heads: latency
        {"name": "latent_one", "op": "latent_step", "dtype": "bf16", "seqs": 1, "median": 1030, "spread": 0.0,
         "max_len": 4096, "heads": 16},
        # a served batch on a slice of 16 heads, mixed lengths: bound by the cache's bytes
        {"name": "latent_batch", "op": "latent_step", "dtype": "bf16", "seqs": 96, "median": 1500, "spread": 0.8,
         "max_len": 8192, "heads": 16},
        # all 128 heads on one GPU: matrix products and bytes near balance
        {"name": "latent_wide", "op": "latent_step", "dtype": "bf16", "seqs": 32, "median": 4000, "spread": 0.4,
         "max_len": 12288, "heads": 128},
        # one long document, 64 heads: the context has to be split
        {"name": "latent_long", "op": "latent_step", "dtype": "f16", "seqs": 1, "median": 100003, "spread": 0.0,
         "max_len": 131072, "heads": 64},
        # a decode step of 256 running requests, one token each
        {"name": "tables_step", "op": "tables", "seqs": 256, "median": 700, "spread": 0.8, "max_len": 4096,
         "new_lo": 1, "new_hi": 1, "padding": 0},
        # requests admitted together with their prompts, the slot map padded to the captured size
        {"name": "tables_prompts", "op": "tables", "seqs": 700, "median": 0, "spread": 0.0, "max_len": 4096,
         "new_lo": 1, "new_hi": 3500, "padding": 4097},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["int4_write", "int4_decode", "int4_decode", "latent_step", "latent_step", "tables"])
    if op == "int4_write":
        heads, dim = rng.choice([1, 2, 3, 5, 8, 16, 32, 40]), rng.choice([64, 128, 256])
        tokens = _log_int(rng, 1, max(1, 12301 * 1024 // (heads * dim)))
        return {"op": op, "dtype": rng.choice(["f16", "bf16"]), "tokens": tokens, "kv_heads": heads, "head_dim": dim,
                "skipped": rng.choice([0, tokens // 7, tokens // 2])}
    if op == "int4_decode":
        while True:
            kv, dim, group = rng.choice([1, 2, 4, 5, 8, 12, 24, 40, 96]), rng.choice([64, 128, 128, 256]), \
                rng.choice([1, 1, 2, 3, 4, 5, 8])
            seqs, median = _log_int(rng, 1, 320), _log_int(rng, 1, 30000)
            if kv * group <= 128 and seqs * median * 1.4 * kv * dim <= 3 * 21845 * 96 * 128:
                break
        spread = rng.choice([0.0, 0.3, 0.8])
        return {"op": op, "dtype": rng.choice(["f16", "bf16"]), "seqs": seqs, "median": median, "spread": spread,
                "max_len": max(16, int(median * (1 + 2 * spread))) + rng.randrange(64), "q_heads": kv * group,
                "kv_heads": kv, "head_dim": dim, "window": rng.choice([0, 0, 0, _log_int(rng, 1, 4096)])}
    if op == "latent_step":
        while True:
            seqs, median, heads = _log_int(rng, 1, 200), _log_int(rng, 1, 120000), \
                rng.choice([1, 8, 12, 16, 24, 32, 40, 64, 96, 128])
            if seqs * median * 1.4 <= 32 * 4000 * 1.5:
                break
        spread = rng.choice([0.0, 0.3, 0.8])
        return {"op": op, "dtype": rng.choice(["f16", "bf16"]), "seqs": seqs, "median": median, "spread": spread,
                "max_len": max(16, int(median * (1 + 2 * spread))) + rng.randrange(64), "heads": heads}
    seqs, hi = _log_int(rng, 1, 1500), _log_int(rng, 1, 1600)
    return {"op": op, "seqs": seqs, "median": rng.choice([0, _log_int(rng, 1, 3000)]), "spread": rng.choice([0.0, 0.8]),
            "max_len": 8192, "new_lo": rng.choice([0, 1]), "new_hi": hi, "padding": rng.choice([0, 1, 333])}


def _lengths(case):
    """The batch's lengths; they are part of the case, not of its seed."""
    rng = np.random.default_rng(case["seqs"] * 7919 + case["median"])
    if case["median"] == 0:
        return np.zeros(case["seqs"], np.int64)
    x = np.exp(rng.normal(math.log(case["median"]), case["spread"], case["seqs"]))
    return np.clip(np.rint(x), 1, case["max_len"]).astype(np.int64)


def _new_tokens(case):
    rng = np.random.default_rng(case["seqs"] * 104729 + case["new_hi"])
    return rng.integers(case["new_lo"], case["new_hi"], size=case["seqs"], endpoint=True)


def work(case):
    op = case["op"]
    if op == "int4_write":
        live = case["tokens"] - case["skipped"]
        rows = live * case["kv_heads"]
        full, packed = 4 * case["head_dim"], 18 * case["head_dim"] // 16  # K and V of one row, 16-bit and packed
        read_back = case["tokens"] * case["kv_heads"] * full
        return {"bytes": rows * (full + 2 * packed) + read_back + 16 * case["tokens"], "flops": 0}
    if op == "int4_decode":
        lens = _lengths(case)
        if case["window"]:
            lens = np.minimum(lens, case["window"])
        tokens = int(lens.sum())
        row = case["head_dim"] * 18 // 16
        ids = int((-(-lens // BLOCK)).sum()) * 4
        return {"bytes": tokens * case["kv_heads"] * row + ids + case["seqs"] * (case["q_heads"] * case["head_dim"] * 4 + 4),
                "flops": 4 * tokens * case["q_heads"] * case["head_dim"]}
    if op == "latent_step":
        lens = _lengths(case)
        tokens = int(lens.sum())
        width = LATENT + ROPE
        ids = int((-(-lens // BLOCK)).sum()) * 4
        return {"bytes": tokens * width * 2 + ids + case["seqs"] * (case["heads"] * (width + LATENT) * 2 + width * 4 + 12),
                "flops": 2 * tokens * case["heads"] * (width + LATENT)}
    lens, new = _lengths(case), _new_tokens(case)
    blocks = int((-(-(lens + new) // BLOCK) - -(-lens // BLOCK)).sum())
    return {"bytes": case["seqs"] * 12 + int(new.sum() + case["padding"]) * 8 + blocks * 8 + 16, "flops": 0}


# ---------------------------------------------------------------------------
# the 4-bit cache's tile: 16 tokens of one KV head, 18 * head_dim bytes
#   K codes (8 D bytes), V codes (8 D), K {scale, offset} pairs (D), V pairs (D)
# ---------------------------------------------------------------------------
def _k_row(token):
    """Row of the tile that holds a token's K codes, and its K and V pairs."""
    return 8 * (token >> 3) + 2 * (token & 3) + ((token >> 2) & 1)


def _code_bytes(dim):
    """For K and V: [16, D / 2] byte offsets in the tile; byte j of a token's row holds elements 2j and 2j + 1."""
    token, word, byte = np.ix_(np.arange(16), np.arange(dim // 8), np.arange(4))
    row, lane, i = _k_row(token), (word % 8) // 2, 2 * (word // 8) + word % 2
    if dim == 256:
        k_at = 16 * ((4 * (i // 4) + lane) ^ (4 * (row & 1))) + 4 * (i % 4)
    else:
        k_at = dim // 8 * lane + 4 * i
    turn = {64: 0 * token, 128: 4 * ((token >> 1) & 1), 256: 2 * (token & 3)}[dim]
    v_at = dim // 16 * ((word % 8) ^ turn) + 4 * (word // 8)
    k = row * (dim // 2) + k_at + byte
    v = 8 * dim + token * (dim // 2) + v_at + byte
    return k.reshape(16, dim // 2), v.reshape(16, dim // 2)


def _pair_bytes(dim):
    """For K and V: [16, D / 64, 4] byte offsets of the {scale, offset} pairs."""
    rows = _k_row(np.arange(16))[:, None, None]
    at = rows * (dim // 16) + 4 * np.arange(dim // GROUP)[None, :, None] + np.arange(4)[None, None, :]
    return 16 * dim + at, 17 * dim + at


def _layout(dim, device):
    kc, vc = _code_bytes(dim)
    kp, vp = _pair_bytes(dim)
    return {n: torch.from_numpy(a).to(device) for n, a in (("kc", kc), ("vc", vc), ("kp", kp), ("vp", vp))}


def _quantise(x):
    """Rows x [..., D] of a 16-bit type -> codes [..., D] (uint8, 0..15), scale and offset [..., D / 64] of that type."""
    f = x.float().unflatten(-1, (-1, GROUP))
    lo, hi = f.amin(-1), f.amax(-1)
    s = ((0.5 * hi - 0.5 * lo) / 7.5).to(x.dtype)
    sf = s.float()
    c = torch.round((0.5 * f - 0.5 * lo[..., None]) / (0.5 * sf)[..., None]).clamp_(0, 15)
    c = torch.where(sf[..., None] > 0, c, torch.zeros_like(c))
    return c.flatten(-2).to(torch.uint8), s, lo.to(x.dtype)


def _pack(x, cache, at, code_at, pair_at):
    """Writes rows x [n, D] into flat tiles: `at` [n] (row of `cache`, token in the tile)."""
    tile, token = at
    c, s, lo = _quantise(x)
    cache[tile[:, None], code_at[token]] = c[:, 0::2] | (c[:, 1::2] << 4)
    pairs = torch.stack((s, lo), -1).view(torch.uint8).view(len(tile), -1, 4)
    cache[tile[:, None, None], pair_at[token]] = pairs


def _unpack(tiles, code_at, pair_at, dtype):
    """fp32 rows [..., 16, D] of tiles [..., 18 D] (uint8): code * scale + offset."""
    codes = tiles[..., code_at]
    x = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float().unflatten(-1, (-1, GROUP))
    pairs = tiles[..., pair_at].view(dtype).float()
    return (x * pairs[..., 0:1] + pairs[..., 1:2]).flatten(-2)


def _read_rows(cache, at, code_at, pair_at, dtype):
    """fp32 rows [n, D] of flat tiles at (row of `cache`, token in the tile)."""
    tile, token = at
    codes = cache[tile[:, None], code_at[token]]
    x = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float().unflatten(-1, (-1, GROUP))
    pairs = cache[tile[:, None, None], pair_at[token]].view(dtype).float()
    return (x * pairs[..., 0:1] + pairs[..., 1:2]).flatten(-2)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _tables(lens, extra_blocks, width, gen, device):
    """Block tables over a shuffled pool; padded with -1."""
    counts = -(-lens // BLOCK)
    blocks = int(counts.sum()) + extra_blocks
    order = torch.randperm(blocks, generator=gen, device=device).to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device=device)
    rows = np.repeat(np.arange(len(lens)), counts)
    cols = np.arange(int(counts.sum())) - np.repeat(np.cumsum(counts) - counts, counts)
    table[torch.from_numpy(rows).to(device), torch.from_numpy(cols).to(device)] = order[:len(rows)]
    return table, order, blocks


def _activations(shape, dtype, gen, device):
    """N(0, 1) values whose last dimension's channels differ in size, as K and V channels do."""
    x = torch.randn(shape, generator=gen, device=device)
    size = torch.exp(0.4 * torch.randn(shape[-1:], generator=gen, device=device))
    return (x * size).to(dtype)


def prepare(case, seed):
    device = torch.device("cuda")
    gen = torch.Generator(device=device)
    gen.manual_seed(int(seed) * 2 + 1)
    op, st = case["op"], {"case": case}
    if op == "int4_write":
        dtype, heads, dim, tokens = DTYPES[case["dtype"]], case["kv_heads"], case["head_dim"], case["tokens"]
        blocks = -(-tokens // BLOCK) + 3
        slots = torch.randperm(blocks * BLOCK, generator=gen, device=device)[:tokens]
        skipped = torch.randperm(tokens, generator=gen, device=device)[:case["skipped"]]
        slots[skipped] = -1
        st |= {"k": _activations((tokens, heads, dim), dtype, gen, device),
               "v": _activations((tokens, heads, dim), dtype, gen, device), "slots": slots,
               "cache": torch.zeros((blocks, heads, 18 * dim), dtype=torch.uint8, device=device),
               "k_out": torch.empty((tokens, heads, dim), dtype=dtype, device=device),
               "v_out": torch.empty((tokens, heads, dim), dtype=dtype, device=device), "layout": _layout(dim, device)}
    elif op == "int4_decode":
        dtype, heads, dim = DTYPES[case["dtype"]], case["kv_heads"], case["head_dim"]
        lens = _lengths(case)
        width = -(-int(lens.max()) // BLOCK)
        table, _, blocks = _tables(lens, 5, width, gen, device)
        layout = _layout(dim, device)
        cache = torch.empty((blocks * heads, 18 * dim), dtype=torch.uint8, device=device)
        step = max(1, (1 << 23) // (BLOCK * dim))
        for first in range(0, blocks * heads, step):
            n = min(step, blocks * heads - first)
            tile = torch.arange(first, first + n, device=device).repeat_interleave(BLOCK)
            token = torch.arange(BLOCK, device=device).repeat(n)
            for code_at, pair_at in (("kc", "kp"), ("vc", "vp")):
                _pack(_activations((n * BLOCK, dim), dtype, gen, device), cache, (tile, token), layout[code_at],
                      layout[pair_at])
        st |= {"cache": cache.view(blocks, heads, 18 * dim), "table": table,
               "lens": torch.from_numpy(lens).to(device=device, dtype=torch.int32),
               "q": torch.randn((case["seqs"], case["q_heads"], dim), generator=gen, device=device).to(dtype),
               "out": torch.empty((case["seqs"], case["q_heads"], dim), dtype=dtype, device=device),
               "layout": layout, "scale": dim ** -0.5}
    elif op == "latent_step":
        dtype, width = DTYPES[case["dtype"]], LATENT + ROPE
        lens = _lengths(case)
        table, _, blocks = _tables(lens, 5, -(-int(lens.max()) // BLOCK), gen, device)
        lens_d = torch.from_numpy(lens).to(device)
        last = lens_d - 1
        slots = table.gather(1, (last // BLOCK)[:, None])[:, 0].long() * BLOCK + last % BLOCK
        st |= {"cache": torch.randn((blocks, BLOCK, width), generator=gen, device=device).to(dtype), "table": table,
               "lens": lens_d.to(torch.int32), "slots": slots,
               "latent": torch.randn((case["seqs"], LATENT), generator=gen, device=device).to(dtype),
               "rope": torch.randn((case["seqs"], ROPE), generator=gen, device=device).to(dtype),
               "q": torch.randn((case["seqs"], case["heads"], width), generator=gen, device=device).to(dtype),
               "out": torch.empty((case["seqs"], case["heads"], LATENT), dtype=dtype, device=device),
               "scale": (128 + ROPE) ** -0.5}
    else:
        lens, new = _lengths(case), _new_tokens(case)
        total, tokens = -(-(lens + new) // BLOCK), int(new.sum())
        fresh = int((total - -(-lens // BLOCK)).sum())
        table, order, blocks = _tables(lens, fresh + 11, max(1, int(total.max())), gen, device)
        used = blocks - fresh - 11
        free = torch.full((blocks,), -1, dtype=torch.int32, device=device)
        free[:fresh + 11] = order[used:]
        st |= {"table": table, "lens": torch.from_numpy(lens).to(device=device, dtype=torch.int32),
               "new": torch.from_numpy(new).to(device=device, dtype=torch.int32), "free": free,
               "count": torch.tensor([fresh + 11], dtype=torch.int32, device=device), "tokens": tokens, "fresh": fresh,
               "slots": torch.empty(tokens + case["padding"], dtype=torch.int64, device=device),
               "new_lens": torch.empty(case["seqs"], dtype=torch.int32, device=device),
               "new_count": torch.empty(1, dtype=torch.int32, device=device)}
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(st):
    return {"int4_write": _int4_write, "int4_decode": _int4_decode, "latent_step": _latent_step,
            "tables": _block_tables}[st["case"]["op"]](st)


def _int4_write(st):
    if own:
        pkv = _library()
        pkv.reshape_and_cache_int4(st["k"], st["v"], st["cache"], st["slots"])
        pkv.gather_cache_int4(st["k_out"], st["v_out"], st["cache"], st["slots"])
        return {"k": st["k_out"], "v": st["v_out"]}
    case, lay, slots = st["case"], st["layout"], st["slots"]
    heads, dim, cache = case["kv_heads"], case["head_dim"], st["cache"]
    flat = cache.view(-1, 18 * dim)
    # a skipped token is sent to a row of its own behind the tiles
    tiles = flat.shape[0]
    wide = torch.cat((flat, flat.new_zeros((heads, 18 * dim))))
    tile = torch.where(slots < 0, tiles // heads, slots // BLOCK)[:, None] * heads + torch.arange(heads, device=flat.device)
    token = torch.where(slots < 0, 0, slots % BLOCK)[:, None].expand(-1, heads)
    at = (tile.flatten(), token.flatten())
    _pack(st["k"].flatten(0, 1), wide, at, lay["kc"], lay["kp"])
    _pack(st["v"].flatten(0, 1), wide, at, lay["vc"], lay["vp"])
    flat.copy_(wide[:tiles])
    live, dtype = (slots >= 0)[:, None, None], st["k"].dtype
    k = _read_rows(wide, at, lay["kc"], lay["kp"], dtype).view(st["k"].shape)
    v = _read_rows(wide, at, lay["vc"], lay["vp"], dtype).view(st["v"].shape)
    return {"k": k.masked_fill(~live, 0).to(dtype), "v": v.masked_fill(~live, 0).to(dtype)}


def _int4_decode(st):
    case = st["case"]
    if own:
        _library().paged_attention_decode_int4(st["out"], st["q"], st["cache"], st["table"], st["lens"], st["scale"],
                                               sliding_window=case["window"])
        return st["out"]
    lay, dtype = st["layout"], st["q"].dtype
    seqs, heads, dim = case["seqs"], case["kv_heads"], case["head_dim"]
    tiles = st["cache"][st["table"].clamp(min=0).long()].transpose(1, 2)          # [S, Hkv, blocks, 18 D]
    k = _unpack(tiles, lay["kc"], lay["kp"], dtype).flatten(2, 3)                 # [S, Hkv, positions, D]
    q = st["q"].float().view(seqs, heads, -1, dim)
    x = torch.matmul(q, k.transpose(2, 3)) * st["scale"]
    del k
    at, lens = torch.arange(x.shape[-1], device=x.device), st["lens"].long()[:, None]
    seen = at < lens
    if case["window"]:
        seen &= at >= lens - case["window"]
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    x = torch.exp(x - x.amax(-1, keepdim=True))
    p = x / x.sum(-1, keepdim=True)
    v = _unpack(tiles, lay["vc"], lay["vp"], dtype).flatten(2, 3)
    return torch.matmul(p, v).view(seqs, case["q_heads"], dim).to(dtype)


def _latent_step(st):
    case = st["case"]
    if own:
        pkv = _library()
        pkv.latent_cache_write(st["latent"], st["rope"], st["cache"], st["slots"])
        pkv.paged_latent_decode(st["out"], st["q"], st["cache"], st["table"], st["lens"], st["scale"])
        return {"out": st["out"], "cache": st["cache"]}
    cache = st["cache"]
    cache.view(-1, LATENT + ROPE)[st["slots"]] = torch.cat((st["latent"], st["rope"]), 1)
    rows = cache[st["table"].clamp(min=0).long()].flatten(1, 2).float()           # [S, positions, 576]
    x = torch.matmul(st["q"].float(), rows.transpose(1, 2)) * st["scale"]
    seen = torch.arange(rows.shape[1], device=rows.device) < st["lens"].long()[:, None]
    x = x.masked_fill(~seen[:, None], -math.inf)
    x = torch.exp(x - x.amax(-1, keepdim=True))
    p = x / x.sum(-1, keepdim=True)
    return {"out": torch.matmul(p, rows[..., :LATENT]).to(cache.dtype), "cache": cache}


def _block_tables(st):
    if own:
        _library().extend_block_tables(st["table"], st["lens"], st["new"], st["free"], st["count"], st["slots"],
                                       new_lens=st["new_lens"], new_free_count=st["new_count"])
        return {"table": st["table"], "lens": st["new_lens"], "slots": st["slots"], "count": st["new_count"]}
    table, lens, new = st["table"], st["lens"].long(), st["new"].long()
    seq = torch.arange(len(lens), device=table.device)
    have = (lens + BLOCK - 1) // BLOCK
    need = (lens + new + BLOCK - 1) // BLOCK - have
    rows = seq.repeat_interleave(need, output_size=st["fresh"])
    nth = torch.arange(st["fresh"], device=table.device)
    cols = have[rows] + nth - (need.cumsum(0) - need)[rows]
    table[rows, cols] = st["free"][st["count"].long() - 1 - nth]
    rows = seq.repeat_interleave(new, output_size=st["tokens"])
    pos = lens[rows] + torch.arange(st["tokens"], device=table.device) - (new.cumsum(0) - new)[rows]
    slots = torch.full_like(st["slots"], -1)
    slots[:st["tokens"]] = table[rows, pos // BLOCK].long() * BLOCK + pos % BLOCK
    return {"table": table, "lens": (lens + new).to(torch.int32), "slots": slots,
            "count": (st["count"] - need.sum()).to(torch.int32)}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_rows(tiles, which, dim, dtype):
    """float64 rows [n, 16, D] of tiles [n, 18 D], read element by element from the tile's definition."""
    code_at, pair_at = _code_bytes(dim)[which], _pair_bytes(dim)[which]
    raw = tiles.cpu().numpy()
    code = raw[:, code_at.reshape(-1)].reshape(len(raw), 16, dim // 2)
    x = np.empty((len(raw), 16, dim))
    x[..., 0::2], x[..., 1::2] = code & 15, code >> 4
    pair = torch.from_numpy(np.ascontiguousarray(raw[:, pair_at.reshape(-1)])).view(dtype).double().numpy()
    pair = pair.reshape(len(raw), 16, dim // GROUP, 2)
    return x * np.repeat(pair[..., 0], GROUP, -1) + np.repeat(pair[..., 1], GROUP, -1)


def _exact_attention(q, k, v, scale):
    """One KV head: q [g, D], k [n, D], v [n, E], float64."""
    x = (q @ k.T) * scale
    x = np.exp(x - x.max(1, keepdims=True))
    return (x / x.sum(1, keepdims=True)) @ v


def exact(case, seed):
    op = case["op"]
    if op == "tables":
        return None
    if op == "int4_decode":
        lens = _lengths(case)
        if int(lens.sum()) * case["kv_heads"] * case["head_dim"] > 100_000_000:
            return None
    if op == "latent_step" and int(_lengths(case).sum()) * (case["heads"] + 40) > 40_000_000:
        return None
    st = prepare(case, seed)
    if op == "int4_write":
        outs = {}
        dead = (st["slots"] < 0).cpu().numpy()
        for name in ("k", "v"):
            x = st[name].double().cpu().numpy().reshape(case["tokens"], case["kv_heads"], -1, GROUP)
            lo, hi = x.min(-1), x.max(-1)
            s = torch.from_numpy((hi - lo) / 15).to(st[name].dtype).double().numpy()[..., None]
            c = np.clip(np.rint((x - lo[..., None]) / np.where(s > 0, s, 1)), 0, 15) * (s > 0)
            y = (c * s + lo[..., None]).reshape(case["tokens"], case["kv_heads"], case["head_dim"])
            y[dead] = 0
            outs[name] = y
        return outs
    if op == "int4_decode":
        heads, dim, group = case["kv_heads"], case["head_dim"], case["q_heads"] // case["kv_heads"]
        q, table = st["q"].double().cpu().numpy(), st["table"].cpu()
        out = np.zeros((case["seqs"], case["q_heads"], dim))
        for s, n in enumerate(lens.tolist()):
            first = max(0, n - case["window"]) if case["window"] else 0
            ids = table[s, :-(-n // BLOCK)].long()
            tiles = st["cache"][ids.to(st["cache"].device)]
            for h in range(heads):
                k, v = (_exact_rows(tiles[:, h], w, dim, st["q"].dtype).reshape(-1, dim)[first:n] for w in (0, 1))
                out[s, h * group:(h + 1) * group] = _exact_attention(q[s, h * group:(h + 1) * group], k, v, st["scale"])
        return out
    q, table, slots = st["q"].double().cpu().numpy(), st["table"].cpu().numpy(), st["slots"].cpu().numpy()
    cache = st["cache"].double().cpu().numpy()
    new = np.concatenate((st["latent"].double().cpu().numpy(), st["rope"].double().cpu().numpy()), 1)
    for s, slot in enumerate(slots.tolist()):
        cache[slot // BLOCK, slot % BLOCK] = new[s]
    out = np.zeros((case["seqs"], case["heads"], LATENT))
    for s, n in enumerate(_lengths(case).tolist()):
        rows = cache[table[s, :-(-n // BLOCK)]].reshape(-1, LATENT + ROPE)[:n]
        out[s] = _exact_attention(q[s], rows, rows[:, :LATENT], st["scale"])
    return {"out": out, "cache": None}
