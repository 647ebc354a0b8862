"""Cases of prompt and cross attention over the paged cache, of decode attention that computes a shared
prefix once for a group, and of the cache write that rotates by position on its way.

Four kinds of case, each one pass as a serving loop makes it:

* ``rotary`` -- a step's queries and keys are rotated by their positions; the keys, and the values as they
  are, go to their slots of the paged cache.
* ``prompt`` -- several query tokens per sequence, the last of its context, attend causally over the paged
  cache (whole prompts, chunks of long ones, drafted tokens to be verified), within a window or not.
* ``cross``  -- every query token attends over all states of its sequence's encoder, kept in pages.
* ``prefix`` -- one query token per sequence; the sequences of a group hold the same first blocks.

``own`` chooses between this file's plain forms (elementary torch operations in 32 bits, rounded once at
the end) and the library's calls.
"""

import math

import numpy as np
import torch

own = False

BLOCK = 16  # tokens per block
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def _library():
    import paged_kv_cache_217_gb300 as pkv
    return pkv


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # a decode step of 64 sequences in a 40-head layer: launch latency counts
        {"name": "rotary_step", "op": "rotary", "dtype": "bf16", "tokens": 64, "q_heads": 40, "kv_heads": 40,
         "head_dim": 128, "rotary_dim": 128, "interleaved": False, "skipped": 0},
        # a prompt step of several requests packed together, padded at the end; half of each head is rotated, in pairs
        {"name": "rotary_partial", "op": "rotary", "dtype": "f16", "tokens": 2999, "q_heads": 16, "kv_heads": 16,
         "head_dim": 256, "rotary_dim": 64, "interleaved": True, "skipped": 57},
        # the same of a layer with 32 query heads on 8 KV heads, a full batch of prompts
        {"name": "rotary_prompt", "op": "rotary", "dtype": "bf16", "tokens": 12301, "q_heads": 32, "kv_heads": 8,
         "head_dim": 128, "rotary_dim": 128, "interleaved": False, "skipped": 211},
        # five drafted tokens each of eight chats are verified: latency, the context has to be split
        {"name": "prompt_verify", "op": "prompt", "dtype": "bf16", "seqs": 8, "new": 5, "new_spread": 0.0, "cached": 1400,
         "cached_spread": 0.6, "max_len": 8192, "q_heads": 32, "kv_heads": 8, "head_dim": 128, "window": 0},
        # whole short prompts of 64 chats
        {"name": "prompt_chats", "op": "prompt", "dtype": "bf16", "seqs": 64, "new": 150, "new_spread": 0.6, "cached": 0,
         "cached_spread": 0.0, "max_len": 1024, "q_heads": 32, "kv_heads": 8, "head_dim": 128, "window": 0},
        # prompts on sliding-window layers with wide heads, the last chunk of each
        {"name": "prompt_window", "op": "prompt", "dtype": "bf16", "seqs": 4, "new": 2000, "new_spread": 0.3, "cached": 1500,
         "cached_spread": 0.3, "max_len": 8192, "q_heads": 16, "kv_heads": 8, "head_dim": 256, "window": 1024},
        # a chunk of one long document in a 96-head layer: bound by the matrix products
        {"name": "prompt_chunk", "op": "prompt", "dtype": "f16", "seqs": 1, "new": 2048, "new_spread": 0.0, "cached": 15953,
         "cached_spread": 0.0, "max_len": 32768, "q_heads": 96, "kv_heads": 96, "head_dim": 128, "window": 0},
        # a decoder's single-token step over its encoder's states, 20 heads of 64
        {"name": "cross_step", "op": "cross", "dtype": "f16", "seqs": 24, "new": 1, "new_spread": 0.0, "states": 1500,
         "states_spread": 0.0, "max_len": 1500, "q_heads": 20, "kv_heads": 20, "head_dim": 64},
        # decoder prompts over encoder states of other lengths
        {"name": "cross_prompt", "op": "cross", "dtype": "bf16", "seqs": 32, "new": 224, "new_spread": 0.4, "states": 900,
         "states_spread": 0.5, "max_len": 4096, "q_heads": 16, "kv_heads": 16, "head_dim": 64},
        # four samples of one short prompt: the smallest decode
        {"name": "prefix_few", "op": "prefix", "dtype": "bf16", "groups": 1, "seqs": 4, "prefix": 512, "tail": 60,
         "tail_spread": 0.5, "q_heads": 32, "kv_heads": 8, "head_dim": 128},
        # 64 requests behind one system prompt, 40 heads with their own K/V
        {"name": "prefix_mha", "op": "prefix", "dtype": "f16", "groups": 1, "seqs": 64, "prefix": 2000, "tail": 200,
         "tail_spread": 0.6, "q_heads": 40, "kv_heads": 40, "head_dim": 128},
        # 256 requests on two long documents, 32 query heads on 8 KV heads
        {"name": "prefix_documents", "op": "prefix", "dtype": "bf16", "groups": 2, "seqs": 256, "prefix": 8192, "tail": 150,
         "tail_spread": 0.6, "q_heads": 32, "kv_heads": 8, "head_dim": 128},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "prompt", "prompt", "prompt", "cross", "prefix", "prefix"])
    dtype = rng.choice(["f16", "bf16"])
    if op == "rotary":
        dim = rng.choice([64, 128, 128, 256])
        kv, group = rng.choice([1, 2, 3, 5, 8, 16, 40]), rng.choice([1, 1, 2, 4, 5, 8])
        most = 12301 * 48 * 128 // (kv * (group + 2) * dim)
        tokens = _log_int(rng, 1, max(1, most))
        return {"op": op, "dtype": dtype, "tokens": tokens, "q_heads": kv * group, "kv_heads": kv, "head_dim": dim,
                "rotary_dim": rng.choice([r for r in (16, 32, 64, 96, 128, 256) if r <= dim] + [dim, dim]),
                "interleaved": rng.random() < 0.4, "skipped": rng.choice([0, tokens // 7, tokens // 2])}
    if op == "prefix":
        while True:
            dim, kv, group = rng.choice([64, 128, 128, 256]), rng.choice([1, 2, 3, 8, 12, 40]), rng.choice([1, 1, 2, 4, 5, 8])
            groups = rng.choice([1, 1, 1, 2, 3, 7])
            seqs, prefix, tail = _log_int(rng, max(2, groups), 300), _log_int(rng, 1, 16000), _log_int(rng, 1, 2000)
            spread = rng.choice([0.0, 0.4, 0.8])
            held = seqs * (prefix + tail * (1 + 2 * spread))
            if held * kv * group <= 60_000_000 and held * kv * dim <= 2_200_000_000 and kv * group <= 128:
                break
        return {"op": op, "dtype": dtype, "groups": groups, "seqs": seqs, "prefix": prefix, "tail": tail,
                "tail_spread": spread, "q_heads": kv * group, "kv_heads": kv, "head_dim": dim}
    while True:
        dim, kv, group = rng.choice([64, 128, 128, 256]), rng.choice([1, 2, 3, 5, 8, 20, 96]), rng.choice([1, 1, 2, 3, 4, 7, 8])
        seqs, new, there = _log_int(rng, 1, 200), _log_int(rng, 1, 3000), rng.choice([0, _log_int(rng, 1, 16000)])
        spread = rng.choice([0.0, 0.4, 0.8])
        if op == "cross":
            there = max(1, there)
        wide, tall = (there + new) * (1 + 2 * spread), new * (1 + 2 * spread)
        if kv * group <= 96 and seqs * tall * wide * kv * group * max(1, dim // 128) <= 3_300_000_000 and seqs * wide * kv * dim <= 1_000_000_000:
            break
    case = {"op": op, "dtype": dtype, "seqs": seqs, "new": new, "new_spread": spread, "q_heads": kv * group, "kv_heads": kv,
            "head_dim": dim}
    if op == "cross":
        return case | {"states": there, "states_spread": rng.choice([0.0, spread]),
                       "max_len": max(16, int(there * (1 + 2 * spread))) + rng.randrange(64)}
    return case | {"cached": there, "cached_spread": rng.choice([0.0, spread]),
                   "max_len": max(16, int(wide)) + rng.randrange(64),
                   "window": rng.choice([0, 0, 0, _log_int(rng, 1, 4096)])}


def _lognormal(rng, median, spread, n, most):
    if median == 0:
        return np.zeros(n, np.int64)
    return np.clip(np.rint(np.exp(rng.normal(math.log(median), spread, n))), 1, most).astype(np.int64)


def _shape(case):
    """(query tokens, context tokens) per sequence; they are part of the case, not of its seed."""
    if case["op"] == "prefix":
        rng = np.random.default_rng(case["seqs"] * 7919 + case["prefix"])
        tail = _lognormal(rng, case["tail"], case["tail_spread"], case["seqs"], 3 * case["tail"])
        return np.ones(case["seqs"], np.int64), case["prefix"] + tail
    rng = np.random.default_rng(case["seqs"] * 7919 + case["new"])
    if case["op"] == "cross":
        new = _lognormal(rng, case["new"], case["new_spread"], case["seqs"], int(case["new"] * (1 + 2 * case["new_spread"])))
        return new, _lognormal(rng, case["states"], case["states_spread"], case["seqs"], case["max_len"])
    new = _lognormal(rng, case["new"], case["new_spread"], case["seqs"], min(case["max_len"], int(case["new"] * (1 + 2 * case["new_spread"])) + 1))
    cached = _lognormal(rng, case["cached"], case["cached_spread"], case["seqs"], case["max_len"])
    return new, np.minimum(new + cached, np.maximum(new, case["max_len"]))


def _groups(case):
    """First sequence of each group, and the end of the last."""
    return np.linspace(0, case["seqs"], case["groups"] + 1).round().astype(np.int64)


def _pairs(new, lens, window):
    """Visible (query, key) pairs of causal attention, and the keys that some query sees."""
    pairs = keys = 0
    for n, length in zip(new.tolist(), lens.tolist()):
        seen = np.arange(length - n + 1, length + 1)
        if window:
            seen = np.minimum(seen, window)
        pairs += int(seen.sum())
        keys += length if not window else length - max(0, length - n + 1 - window)
    return pairs, keys


def work(case):
    dim, hq, hkv = case["head_dim"], case["q_heads"], case["kv_heads"]
    if case["op"] == "rotary":
        live = case["tokens"] - case["skipped"]
        q, kv = case["tokens"] * hq * dim * 4, live * hkv * dim * 8
        # a position and a slot of each token, the cosines and sines of each position
        return {"bytes": q + kv + case["tokens"] * (12 + 4 * case["rotary_dim"]),
                "flops": (case["tokens"] * hq + live * hkv) * case["rotary_dim"] * 3}
    new, lens = _shape(case)
    io = int(new.sum()) * hq * dim * 4
    if case["op"] == "prompt":
        pairs, keys = _pairs(new, lens, case["window"])
    elif case["op"] == "cross":
        pairs, keys = int((new * lens).sum()), int(lens.sum())
    else:
        shared = case["prefix"] // BLOCK * BLOCK
        pairs, keys = int(lens.sum()), int((lens - shared).sum()) + case["groups"] * shared
    return {"bytes": io + keys * hkv * dim * 4 + keys // BLOCK * 4 + case["seqs"] * 8, "flops": 4 * pairs * hq * dim}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _activations(shape, dtype, gen, device):
    """N(0, 1) values whose last dimension's channels differ in size, as K and V channels do."""
    x = torch.randn(shape, generator=gen, device=device)
    size = torch.exp(0.4 * torch.randn(shape[-1:], generator=gen, device=device))
    return (x * size).to(dtype)


def _tables(lens, gen, device):
    """Block tables over a shuffled pool, padded with -1, and the pool's blocks."""
    counts = -(-lens // BLOCK)
    blocks, width = int(counts.sum()) + 5, max(1, int(counts.max()))
    order = torch.randperm(blocks, generator=gen, device=device).to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device=device)
    rows = np.repeat(np.arange(len(lens)), counts)
    cols = np.arange(len(rows)) - np.repeat(np.cumsum(counts) - counts, counts)
    table[torch.from_numpy(rows).to(device), torch.from_numpy(cols).to(device)] = order[:len(rows)]
    return table, blocks


def prepare(case, seed):
    device = torch.device("cuda")
    gen = torch.Generator(device=device)
    gen.manual_seed(int(seed) * 2 + 1)
    dtype, dim, hq, hkv = DTYPES[case["dtype"]], case["head_dim"], case["q_heads"], case["kv_heads"]
    st = {"case": case}
    if case["op"] == "rotary":
        tokens, rot = case["tokens"], case["rotary_dim"]
        blocks = -(-tokens // BLOCK) + 3
        slots = torch.randperm(blocks * BLOCK, generator=gen, device=device)[:tokens]
        slots[torch.randperm(tokens, generator=gen, device=device)[:case["skipped"]]] = -1
        # prompts of random lengths one behind the other, their positions anywhere in a long context
        positions = (torch.arange(tokens, device=device) + torch.randint(0, 30000, (1,), generator=gen, device=device)) % 32768
        # the table that a model keeps: cos, then sin, of position x frequency
        angle = torch.outer(torch.arange(32768, device=device, dtype=torch.float64),
                            10000.0 ** (-torch.arange(0, rot, 2, device=device, dtype=torch.float64) / rot))
        # one projection's output, sliced
        qkv = _activations((tokens, hq + 2 * hkv, dim), dtype, gen, device)
        # (one block behind the pool, where the plain form sends the tokens that are skipped)
        k_all = torch.zeros((blocks + 1, hkv, BLOCK, dim), dtype=dtype, device=device)
        v_all = torch.zeros_like(k_all)
        return st | {"q": qkv[:, :hq], "k": qkv[:, hq:hq + hkv], "v": qkv[:, hq + hkv:], "slots": slots,
                     "positions": positions.to(torch.int32), "cos_sin": torch.cat((angle.cos(), angle.sin()), 1).float(),
                     "k_all": k_all, "v_all": v_all, "k_pool": k_all[:blocks], "v_pool": v_all[:blocks],
                     "q_out": torch.empty((tokens, hq, dim), dtype=dtype, device=device)}
    new, lens = _shape(case)
    held = lens
    if case["op"] == "prefix":
        shared, starts = case["prefix"] // BLOCK, _groups(case)
        held = lens - shared * BLOCK                      # own blocks; a group's first sequence holds the prefix too
        held[starts[:-1]] += shared * BLOCK
    table, blocks = _tables(held, gen, device)
    if case["op"] == "prefix":
        wide = torch.full((case["seqs"], -(-int(lens.max()) // BLOCK)), -1, dtype=torch.int32, device=device)
        wide[:, :table.shape[1]] = table[:, :wide.shape[1]]
        first = torch.from_numpy(np.repeat(starts[:-1], np.diff(starts))).to(device)
        rest = first != torch.arange(case["seqs"], device=device)
        moved = torch.cat((table[first][:, :shared], table), 1)[:, :wide.shape[1]]
        wide[rest, :moved.shape[1]] = moved[rest]
        table = wide
        st |= {"group_starts": torch.from_numpy(starts).to(device=device, dtype=torch.int32),
               "prefix_blocks": torch.full((case["groups"],), shared, dtype=torch.int32, device=device)}
    ends = np.cumsum(new)
    tokens = int(ends[-1])
    return st | {"table": table, "lens": torch.from_numpy(lens).to(device=device, dtype=torch.int32),
                 "k_pool": _activations((blocks, hkv, BLOCK, dim), dtype, gen, device),
                 "v_pool": _activations((blocks, hkv, BLOCK, dim), dtype, gen, device),
                 "q": torch.randn((tokens, hq, dim), generator=gen, device=device).to(dtype),
                 "starts": torch.from_numpy(np.concatenate(([0], ends))).to(device=device, dtype=torch.int32),
                 # of each query token: its sequence, and its place there
                 "row": torch.from_numpy(np.repeat(np.arange(len(new)), new)).to(device),
                 "place": torch.from_numpy(np.arange(tokens) - np.repeat(ends - new, new)).to(device),
                 "most": int(new.max()), "out": torch.empty((tokens, hq, dim), dtype=dtype, device=device),
                 "scale": dim ** -0.5}


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(st):
    op = st["case"]["op"]
    if op == "rotary":
        return _rotary(st)
    if own:
        pkv = _library()
        if op == "prefix":
            pkv.paged_prefix_decode(st["out"], st["q"], st["k_pool"], st["v_pool"], st["table"], st["lens"],
                                    st["group_starts"], st["prefix_blocks"], st["scale"])
        else:
            pkv.paged_prompt_attention(st["out"], st["q"], st["k_pool"], st["v_pool"], st["table"], st["lens"],
                                       st["starts"], st["scale"], causal=op == "prompt",
                                       sliding_window=st["case"].get("window", 0))
        return st["out"]
    return _attention(st)


def _rotary(st):
    if own:
        _library().rotary_and_cache(st["q_out"], st["q"], st["k"], st["v"], st["positions"], st["cos_sin"], st["k_pool"],
                                    st["v_pool"], st["slots"], interleaved=st["case"]["interleaved"])
        return {"q": st["q_out"], "k": st["k_pool"], "v": st["v_pool"]}
    rot, pairs, slots = st["case"]["rotary_dim"], st["case"]["interleaved"], st["slots"]
    cos, sin = st["cos_sin"][st["positions"].long()][:, None].chunk(2, -1)

    def turn(x):
        f = x.float()
        a, b = (f[..., 0:rot:2], f[..., 1:rot:2]) if pairs else (f[..., :rot // 2], f[..., rot // 2:rot])
        y = (a * cos - b * sin, b * cos + a * sin)
        y = torch.stack(y, -1).flatten(-2) if pairs else torch.cat(y, -1)
        return torch.cat((y, f[..., rot:]), -1).to(x.dtype)

    slots = torch.where(slots < 0, st["k_pool"].shape[0] * BLOCK, slots)
    st["k_all"][slots // BLOCK, :, slots % BLOCK] = turn(st["k"])
    st["v_all"][slots // BLOCK, :, slots % BLOCK] = st["v"]
    return {"q": turn(st["q"]), "k": st["k_pool"], "v": st["v_pool"]}


def _attention(st):
    """softmax(scale q k + mask) v over the pages, every sequence padded to the longest of the batch."""
    case, q, lens, table = st["case"], st["q"], st["lens"].long(), st["table"]
    seqs, most, dim, hq, hkv = case["seqs"], st["most"], case["head_dim"], case["q_heads"], case["kv_heads"]
    ids = table.clamp(min=0).long()
    k = st["k_pool"][ids].transpose(1, 2).flatten(2, 3).float()                       # [S, Hkv, positions, D]
    wide = torch.zeros((seqs, most, hq, dim), dtype=torch.float32, device=q.device)
    wide[st["row"], st["place"]] = q.float()
    wide = wide.view(seqs, most, hkv, -1, dim).permute(0, 2, 3, 1, 4).reshape(seqs, hkv, -1, dim)
    x = torch.matmul(wide, k.transpose(2, 3)).mul_(st["scale"]).view(seqs, hkv, -1, most, k.shape[2])
    del k
    at = torch.arange(x.shape[-1], device=q.device)
    seen = at < lens[:, None, None]
    if case["op"] == "prompt":
        new = (st["starts"][1:] - st["starts"][:-1]).long()[:, None]
        place = (lens[:, None] - new + torch.arange(most, device=q.device))[..., None]    # position of each query
        seen = seen & (at <= place)
        if case["window"]:
            seen &= at > place - case["window"]
    x.masked_fill_(~seen[:, None, None], -math.inf)
    x.sub_(x.amax(-1, keepdim=True).clamp_(min=-1e38)).exp_()
    x.div_(x.sum(-1, keepdim=True).clamp_(min=1e-38))
    v = st["v_pool"][ids].transpose(1, 2).flatten(2, 3).float()
    y = torch.matmul(x.flatten(2, 3), v).view(seqs, hkv, -1, most, dim)
    y = y.permute(0, 3, 1, 2, 4).reshape(seqs, most, hq, dim)
    return y[st["row"], st["place"]].to(q.dtype)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_rotary(st):
    case, rot = st["case"], st["case"]["rotary_dim"]
    table = st["cos_sin"].double().cpu().numpy()[st["positions"].cpu().numpy()]
    factor = table[:, :rot // 2] + 1j * table[:, rot // 2:]

    def turn(x):
        y = x.double().cpu().numpy().copy()
        first = slice(0, rot, 2) if case["interleaved"] else slice(0, rot // 2)
        second = slice(1, rot, 2) if case["interleaved"] else slice(rot // 2, rot)
        z = (y[..., first] + 1j * y[..., second]) * factor[:, None]
        y[..., first], y[..., second] = z.real, z.imag
        return y

    pools = {}
    slots = st["slots"].cpu().numpy()
    for name, rows in (("k", turn(st["k"])), ("v", st["v"].double().cpu().numpy())):
        pool = np.zeros(tuple(st["k_pool"].shape))
        live = slots >= 0
        pool[slots[live] // BLOCK, :, slots[live] % BLOCK] = rows[live]
        pools[name] = pool
    return {"q": turn(st["q"]), **pools}


def exact(case, seed):
    if case["op"] == "rotary":
        return _exact_rotary(prepare(case, seed))
    # (64-bit products at about 1e12 operations a second)
    if work(case)["flops"] * (2 if case["op"] == "prompt" else 1) > 5e12:
        return None
    st = prepare(case, seed)
    new, lens = _shape(case)
    group, dim = case["q_heads"] // case["kv_heads"], case["head_dim"]
    out = torch.empty(st["out"].shape, dtype=torch.float64, device=st["q"].device)
    begin, window = 0, case.get("window", 0)
    for s, (n, length) in enumerate(zip(new.tolist(), lens.tolist())):
        ids = st["table"][s, :-(-length // BLOCK)].long()
        k, v = (st[p][ids].transpose(0, 1).reshape(case["kv_heads"], -1, dim)[:, :length] for p in ("k_pool", "v_pool"))
        for h in range(case["kv_heads"]):
            q = st["q"][begin:begin + n, h * group:(h + 1) * group].double()
            x = torch.einsum("ngd,ld->gnl", q, k[h].double()) * st["scale"]
            if case["op"] == "prompt":
                behind = torch.arange(length - n, length, device=x.device)[:, None] - torch.arange(length, device=x.device)
                x[:, (behind < 0) | (behind >= (window or length))] = -math.inf
            out[begin:begin + n, h * group:(h + 1) * group] = torch.einsum("gnl,ld->ngd", torch.softmax(x, -1), v[h].double())
        begin += n
    return out
