"""GPU parity where a decode grid joins the prompt kernels (at least 456 pairs of sequence and KV head): single
tokens in batches of prompts, what follows shared prefixes, and the calls run one behind the other as a model runs
them, eagerly, captured, and on two streams at once."""

import numpy as np
import pytest
import torch

import oracle.prompt as OP
import test_gpu_prompt as P
import test_gpu_rotary as R
from paged_kv_cache_217_gb300 import binding as B
from paged_kv_cache_217_gb300 import workloads as W
from test_gpu_prompt import _built  # noqa: F401

pytestmark = pytest.mark.gpu

HEADS = [(2, 2, 64), (4, 2, 128), (8, 2, 64), (10, 2, 128), (2, 2, 256), (16, 2, 256)]


def batch(seqs, top, seed, new):
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, top, seqs)
    lens[:8] = [0, 1, 15, 16, 17, 31, top - 1, top - 1]
    many = rng.choice(new, seqs)
    many[:8] = 1
    return lens, np.minimum(many, np.maximum(lens, 1))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hkv,d", HEADS)
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 1), (True, 33), (False, 0)])
def test_single_tokens_among_others(hq, hkv, d, causal, window, dtype):
    lens, new = batch(240, 210, 1, [0, 1, 1, 1, 2, 3])
    assert new.sum() < 480
    c = P.Case(lens, new, hq, hkv, d, dtype, seed=30, behind=2)
    out = c.run(causal, window)
    assert out[int(c.starts_np[-1]):].isnan().all()
    c.check(out, causal, window, heads=[0, hq - 1])


@pytest.mark.parametrize("seqs", [227, 228, 229])
@pytest.mark.parametrize("extra", [-1, 0])
def test_both_sides_of_the_rule(seqs, extra):
    """Sequences from where the grid is used on, and one token fewer than two a sequence or exactly two."""
    lens, _ = batch(seqs, 100, 2, [1])
    new = np.full(seqs, 2)
    new[3] += extra
    c = P.Case(np.maximum(lens, 2), new, 4, 2, 64, "bf16", seed=31)
    c.check(c.run(), heads=[1])


def test_a_padded_batch():
    """One prompt, one token of each of a few sequences, and places that hold no sequence."""
    lens, new = np.zeros(300, int), np.zeros(300, int)
    lens[:5], new[:5] = [900, 70, 16, 1, 300], [200, 1, 1, 1, 1]
    c = P.Case(lens, new, 8, 2, 128, "bf16", seed=32, extra_cols=2)
    c.check(c.run(), heads=[0, 7])


def test_long_single_tokens():
    lens = np.full(60, 40)
    lens[[3, 17]] = [5001, 3000]
    c = P.Case(lens, np.ones(60, int), 8, 8, 128, "f16", seed=33)
    c.check(c.run(), heads=[0, 7])
    c.check(c.run(window=500), window=500, heads=[3])


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("group", [1, 4])
def test_masked_rows_of_single_tokens_may_hold_anything(d, group):
    lens, new = batch(240, 120, 3, [1])
    c = P.Case(lens, new, 2 * group, 2, d, "bf16", seed=34)
    live = torch.zeros(c.k.shape[0], 16, dtype=torch.bool, device="cuda")
    for s, n in enumerate(lens):
        for p in range(n):
            live[int(c.tables_np[s, p // 16]), p % 16] = True
    want = c.run()
    for bad in (float("nan"), float("inf"), torch.finfo(torch.bfloat16).min):
        for x in (c.k, c.v):
            x.masked_fill_(~live[:, None, :, None], bad)
        assert torch.equal(c.run(), want)


def test_bad_tables_and_lengths_of_single_tokens_are_flagged():
    c = P.Case([40] * 240, [1] * 240, 4, 2, 128, "f16", seed=35)
    c.tables[7, 1] = c.k.shape[0]
    c.run()
    assert B.device_status(clear=True) == 0x1
    c = P.Case([40] * 240, [1] * 240, 4, 2, 128, "f16", seed=35)
    c.lens[9] = -4
    out = c.run()
    assert B.device_status(clear=True) == 0x2 and not out[9].any()


GROUPS = [([0, 240], [3]), ([5, 100, 100, 230], [2, 1, 5]), ([0], []), ([0, 1, 239], [0, 6])]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hkv,d", HEADS)
@pytest.mark.parametrize("starts,blocks", GROUPS)
def test_what_follows_prefixes(starts, blocks, hq, hkv, d, dtype):
    lens, new = batch(240, 150, 4, [1])
    for g, n in enumerate(blocks):                       # the first member has all of its prefix
        lens[starts[g]] = max(lens[starts[g]], 16 * n)
    c = P.prefix_case(lens, hq, hkv, d, dtype, starts, blocks, seed=36)
    c.check(P.prefix_run(c), causal=False, heads=[0, hq - 1], tables=c.shared)


def test_a_workspace_may_hold_anything():
    lens, new = batch(240, 150, 5, [0, 1, 1, 2])
    c = P.Case(lens, new, 4, 2, 128, "f16", seed=37)
    p = P.prefix_case(np.maximum(lens, 50), 4, 2, 128, "f16", [0, 200], [3], seed=38)
    n = max(B.prompt_workspace_size(c.q.shape[0], 240, 4, 2, 128, c.tables.shape[1]),
            B.prefix_workspace_size(240, 1, 4, 2, 128, p.tables.shape[1]))
    want, behind, ws = c.run(), P.prefix_run(p), torch.empty(n, dtype=torch.uint8, device="cuda")
    for fill in (0xff, 0x7f, 0):
        ws.fill_(fill)
        assert torch.equal(c.run(workspace=ws), want)
        ws.fill_(fill)
        out = torch.empty_like(p.q)
        B.paged_prefix_decode(out, p.q, p.k, p.v, p.tables, p.lens, p.groups, p.blocks, p.scale, workspace=ws)
        assert torch.equal(out, behind)
    assert B.device_status(clear=True) == 0


# ---- the calls of a model's step ---------------------------------------------------------------
class Step:
    """Sequences that share a prompt: its tokens rotated and written, attended, then one token of each sequence."""

    def __init__(self, seqs, seed, dtype="bf16", hq=8, hkv=2, d=128):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        dt = {"f16": torch.float16, "bf16": torch.bfloat16}[dtype]
        self.dtype, self.seqs, self.hq, self.hkv, self.d, self.prompt = dtype, seqs, hq, hkv, d, 64
        shared, own = self.prompt // 16, 2
        nb = shared + own * seqs + 1
        self.tables_np = np.concatenate((np.tile(np.arange(1, shared + 1), (seqs, 1)),
                                         shared + 1 + np.arange(own * seqs).reshape(seqs, own)), 1).astype(np.int32)
        self.lens_np = np.full(seqs, self.prompt + 1, np.int32)
        cuda = lambda x, t=torch.int32: torch.as_tensor(np.asarray(x), dtype=t, device="cuda")  # noqa: E731
        self.tables, self.lens, self.one = cuda(self.tables_np), cuda(self.lens_np), cuda([self.prompt])
        self.starts, self.groups, self.blocks = cuda([0, self.prompt]), cuda([0, seqs]), cuda([shared])
        self.positions = [cuda(np.arange(self.prompt)), cuda([self.prompt] * seqs)]
        self.slots = [cuda(np.arange(self.prompt) + 16, torch.int64), cuda(16 * (shared + 1 + own * np.arange(seqs)), torch.int64)]
        self.x = [torch.randn((n, hq + 2 * hkv, d), generator=gen, device="cuda").to(dt) for n in (self.prompt, seqs)]
        self.q = [torch.empty((n, hq, d), dtype=dt, device="cuda") for n in (self.prompt, seqs)]
        self.out = [torch.empty_like(q) for q in self.q]
        self.k, self.v = (torch.zeros((nb, hkv, 16, d), dtype=dt, device="cuda") for _ in range(2))
        self.angles = R.table(d)
        self.ws = [torch.empty(B.prompt_workspace_size(self.prompt, 1, hq, hkv, d, self.tables.shape[1]), dtype=torch.uint8, device="cuda"),
                   torch.empty(B.prefix_workspace_size(seqs, 1, hq, hkv, d, self.tables.shape[1]), dtype=torch.uint8, device="cuda")]

    def run(self):
        for i in range(2):
            q, k, v = self.x[i].split([self.hq, self.hkv, self.hkv], 1)
            B.rotary_and_cache(self.q[i], q, k, v, self.positions[i], self.angles, self.k, self.v, self.slots[i])
            if i == 0:
                B.paged_prompt_attention(self.out[0], self.q[0], self.k, self.v, self.tables[:1], self.one, self.starts,
                                         self.d ** -0.5, workspace=self.ws[0])
            else:
                B.paged_prefix_decode(self.out[1], self.q[1], self.k, self.v, self.tables, self.lens, self.groups,
                                      self.blocks, self.d ** -0.5, workspace=self.ws[1])

    def check(self):
        torch.cuda.synchronize()
        assert B.device_status(clear=True) == 0
        host = [W.to_numpy_storage(t, self.dtype) for t in (self.k, self.v)]
        for i in range(2):
            q, k, v = self.x[i].split([self.hq, self.hkv, self.hkv], 1)
            assert torch.equal(self.q[i], R.turned(q, self.positions[i], self.angles, False))
            at = self.slots[i]
            assert torch.equal(self.k[at // 16, :, at % 16], R.turned(k, self.positions[i], self.angles, False))
            assert torch.equal(self.v[at // 16, :, at % 16], v)
            n = self.prompt if i == 0 else self.seqs
            want, bound = OP.attention(W.to_numpy_storage(self.q[i], self.dtype), *host, self.tables_np[:1] if i == 0 else self.tables_np,
                                       self.lens_np[:1] - 1 if i == 0 else self.lens_np,
                                       np.array([0, n]) if i == 0 else np.arange(n + 1), self.d ** -0.5, self.dtype, i == 0)
            allowed = bound + P.HALF_STEP[self.dtype] * (np.abs(want) + bound) + P.TINY[self.dtype]
            assert (np.abs(self.out[i].double().cpu().numpy() - want) <= allowed).all()


@pytest.mark.parametrize("seqs", [5, 240])
def test_a_step(seqs):
    s = Step(seqs, 40)
    s.run()
    s.check()


@pytest.mark.parametrize("seqs", [5, 240])
def test_captured_steps_on_two_streams(seqs):
    """Two graphs with workspaces of their own, replayed at once, again with other inputs."""
    steps, graphs, streams = [Step(seqs, 41), Step(seqs, 42)], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in steps:
        s.run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.run()
        graphs.append(g)
    for again in range(3):
        for s, g, st in zip(steps, graphs, streams):
            for x in s.x:
                x.mul_(-0.9)
            for x in s.out + [s.k, s.v]:
                x.zero_()
        torch.cuda.synchronize()
        for s, g, st in zip(steps, graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        for s in steps:
            s.check()


def test_positions_past_32_bit_offsets():
    """Blocks behind 2^32 bytes of a pool, and rows of one behind 2^31 elements."""
    nb, hkv, d = 70000, 16, 128
    pools = [torch.zeros((nb, hkv, 16, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for new, seqs in ((1, 30), (3, 2)):
        lens = [50] * seqs
        c = P.Case(lens, [new] * seqs, hkv, hkv, d, "bf16", seed=43)
        at = nb - c.k.shape[0]
        for pool, x in zip(pools, (c.k, c.v)):
            pool[at:] = x
        want, out = c.run(), torch.empty_like(c.q)
        B.paged_prompt_attention(out, c.q, *pools, c.tables + at, c.lens, c.starts, c.scale)
        assert torch.equal(out, want)
    x = torch.randn((5, 3 * hkv, d), dtype=torch.bfloat16, device="cuda")
    slots = torch.arange(5, device="cuda") + 16 * (nb - 1)
    q, k, v = x.split(hkv, 1)
    B.rotary_and_cache(torch.empty_like(q.contiguous()), q, k, v, torch.zeros(5, dtype=torch.int32, device="cuda"), R.table(d), *pools, slots)
    assert torch.equal(pools[0][-1, :, :5].transpose(0, 1), k) and torch.equal(pools[1][-1, :, :5].transpose(0, 1), v)
    assert B.device_status(clear=True) == 0
