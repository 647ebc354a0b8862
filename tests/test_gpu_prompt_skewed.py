"""A few single tokens, or rests behind prefixes, far longer than the batch's others: the decode grid leaves them to
the prompt kernels, which cut them. Values at, below and above the length from which that is so."""

import numpy as np
import pytest
import torch

import test_gpu_prompt as P
from paged_kv_cache_217_gb300 import binding as B
from test_gpu_prompt import _built  # noqa: F401

pytestmark = pytest.mark.gpu

HEADS = [(2, 2, 64), (4, 2, 128), (10, 2, 128), (2, 2, 256), (16, 2, 256)]
SHORT = 1024                                  # up to here no token is long


def lengths(seqs, long, seed=0):
    lens = np.random.default_rng(seed).integers(0, 9, seqs)
    lens[[3, 9, seqs - 1]] = long
    return lens


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hkv,d", HEADS)
@pytest.mark.parametrize("long", [(SHORT, 700, 1), (SHORT + 1, SHORT, SHORT - 1), (9000, SHORT + 1, 5)])
def test_single_tokens(long, hq, hkv, d, dtype):
    c = P.Case(lengths(240, long), [1] * 240, hq, hkv, d, dtype, seed=110, behind=3)
    out = c.run()
    assert out[240:].isnan().all()
    c.check(out, heads=[0, hq - 1])
    c.check(c.run(causal=False), causal=False, heads=[hq - 1])


@pytest.mark.parametrize("hq,hkv,d", HEADS)
@pytest.mark.parametrize("window", [5, SHORT, SHORT + 1, 3000])
def test_windows(window, hq, hkv, d):
    """What counts is what a token sees."""
    c = P.Case(lengths(240, (9000, 3001, 1030)), [1] * 240, hq, hkv, d, "bf16", seed=111)
    for s, n in enumerate(c.lens_np):
        c.tables[s, :max(0, int(n) - window) // 16] = -1
    c.check(c.run(window=window), window=window, heads=[0, hq - 1])


@pytest.mark.parametrize("seqs", [240, 500])
def test_among_prompts(seqs):
    lens, new = lengths(seqs, (5000, 2000, 1500)), np.ones(seqs, int)
    new[[0, 5, 9, 20]] = [0, 3, 200, 90]
    lens[20] = 100
    c = P.Case(lens, new, 4, 2, 128, "bf16", seed=112)
    c.check(c.run(), heads=[0, 3], wanted=set(range(0, int(new.sum()), 3)) | {3, 4, 5, 6, 7, 8})


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hkv,d", HEADS)
@pytest.mark.parametrize("starts,blocks", [([0, 100, 238], [3, 70]), ([20], [])])
def test_behind_prefixes(starts, blocks, hq, hkv, d, dtype):
    seqs = 500 if hkv == 1 else 240
    lens = lengths(seqs, (48 + SHORT, 48 + SHORT + 1, 7000))
    lens[120] = 70 * 16 + SHORT + 1
    lens[[0, 100]] = [50, 70 * 16]
    c = P.prefix_case(lens, hq, hkv, d, dtype, starts, blocks, seed=113)
    out = P.prefix_run(c)
    c.check(out, causal=False, heads=[0, hq - 1], tables=c.shared)
    for fill in (0xff, 0):
        ws = torch.full((B.prefix_workspace_size(seqs, len(blocks), hq, hkv, d, c.tables.shape[1]),), fill, dtype=torch.uint8,
                        device="cuda")
        again = torch.empty_like(c.q)
        B.paged_prefix_decode(again, c.q, c.k, c.v, c.tables, c.lens, c.groups, c.blocks, c.scale, workspace=ws)
        assert torch.equal(again, out)


@pytest.mark.parametrize("seqs", [500, 3000, 9001])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 2)])
@pytest.mark.parametrize("at", [(0, 1, -1), (-1,), (0,), (400, 401, 2), (3,)])
def test_few_among_thousands(at, hq, hkv, seqs):
    """More than are listed in shared memory, long runs of which the grid takes; prompts among them, too."""
    lens = np.random.default_rng(seqs).integers(0, 12, seqs)
    new = np.ones(seqs, int)
    new[7::1000] = 5
    for i in at:
        lens[i] = 2500
    c = P.Case(lens, new, hq, hkv, 64, "bf16", seed=115)
    rows = set(range(0, int(new.sum()), 37)) | {int(c.starts_np[i % seqs]) for i in at} | {int(c.starts_np[7]) + i for i in range(5)}
    c.check(c.run(), heads=[hq - 1], wanted=rows)
    held = lens.copy()
    held[10] = 64
    p = P.prefix_case(held, hq, hkv, 64, "bf16", [10, seqs - 5], [3], seed=116)
    p.check(P.prefix_run(p), causal=False, heads=[0], tables=p.shared, wanted=set(range(0, seqs, 41)) | {i % seqs for i in at})


def test_replayed_with_other_lengths():
    """A captured call: which tokens are long is read on the GPU."""
    seqs = 240
    c = P.Case(np.full(seqs, 3000), [1] * seqs, 4, 2, 128, "bf16", seed=114)
    out = torch.empty_like(c.q)
    ws = torch.empty(B.prompt_workspace_size(seqs, seqs, 4, 2, 128, c.tables.shape[1]), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.paged_prompt_attention(out, c.q, c.k, c.v, c.tables, c.lens, c.starts, c.scale, workspace=ws)
    for long in ((3000, 2000, 1), (0, 1025, 1024), (10, 20, 30)):
        c.lens_np = lengths(seqs, long).astype(np.int32)
        c.lens.copy_(torch.from_numpy(c.lens_np))
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        c.check(out, heads=[3])
    c.lens_np = np.full(seqs, 3000, np.int32)
    c.lens.fill_(3000)
    graph.replay()
    torch.cuda.synchronize()
    c.check(out, heads=[0], wanted=set(range(0, seqs, 17)))
