"""Up to 128 query heads a KV head: tiles of rows that no power of two fills, one token a tile, and more sequences and
groups than the kernels list in shared memory. Calls stay within the workspace that their size call names."""

import numpy as np
import pytest
import torch

import test_gpu_prompt as P
from paged_kv_cache_217_gb300 import binding as B
from test_gpu_prompt import _built  # noqa: F401

pytestmark = pytest.mark.gpu

GROUPS = [(17, 1), (66, 2), (43, 1), (64, 1), (65, 1), (71, 1), (200, 2), (127, 1), (128, 1)]


def some(hq):
    return sorted({0, hq // 2, hq - 1})


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv", GROUPS)
def test_prompts(hq, hkv, d):
    lens, new = [300, 0, 1, 2, 65, 130, 40], [5, 0, 1, 2, 65, 17, 1]
    c = P.Case(lens, new, hq, hkv, d, "bf16", seed=100)
    c.check(c.run(), heads=some(hq))
    c.check(c.run(window=33), window=33, heads=some(hq))
    c.check(c.run(causal=False), causal=False, heads=[hq - 1])


@pytest.mark.parametrize("hq,hkv", GROUPS)
def test_long_contexts(hq, hkv):
    c = P.Case([9001, 700], [3, 1], hq, hkv, 128, "f16", seed=101)
    c.check(c.run(), heads=some(hq))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv", GROUPS)
def test_prefixes(hq, hkv, d):
    c = P.prefix_case([330, 300, 321, 40, 700, 500, 501], hq, hkv, d, "f16", [0, 4, 6], [20, 30], seed=102)
    c.check(P.prefix_run(c), causal=False, heads=some(hq), tables=c.shared)


@pytest.mark.parametrize("seqs", [383, 384, 400, 1000])
@pytest.mark.parametrize("hq,hkv,d", [(16, 1, 128), (9, 1, 64), (4, 1, 256)])
def test_many_sequences(seqs, hq, hkv, d):
    """Segments up to, and beyond, what is kept in shared memory."""
    rng = np.random.default_rng(seqs)
    lens = rng.integers(0, 120, seqs)
    c = P.Case(lens, rng.integers(0, 4, seqs), hq, hkv, d, "bf16", seed=103)
    c.check(c.run(), heads=[hq - 1])
    starts, blocks = [3, 3, 100, 101, seqs - 7], [2, 5, 1, 4]
    for g, n in enumerate(blocks):
        lens[starts[g]] = max(lens[starts[g]], 16 * n + 3)
    p = P.prefix_case(lens, hq, hkv, d, "bf16", starts, blocks, seed=104)
    p.check(P.prefix_run(p), causal=False, heads=[hq - 1], tables=p.shared)


@pytest.mark.parametrize("seqs", [5, 100, 240, 500])
@pytest.mark.parametrize("hq,hkv,d", [(2, 2, 64), (8, 2, 128), (8, 2, 256), (71, 1, 128)])
def test_nothing_behind_the_workspace_is_written(seqs, hq, hkv, d):
    rng = np.random.default_rng(seqs + 1)
    lens = rng.integers(0, 150, seqs)
    lens[2] = 3000
    c = P.Case(lens, rng.integers(0, 3, seqs), hq, hkv, d, "bf16", seed=105)
    p = P.prefix_case(np.maximum(lens, 40), hq, hkv, d, "bf16", [0, seqs - 2], [2], seed=106)
    n = B.prompt_workspace_size(c.q.shape[0], seqs, hq, hkv, d, c.tables.shape[1])
    m = B.prefix_workspace_size(seqs, 1, hq, hkv, d, p.tables.shape[1])
    ws = torch.full((max(n, m) + 65536,), 0x5a, dtype=torch.uint8, device="cuda")
    want, behind = c.run(), P.prefix_run(p)
    assert torch.equal(torch.nan_to_num(c.run(workspace=ws[:n])), torch.nan_to_num(want))
    assert (ws[n:] == 0x5a).all()
    ws.fill_(0x5a)
    out = torch.empty_like(p.q)
    B.paged_prefix_decode(out, p.q, p.k, p.v, p.tables, p.lens, p.groups, p.blocks, p.scale, workspace=ws[:m])
    assert torch.equal(out, behind) and (ws[m:] == 0x5a).all()
