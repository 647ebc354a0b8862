"""Groups whose members are all shorter than their prefix, as samples are right after a fork: what lies behind the
longest member may hold anything, and its blocks' table entries are not read."""

import numpy as np
import pytest
import torch

import oracle.prompt as OP
import test_gpu_prompt as P
from paged_kv_cache_217_gb300 import binding as B
from test_gpu_prompt import _built  # noqa: F401

pytestmark = pytest.mark.gpu

HEADS = [(2, 2, 64), (4, 2, 128), (6, 2, 256), (10, 2, 128)]
GROUPS = [  # lengths, group starts, prefix blocks
    ([40, 17, 33, 40], [0, 4], [3]),
    ([1, 0, 5], [0, 3], [7]),
    ([0, 0], [0, 2], [4]),
    ([600, 40, 30, 35, 170], [1, 4], [20]),              # an ordinary sequence on each side
    ([300, 200, 31, 5, 16, 700, 900], [0, 3, 5, 7], [30, 2, 60]),
    ([1000] * 3, [0, 3], [200]),                         # cut into pieces
]


def wide(seqs, seed):
    """Three groups of many, the first member not the longest, and some sequences by themselves."""
    lens = np.random.default_rng(seed).integers(0, 60, seqs)
    return lens, [0, seqs // 2, seqs // 2 + 9, seqs - 20], [4, 9, 5]


class Unseen:
    def __init__(self, lens, starts, blocks, hq, hkv, d, dtype, seed=50):
        lens, held, top = np.asarray(lens), np.array(lens), [0] * len(lens)
        for i, n in enumerate(blocks):                   # a group's first member holds the blocks that its longest sees
            lo, hi = starts[i], starts[i + 1]
            assert lens[lo:hi].max() <= 16 * n
            held[lo:hi] = 0
            held[lo] = lens[lo:hi].max()
        c = self.c = P.Case(held, [1] * len(lens), hq, hkv, d, dtype, seed=seed, extra_cols=max(blocks))
        c.lens_np = lens.astype(np.int32)
        c.lens.copy_(torch.from_numpy(c.lens_np))
        c.groups, c.blocks = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (starts, blocks))
        c.shared = OP.prefix_tables(c.tables_np, starts, blocks)
        self.live = torch.zeros(c.k.shape[0], 16, dtype=torch.bool, device="cuda")
        for s, n in enumerate(held):
            at = np.arange(n)
            self.live[torch.from_numpy(c.tables_np[s, at // 16]).long(), torch.from_numpy(at % 16)] = True

    def check(self, hq):
        clean = P.prefix_run(self.c)
        assert B.device_status(clear=True) == 0
        for bad in (float("nan"), float("inf"), torch.finfo(self.c.k.dtype).min):
            for x in (self.c.k, self.c.v):
                x.masked_fill_(~self.live[:, None, :, None], bad)
            assert torch.equal(P.prefix_run(self.c), clean)
            self.c.check(clean, causal=False, heads=[0, hq - 1], tables=self.c.shared)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hkv,d", HEADS)
@pytest.mark.parametrize("lens,starts,blocks", GROUPS)
def test_members_shorter_than_their_prefix(lens, starts, blocks, hq, hkv, d, dtype):
    Unseen(lens, starts, blocks, hq, hkv, d, dtype).check(hq)


@pytest.mark.parametrize("seqs", [100, 240, 700])
@pytest.mark.parametrize("hq,hkv,d", HEADS)
def test_wide_groups_shorter_than_their_prefix(seqs, hq, hkv, d):
    """Below and above the pairs from which a decode grid takes what follows the prefixes, and more members than a
    block of rows."""
    Unseen(*wide(seqs, seqs), hq, hkv, d, "bf16", seed=51).check(hq)
