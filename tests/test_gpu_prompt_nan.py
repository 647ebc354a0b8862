"""A query that holds NaN gets NaN, and no other row does, however its work is cut, split or shared with a decode grid."""

import numpy as np
import pytest
import torch

import test_gpu_prompt as P
from test_gpu_prompt import _built  # noqa: F401

pytestmark = pytest.mark.gpu


def check(c, run, rows, head):
    clean = run()
    assert clean.isfinite().all()
    c.q[rows, head, 3] = float("nan")
    bad = torch.zeros(c.q.shape[:2], dtype=torch.bool, device="cuda")
    bad[rows, head] = True
    out = run()
    assert out[bad].isnan().all()
    assert torch.equal(out[~bad], clean[~bad])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hkv,d", [(4, 4, 64), (4, 1, 128), (6, 2, 256)])
@pytest.mark.parametrize("causal", [True, False])
def test_prompts(hq, hkv, d, causal, dtype):
    """Whole items (the short ones) and ones of many pieces."""
    c = P.Case([20011, 30, 5000, 700], [3, 30, 1, 300], hq, hkv, d, dtype, seed=80)
    check(c, lambda: c.run(causal), [1, 5, 33, 40, 333], hq - 1)


@pytest.mark.parametrize("seqs", [20, 240])
@pytest.mark.parametrize("hq,hkv,d", [(2, 2, 64), (8, 2, 128), (4, 2, 256)])
def test_single_tokens(seqs, hq, hkv, d):
    lens = np.random.default_rng(81).integers(1, 200, seqs)
    lens[3] = 3000
    c = P.Case(lens, np.ones(seqs, int), hq, hkv, d, "bf16", seed=81)
    check(c, c.run, [0, 3, seqs - 1], 1)


@pytest.mark.parametrize("seqs", [20, 240])
@pytest.mark.parametrize("hq,hkv,d", [(2, 2, 64), (8, 2, 128), (4, 2, 256)])
@pytest.mark.parametrize("blocks", [3, 100])
def test_behind_prefixes(seqs, hq, hkv, d, blocks):
    lens = np.random.default_rng(82).integers(1, 16 * blocks + 80, seqs)
    lens[[0, 1, 2]] = [16 * blocks, 16 * blocks + 1, 5]
    c = P.prefix_case(lens, hq, hkv, d, "bf16", [0, seqs - 4], [blocks], seed=82)
    check(c, lambda: P.prefix_run(c), [0, 1, 2, 7, seqs - 2], 1)
