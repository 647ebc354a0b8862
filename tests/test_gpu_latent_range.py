"""Latent decode where most tokens weigh little: one leading token and a long tail many powers of two below it, which
16-bit weights must not lose."""

import numpy as np
import pytest
import torch

import helpers as H
import oracle.latent as OL
from paged_kv_cache_217_gb300 import binding as B
from paged_kv_cache_217_gb300 import workloads as W
from test_gpu_latent import HALF_STEP, TINY, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    H.ensure_built()
    B.device_status(clear=True)
    yield


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("heads", [16, 40, 128])
@pytest.mark.parametrize("below,leader", [(24, 0), (25, 9000), (14, 777), (20, 16384)])
def test_a_long_tail_far_below_one_token(dtype, heads, below, leader):
    """Scores in powers of two: `below` + 2 for one token, 0 to 2 for the others, whose latents are near 8 against its
    1/64; as many sequences (over the same rows) as a wave has CTAs, so that one CTA has a whole sequence. On top of the
    oracle's bound, which counts weights as rounded relative to their size, comes what fp16 adds for small ones: a
    weight is kept times 2^7 at least and fp16 is off by 2^-25 at most below 2^-14, so by 2^-32 of the largest weight,
    which the sum of weights is no smaller than: L 2^-32 max |c - out| in all."""
    L, S = 16385, 152
    c = Case([L], heads, dtype, 21, scale=float(np.log(2.0)))
    rng = np.random.default_rng(below + leader)
    slots = torch.from_numpy(c.tables_np[0, np.arange(L) // 16].astype(np.int64) * 16 + np.arange(L) % 16).cuda()
    rows = c.cache.view(-1, 576)
    rows[slots, :512] = (W.normal_values((L, 512), dtype, 22, "cuda").float() + 8).to(c.cache.dtype)
    rows[slots[leader], :512] = (W.normal_values((512,), dtype, 23, "cuda").float() / 64).to(c.cache.dtype)
    score = rng.uniform(0, 2, L)
    score[leader] = below + 2
    rows[slots, 512] = torch.from_numpy(score).cuda().to(c.cache.dtype)
    c.q = torch.zeros((S, heads, 576), dtype=c.cache.dtype, device="cuda")
    c.q[:, :, 512] = 1
    want, bound = OL.decode(W.to_numpy_storage(c.q[:1, :1], dtype), W.to_numpy_storage(c.cache, dtype), c.tables_np,
                            c.lens_np, c.scale, dtype)
    c.tables, c.lens = c.tables.expand(S, -1).contiguous(), c.lens.expand(S).contiguous()
    got = H.to_f64(c.run())                       # (queries and rows are alike)
    spread = np.abs(H.to_f64(rows[slots, :512]) - want[0, 0]).max()
    small = L * 2.0 ** -32 * spread if dtype == "f16" else 0.0
    allowed = bound + HALF_STEP[dtype] * (np.abs(want) + bound) + TINY[dtype] + small
    worst = np.max((np.abs(got - want) - allowed) / allowed)
    assert worst <= 0, f"over the bound by {worst:.3g} of it"
    assert B.device_status(clear=True) == 0
