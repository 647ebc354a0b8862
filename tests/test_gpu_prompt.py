"""GPU parity of prompt and cross attention over the paged cache, and of decode behind a shared prefix, against
the float64 oracle: within the bound that it derives from the roundings of the softmax weights, and the output's
own rounding."""

import numpy as np
import pytest
import torch

import helpers as H
import oracle.prompt as OP
from paged_kv_cache_217_gb300 import binding as B
from paged_kv_cache_217_gb300 import workloads as W

pytestmark = pytest.mark.gpu

HALF_STEP = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f16": 2.0 ** -25, "bf16": 0.0}


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    H.ensure_built()
    B.device_status(clear=True)
    yield


class Case:
    """Ragged queries over scattered pools. lens: context tokens; new: query tokens of each sequence."""

    def __init__(self, lens, new, hq, hkv, d, dtype, seed=1, behind=0, extra_cols=0, scale=None):
        self.lens_np, self.new = np.asarray(lens, np.int32), np.asarray(new, np.int32)
        self.dtype, self.scale = dtype, scale if scale is not None else d ** -0.5
        nb = W.pool_size(self.lens_np, 1.2) + 1
        self.tables_np, _ = W.scattered_tables(self.lens_np, nb, seed, extra_cols=extra_cols)
        self.starts_np = np.concatenate(([0], np.cumsum(self.new))).astype(np.int32)
        self.k = W.normal_values((nb, hkv, 16, d), dtype, seed + 1, "cuda")
        self.v = W.normal_values((nb, hkv, 16, d), dtype, seed + 2, "cuda")
        self.q = W.normal_values((int(self.starts_np[-1]) + behind, hq, d), dtype, seed + 3, "cuda")
        self.tables, self.lens = torch.from_numpy(self.tables_np).cuda(), torch.from_numpy(self.lens_np).cuda()
        self.starts = torch.from_numpy(self.starts_np).cuda()

    def run(self, causal=True, window=0, workspace=None):
        out = torch.full_like(self.q, float("nan"))
        B.paged_prompt_attention(out, self.q, self.k, self.v, self.tables, self.lens, self.starts, self.scale,
                                 causal=causal, sliding_window=window, workspace=workspace)
        torch.cuda.synchronize()
        return out

    def check(self, out, causal=True, window=0, heads=None, wanted=None, tables=None, starts=None):
        starts = self.starts_np if starts is None else starts
        want, bound = OP.attention(W.to_numpy_storage(self.q, self.dtype), W.to_numpy_storage(self.k, self.dtype),
                                   W.to_numpy_storage(self.v, self.dtype),
                                   self.tables_np if tables is None else tables, self.lens_np, starts, self.scale,
                                   self.dtype, causal, window, heads, wanted)
        got = H.to_f64(out if heads is None else out[:, heads])
        rows = ~np.isnan(want[:, 0, 0])
        assert np.isfinite(got[rows]).all()
        allowed = bound + HALF_STEP[self.dtype] * (np.abs(want) + bound) + TINY[self.dtype]
        worst = np.max((np.abs(got - want) - allowed)[rows])
        assert worst <= 0, f"over the bound by {worst:.3g}"
        assert B.device_status(clear=True) == 0


HEADS = [(4, 4, 64), (4, 1, 128), (6, 2, 64), (10, 2, 128), (7, 1, 64), (8, 1, 256), (3, 3, 256), (16, 1, 128)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hkv,d", HEADS)
def test_whole_prompts(hq, hkv, d, dtype):
    lens = [1, 0, 15, 16, 17, 63, 64, 65, 127, 130]
    c = Case(lens, lens, hq, hkv, d, dtype)
    c.check(c.run())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hkv,d", HEADS)
def test_chunks_behind_cached_tokens(hq, hkv, d, dtype):
    c = Case([300, 129, 517, 40, 16, 9], [5, 1, 130, 40, 0, 3], hq, hkv, d, dtype, seed=2, extra_cols=3)
    c.check(c.run(), heads=[0, hq - 1])


@pytest.mark.parametrize("hq,hkv,d", HEADS)
def test_cross_attention(hq, hkv, d):
    c = Case([300, 0, 129, 1, 517], [5, 2, 1, 60, 130], hq, hkv, d, "bf16", seed=3)
    c.check(c.run(causal=False), causal=False, heads=[0, hq - 1])


@pytest.mark.parametrize("window", [1, 2, 16, 33, 100, 128, 400, 10000])
@pytest.mark.parametrize("hq,hkv,d", [(4, 4, 64), (4, 1, 128), (6, 2, 256)])
def test_windows(window, hq, hkv, d):
    c = Case([700, 64, 257, 3], [300, 64, 1, 3], hq, hkv, d, "bf16", seed=4)
    c.check(c.run(window=window), window=window, heads=[hq - 1], wanted=set(range(0, 368, 7)) | {299, 300, 363, 364, 365, 367})


def test_long_contexts_are_split_and_joined():
    """Few rows over a long context: many pieces of one row, in every head."""
    c = Case([20011, 5000], [3, 1], 8, 2, 128, "f16", seed=5)
    c.check(c.run(), heads=[0, 5])
    c.check(c.run(causal=False), causal=False, heads=[7])


def test_long_prompt():
    c = Case([4100], [4100], 4, 2, 128, "bf16", seed=6)
    out = c.run()
    c.check(out, heads=[3], wanted={0, 1, 127, 128, 129, 2047, 2048, 3000, 4095, 4096, 4099})


def test_many_short_sequences():
    rng = np.random.default_rng(0)
    lens = rng.integers(0, 90, 700)
    new = np.minimum(rng.integers(0, 5, 700), lens)
    c = Case(lens, new, 4, 2, 64, "f16", seed=7)
    c.check(c.run(), heads=[0, 3])


def test_more_queries_than_tokens():
    """Positions before the first token: nothing is seen, zeros."""
    c = Case([3, 0, 200], [5, 4, 1], 4, 2, 128, "bf16", seed=8)
    out = c.run()
    c.check(out)
    assert not out[:2].any() and not out[5:9].any()


def test_rows_of_no_sequence_are_left():
    c = Case([40, 50], [7, 9], 4, 4, 64, "f16", seed=9, behind=5)
    c.starts_np = c.starts_np + 3
    c.starts.copy_(torch.from_numpy(c.starts_np))
    out = c.run()
    assert out[:3].isnan().all() and out[19:].isnan().all() and out[3:19].isfinite().all()
    c.check(out)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 50), (False, 0)])
def test_rows_that_no_query_sees_may_hold_anything(d, causal, window):
    lens, new = [1, 21, 130, 203, 300], [1, 4, 70, 2, 128]
    c = Case(lens, new, 4, 2, d, "bf16", seed=10)
    clean = c.run(causal, window)
    live = torch.zeros(c.k.shape[0], 16, dtype=torch.bool, device="cuda")
    for s, (n, L) in enumerate(zip(new, lens)):
        first = max(0, L - n + 1 - window) if window else 0
        for p in range(first, L):
            live[int(c.tables_np[s, p // 16]), p % 16] = True
        if window:
            c.tables[s, :first // 16] = -1
    for x in (c.k, c.v):
        x.masked_fill_(~live[:, None, :, None], float("nan"))
    assert torch.equal(c.run(causal, window), clean)
    for x in (c.k, c.v):
        x.masked_fill_(~live[:, None, :, None], float("inf"))
    assert torch.equal(c.run(causal, window), clean)
    assert B.device_status(clear=True) == 0


def test_large_scores_and_negative_scale():
    for scale in (40.0, -3.0, 0.0):
        c = Case([150, 33], [60, 33], 4, 1, 128, "f16", seed=11, scale=scale)
        c.check(c.run())


def test_bad_tables_lengths_and_starts_are_flagged():
    c = Case([100, 60], [4, 4], 4, 2, 128, "f16", seed=12)
    c.tables[0, 2] = c.k.shape[0] + 7
    c.run()
    assert B.device_status(clear=True) == 0x1
    c = Case([100, 60], [4, 4], 4, 2, 128, "f16", seed=12)
    c.lens[1] = 16 * c.tables.shape[1] + 1
    c.run()
    assert B.device_status(clear=True) & 0x2
    for starts in ([0, 6, 4], [-3, 4, 8], [0, 4, 9]):
        c = Case([100, 60], [4, 4], 4, 2, 128, "f16", seed=12)
        c.starts.copy_(torch.tensor(starts))
        c.run()
        assert B.device_status(clear=True) == 0x100


def test_same_bits_each_time():
    c = Case([3000, 700, 64], [40, 300, 64], 8, 2, 128, "bf16", seed=13)
    first = c.run()
    for _ in range(3):
        assert torch.equal(first, c.run())


# ---- groups behind a shared prefix --------------------------------------------------------------
def prefix_case(lens, hq, hkv, d, dtype, group_starts, prefix_blocks, seed=20):
    c = Case(lens, [1] * len(lens), hq, hkv, d, dtype, seed=seed)
    c.groups = torch.tensor(group_starts, dtype=torch.int32, device="cuda")
    c.blocks = torch.tensor(prefix_blocks, dtype=torch.int32, device="cuda")
    c.shared = OP.prefix_tables(c.tables_np, group_starts, prefix_blocks)
    return c


def prefix_run(c):
    out = torch.full_like(c.q, float("nan"))
    B.paged_prefix_decode(out, c.q, c.k, c.v, c.tables, c.lens, c.groups, c.blocks, c.scale)
    torch.cuda.synchronize()
    return out


PREFIX = [  # lengths, group starts, prefix blocks
    ([70, 64, 65, 100, 81], [0, 5], [4]),
    ([70, 64, 65, 100, 500, 300, 310, 81], [1, 4, 7], [2, 16]),
    ([200] * 3, [0, 3], [0]),
    ([33], [0, 1], [1]),
    ([160, 10, 0, 161, 48, 47], [0, 6], [10]),          # members shorter than the prefix, and an empty one
    ([1000, 1007, 1016] + [999] * 40, [0, 2, 2, 43], [60, 1, 62]),
]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hkv,d", [(4, 4, 64), (4, 1, 128), (6, 2, 256), (10, 2, 128), (16, 1, 64)])
@pytest.mark.parametrize("lens,starts,blocks", PREFIX)
def test_prefix_decode(lens, starts, blocks, hq, hkv, d, dtype):
    c = prefix_case(lens, hq, hkv, d, dtype, starts, blocks)
    c.check(prefix_run(c), causal=False, heads=[0, hq - 1], tables=c.shared)


def test_prefix_of_a_wide_batch():
    rng = np.random.default_rng(1)
    lens = 2048 + rng.integers(1, 300, 300)
    c = prefix_case(lens, 8, 2, 128, "bf16", [0, 290], [128])
    c.check(prefix_run(c), causal=False, heads=[5], tables=c.shared, wanted=set(range(0, 300, 11)) | {289, 290, 299})


def test_long_own_parts_are_split():
    c = prefix_case([9000, 16 * 300, 7000], 4, 2, 128, "f16", [0, 3], [300])
    c.check(prefix_run(c), causal=False, heads=[3], tables=c.shared)


def test_prefix_decode_equals_decode_without_groups():
    c = prefix_case([70, 640, 65, 0, 81], 8, 8, 128, "bf16", [0], [])
    c.check(prefix_run(c), causal=False, tables=c.tables_np)


def test_members_tables_before_the_prefix_end_are_not_read():
    c = prefix_case([300, 310, 333], 4, 2, 128, "f16", [0, 3], [10])
    want = prefix_run(c)
    c.tables[1:, :10] = -1
    assert torch.equal(prefix_run(c), want)
    assert B.device_status(clear=True) == 0


def test_bad_groups_are_flagged():
    for starts in ([0, 9], [-1, 3], [2, 1]):
        c = prefix_case([70, 64, 65], 4, 2, 64, "f16", [0, 3], [2])
        c.groups.copy_(torch.tensor(starts))
        prefix_run(c)
        assert B.device_status(clear=True) == 0x100
    c = prefix_case([70, 64, 65], 4, 2, 64, "f16", [0, 3], [2])
    c.blocks.fill_(10 ** 6)                                   # as many blocks as the first member has
    c.lens.fill_(0)
    assert not prefix_run(c).any()
