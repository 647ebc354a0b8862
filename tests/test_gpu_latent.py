"""GPU parity of latent attention over a paged cache (through the C ABI) against the oracle: bit-exact cache
writes and block copies, decode within the bound that the oracle derives from the roundings of the softmax
weights and of the output."""

import numpy as np
import pytest
import torch

import helpers as H
import oracle.latent as OL
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
    def __init__(self, lens, heads, dtype, seed, extra_cols=0, scale=192 ** -0.5, cache_factor=1.0):
        self.lens_np = np.asarray(lens, np.int32)
        self.dtype, self.scale = dtype, scale
        nb = W.pool_size(self.lens_np, 1.2) + 1
        self.tables_np, _ = W.scattered_tables(self.lens_np, nb, seed, extra_cols=extra_cols)
        self.cache = (W.normal_values((nb, 16, 576), dtype, seed + 1, "cuda").float() * cache_factor).to(
            H.torch_dtype(dtype))
        self.q = W.normal_values((len(lens), heads, 576), dtype, seed + 2, "cuda")
        self.tables = torch.from_numpy(self.tables_np).cuda()
        self.lens = torch.from_numpy(self.lens_np).cuda()

    def run(self):
        out = torch.full((*self.q.shape[:2], 512), float("nan"), dtype=self.q.dtype, device="cuda")
        B.paged_latent_decode(out, self.q, self.cache, self.tables, self.lens, self.scale)
        torch.cuda.synchronize()
        return out

    def check(self, out, heads=None):
        heads = list(range(self.q.shape[1])) if heads is None else heads
        want, bound = OL.decode(W.to_numpy_storage(self.q[:, heads], self.dtype),
                                W.to_numpy_storage(self.cache, self.dtype), self.tables_np, self.lens_np, self.scale,
                                self.dtype)
        got = H.to_f64(out[:, heads])
        assert np.isfinite(got).all()
        allowed = bound + HALF_STEP[self.dtype] * (np.abs(want) + bound) + TINY[self.dtype]
        worst = np.max(np.abs(got - want) - allowed)
        assert worst <= 0, f"over the bound by {worst:.3g}"


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("heads", [1, 3, 8, 16, 17, 33, 64, 65, 128])
def test_decode(dtype, heads):
    c = Case([1, 0, 15, 16, 17, 63, 64, 65, 130], heads, dtype, 3)
    c.check(c.run())
    assert B.device_status(clear=True) == 0


@pytest.mark.parametrize("heads", [16, 64, 128])
@pytest.mark.parametrize("lens", [[5000], [1, 3001], [128] * 20, [700, 1, 64, 1333, 0, 65, 2000]])
def test_long_and_mixed_lengths(heads, lens):
    c = Case(lens, heads, "bf16", 4, extra_cols=2)
    c.check(c.run(), heads=[0, heads // 2, heads - 1])


def test_many_sequences():
    lens = np.random.default_rng(0).integers(0, 200, 700)
    c = Case(lens, 16, "f16", 5)
    c.check(c.run(), heads=[0, 15])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_rows_past_the_end_may_hold_anything(dtype):
    c = Case([1, 7, 21, 40, 64, 70], 16, dtype, 6)
    live = torch.zeros(c.cache.shape[0] * 16, dtype=torch.bool)
    for s, L in enumerate(c.lens_np):
        for p in range(L):
            live[int(c.tables_np[s, p // 16]) * 16 + p % 16] = True
    flat = c.cache.view(-1, 576)
    clean = c.run()
    dead = (~live).cuda()
    flat[dead] = float("nan")
    assert torch.equal(c.run(), clean)
    flat[dead] = float("inf")
    assert torch.equal(c.run(), clean)
    flat[dead] = 0
    c.check(clean)


def test_nan_in_a_live_row_shows():
    c = Case([40, 40], 16, "bf16", 7)
    c.cache[int(c.tables_np[1, 1]), 3, 70] = float("nan")
    out = c.run()
    assert torch.isfinite(out[0]).all() and torch.isnan(out[1]).all()


def test_growing_scores_move_the_running_maximum():
    L = 900
    c = Case([L], 16, "bf16", 8)
    rows = c.cache.view(-1, 576)
    for p in range(L):
        rows[int(c.tables_np[0, p // 16]) * 16 + p % 16, 512:] = p / 16
    c.q[:, :, 512:] = 1
    c.q[:, ::2, 512:] = -1
    c.scale = 0.03
    c.check(c.run())


@pytest.mark.parametrize("factor", [64.0, 2.0 ** -10])
def test_peaked_and_flat_softmax(factor):
    c = Case([200, 333], 16, "bf16", 9)
    c.q = (c.q.float() * factor).to(c.q.dtype)
    c.scale = 192 ** -0.5 / 8
    c.check(c.run())


@pytest.mark.parametrize("dtype,factor", [("bf16", 1e15), ("bf16", 1e-18), ("f16", 1000.0)])
def test_extreme_magnitudes(dtype, factor):
    c = Case([1, 100, 64], 16, dtype, 10, cache_factor=factor, scale=192 ** -0.5 / factor)
    c.check(c.run())


def test_bad_ids_and_lengths_are_flagged():
    c = Case([40, 40, 40], 16, "bf16", 11)
    good = c.run()
    t, n = c.tables_np.copy(), c.lens_np.copy()
    t[0, 1], n[2] = -7, -2
    c.tables, c.lens = torch.from_numpy(t).cuda(), torch.from_numpy(n).cuda()
    out = c.run()
    assert B.device_status(clear=True) == 0x3
    assert torch.equal(out[1], good[1]) and not out[2].any()
    n[2] = 16 * t.shape[1] + 1
    c.lens = torch.from_numpy(n).cuda()
    assert torch.equal(c.run()[1], good[1])
    assert B.device_status(clear=True) == 0x3


def test_write_with_strides_and_skipped_slots():
    nb, T = 30, 101
    for dtype in ("f16", "bf16"):
        cache = W.normal_values((nb, 16, 576), dtype, 1, "cuda")
        before = W.to_numpy_storage(cache, dtype).copy()
        proj = W.normal_values((T, 640), dtype, 2, "cuda")
        rng = np.random.default_rng(3)
        slots = rng.choice(nb * 16, size=T, replace=False).astype(np.int64)
        slots[::7] = -1
        B.latent_cache_write(proj[:, :512], proj[:, 520:584], cache, torch.from_numpy(slots).cuda())
        p = W.to_numpy_storage(proj, dtype)
        want = OL.cache_write(p[:, :512], p[:, 520:584], before, slots)
        assert np.array_equal(W.to_numpy_storage(cache, dtype).view(np.uint16), want.view(np.uint16))
        one = proj[:1].expand(4, 640)             # the same row for several tokens
        B.latent_cache_write(one[:, :512], one[:, 512:576], cache, torch.arange(4, device="cuda"))
        assert torch.equal(cache[0, :4], proj[:1, :576].expand(4, 576))
    assert B.device_status(clear=True) == 0
    B.latent_cache_write(proj[:2, :512], proj[:2, 512:576], cache, torch.tensor([nb * 16, 2 ** 41], device="cuda"))
    assert B.device_status(clear=True) == 0x4


def test_copy_blocks_with_padding():
    cache = W.normal_values((12, 16, 576), "bf16", 1, "cuda")
    want = cache.clone()
    pairs = [[0, 5], [3, 7], [3, 9]]
    for a, b in pairs:
        want[b] = want[a]
    B.copy_blocks_latent(cache, torch.tensor(pairs + [[-1, -1]], device="cuda"))
    assert torch.equal(cache, want) and B.device_status(clear=True) == 0
    B.copy_blocks_latent(cache, torch.tensor([[0, 12], [-1, 0]], device="cuda"))
    assert torch.equal(cache, want) and B.device_status(clear=True) == 0x8


def test_a_pool_past_four_gigabytes():
    c = Case([100], 16, "f16", 12)
    near = c.run()
    nb = (1 << 32) // (16 * 576 * 2) + 5000
    cache = torch.empty((nb, 16, 576), dtype=torch.float16, device="cuda")
    far = nb - 1 - np.arange(7, dtype=np.int32) * 3
    for a, b in zip(c.tables_np[0, :7].tolist(), far.tolist()):
        cache[b] = c.cache[a]
    c.cache, c.tables = cache, torch.from_numpy(far[None].copy()).cuda()
    assert torch.equal(c.run(), near)


def test_calls_are_reproducible():
    c = Case([300, 4000, 77], 128, "bf16", 13)
    first = c.run()
    for _ in range(3):
        assert torch.equal(c.run(), first)


@pytest.mark.parametrize("heads", [129, 200, 513, 1024])
def test_many_heads(heads):
    c = Case([130, 1, 0, 700], heads, "bf16", 17)
    c.check(c.run(), heads=[0, 43, 64, heads // 2, heads - 1])
    assert B.device_status(clear=True) == 0


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("heads", [16, 128])
def test_latents_alike_come_back_as_they_are(dtype, heads):
    """A weighted mean of equal values is the value, whatever the (rounded) weights: they differ here by the rotary
    parts. The two fp32 sums of n terms are off by n 2^-24 relative each at most, 2^-10.7 together for 5000: under
    half a bf16 step (2^-9 at least), and under one and a half of fp16 (2^-11 each at least), so that rounds to the
    value or, in fp16, to one at most two steps (2^-10 each at most) from it."""
    c = Case([1, 63, 700, 5000], heads, dtype, 19)
    rows = W.normal_values((4, 512), dtype, 20, "cuda")
    for s, n in enumerate(c.lens_np.tolist()):
        ids = torch.from_numpy(c.tables_np[s, :-(-n // 16)].astype(np.int64)).cuda()
        c.cache[ids, :, :512] = rows[s]
    out, want = H.to_f64(c.run()), H.to_f64(rows)[:, None]
    step = 0.0 if dtype == "bf16" else 2.0 ** -9
    assert (np.abs(out - want) <= step * np.abs(want)).all()
