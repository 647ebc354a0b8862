"""GPU parity of the 4-bit KV cache (through the C ABI) against the oracle: the quantising write bit-exact,
the read-back one rounding from the stored values, decode within the bound that the oracle derives from the
roundings of the softmax weights and of the output."""

import numpy as np
import pytest
import torch

import helpers as H
import oracle.int4 as O4
from paged_kv_cache_217_gb300 import binding as B
from paged_kv_cache_217_gb300 import workloads as W

pytestmark = pytest.mark.gpu

HALF_STEP = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}   # one rounding of an output to the 16-bit type
TINY = {"f16": 2.0 ** -25, "bf16": 0.0}              # half of fp16's smallest subnormal


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    H.ensure_built()
    B.device_status(clear=True)
    yield


def _cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _values(shape, dtype, seed):
    rng = np.random.default_rng(seed)
    x = rng.normal(size=shape) * np.exp(0.5 * rng.normal(size=shape[-1:]))
    return O4.round_to(x, dtype)


def _tensor(x, dtype):
    return _cuda(np.asarray(x, np.float32)).to(H.torch_dtype(dtype))


class Case:
    """An oracle-quantised cache with scattered blocks, uploaded as tiles."""

    def __init__(self, lens, hq, hkv, D, dtype, seed, k=None, v=None, extra_cols=0, scale=None):
        self.lens_np = np.asarray(lens, np.int32)
        self.dtype, self.D, self.hkv = dtype, D, hkv
        nb = W.pool_size(self.lens_np, 1.2) + 1
        self.tables_np, _ = W.scattered_tables(self.lens_np, nb, seed, extra_cols=extra_cols)
        k = _values((nb, hkv, 16, D), dtype, seed) if k is None else k(nb)
        v = _values((nb, hkv, 16, D), dtype, seed + 1) if v is None else v(nb)
        self.kc, self.kp = O4.quantize(k, dtype)
        self.vc, self.vp = O4.quantize(v, dtype)
        self.cache = _cuda(O4.tile_bytes(self.kc, self.kp, self.vc, self.vp, dtype))
        self.q = _tensor(_values((len(lens), hq, D), dtype, seed + 2), dtype)
        self.tables, self.lens = _cuda(self.tables_np), _cuda(self.lens_np)
        self.scale = D ** -0.5 if scale is None else scale

    def run(self, **kw):
        out = torch.full_like(self.q, float("nan"))
        B.paged_attention_decode_int4(out, self.q, self.cache, self.tables, self.lens, self.scale, **kw)
        torch.cuda.synchronize()
        return out

    def check(self, out, window=0):
        want, bound = O4.decode(W.to_numpy_storage(self.q, self.dtype), self.kc, self.kp, self.vc, self.vp,
                                self.tables_np, np.maximum(self.lens_np, 0), self.scale, self.dtype, window)
        got = H.to_f64(out)
        assert np.isfinite(got).all()
        # the bound of the weights, then one rounding of the (slightly off) sum to T
        allowed = bound + HALF_STEP[self.dtype] * (np.abs(want) + bound) + TINY[self.dtype]
        worst = np.max(np.abs(got - want) - allowed)
        assert worst <= 0, f"over the bound by {worst:.3g}"


# ---- write and read-back -------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hkv,D", [(4, 64), (8, 128), (3, 256), (40, 128)])
def test_write_is_bit_exact(dtype, hkv, D):
    nb, T = 20, 77
    rng = np.random.default_rng(hkv * 1000 + D)
    slots = rng.choice(nb * 16, size=T, replace=False).astype(np.int64)
    slots[::9] = -1
    k, v = _values((T, hkv, D), dtype, 1), _values((T, hkv, D), dtype, 2)
    k[5] = 0.75                                   # constant groups: scale 0
    k[6, 0, :64], v[7, 0, 64 % D:64 % D + 64] = 0, np.tile(np.arange(16.0), 4)
    k[8, 0, 3], v[10, hkv - 1, D - 1] = np.inf, np.nan
    cache = torch.randint(0, 256, (nb, hkv, 18 * D), dtype=torch.uint8, device="cuda")
    before = cache.cpu().numpy()
    B.reshape_and_cache_int4(_tensor(k, dtype), _tensor(v, dtype), cache, _cuda(slots))
    got = cache.cpu().numpy()
    kc, kp = O4.quantize(k, dtype)
    vc, vp = O4.quantize(v, dtype)
    written = np.zeros((nb, 16), bool)
    dense = [np.zeros((nb, hkv, 16, D), np.uint8), np.zeros((nb, hkv, 16, D // 64, 2)),
             np.zeros((nb, hkv, 16, D), np.uint8), np.zeros((nb, hkv, 16, D // 64, 2))]
    for t, slot in enumerate(slots.tolist()):
        if slot >= 0:
            written[slot // 16, slot % 16] = True
            for a, x in zip(dense, (kc, kp, vc, vp)):
                a[slot // 16, :, slot % 16] = x[t]
    finite = [np.nan_to_num(dense[1], nan=0.0), np.nan_to_num(dense[3], nan=0.0)]
    want = O4.tile_bytes(dense[0], finite[0], dense[2], finite[1], dtype)
    # which bytes belong to written rows whose pairs are numbers, and which to no written row
    ones = [np.ones((nb, hkv, 16, D), np.uint8) * 15, np.ones((nb, hkv, 16, D // 64, 2))]
    on = ones[0] * written[:, None, :, None]
    pairs_on = [(np.isfinite(p) & written[:, None, :, None, None]) for p in (dense[1], dense[3])]
    nan_on = [(np.isnan(p) & written[:, None, :, None, None]) for p in (dense[1], dense[3])]
    mask = O4.tile_bytes(on, np.zeros_like(dense[1]), on, np.zeros_like(dense[3]), dtype) > 0
    byte = np.zeros((nb, hkv, 18 * D), bool)
    nan_byte = np.zeros_like(byte)
    for base, p, n in ((16 * D, pairs_on[0], nan_on[0]), (17 * D, pairs_on[1], nan_on[1])):
        for slot in range(16):
            row = 8 * (slot // 8) + 2 * (slot % 4) + (slot // 4) % 2
            for g in range(D // 64):
                for e in range(4):
                    byte[:, :, base + row * (D // 16) + 4 * g + e] = p[:, :, slot, g, e // 2]
                    nan_byte[:, :, base + row * (D // 16) + 4 * g + e] = n[:, :, slot, g, e // 2]
    exact = mask | byte
    assert np.array_equal(got[exact], want[exact])
    untouched = ~(exact | nan_byte)
    assert np.array_equal(got[untouched], before[untouched])
    # NaN groups read back as NaN, all others one rounding from z + c s
    ko, vo = torch.empty_like(_tensor(k, dtype)), torch.empty_like(_tensor(v, dtype))
    B.gather_cache_int4(ko, vo, cache, _cuda(slots))
    for out, c, p in ((ko, kc, kp), (vo, vc, vp)):
        x = O4.dequantize(c, p)
        x[slots < 0] = 0
        y = H.to_f64(out)
        assert np.array_equal(np.isnan(x), np.isnan(y))
        ok = ~np.isnan(x)
        # the fp32 value is one rounding (2^-24) from exact, the stored one another of T
        room = (HALF_STEP[dtype] + 2.0 ** -23) * np.abs(x[ok]) + TINY[dtype]
        assert np.all(np.abs(y[ok] - x[ok]) <= room)
    assert B.device_status(clear=True) == 0


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_widest_values(dtype):
    big = {"f16": 65504.0, "bf16": float(O4.round_to(3.3e38, "bf16"))}[dtype]
    small = {"f16": 2.0 ** -24, "bf16": 2.0 ** -133}[dtype]
    k = np.zeros((2, 1, 64))
    k[0, 0, ::2], k[0, 0, 1::2] = big, -big
    k[1, 0, ::2] = small
    v = -k
    cache = torch.zeros((1, 1, 18 * 64), dtype=torch.uint8, device="cuda")
    slots = torch.tensor([3, 14], device="cuda")
    B.reshape_and_cache_int4(_tensor(k, dtype), _tensor(v, dtype), cache, slots)
    ko, vo = torch.empty_like(_tensor(k, dtype)), torch.empty_like(_tensor(k, dtype))
    B.gather_cache_int4(ko, vo, cache, slots)
    for out, x in ((ko, k), (vo, v)):
        c, p = O4.quantize(x, dtype)
        want = O4.round_to(O4.dequantize(c, p), dtype)
        assert np.array_equal(H.to_f64(out), want)


def test_bad_slots_and_bad_pairs_are_flagged_and_skipped():
    D, hkv, nb = 128, 2, 4
    cache = torch.randint(0, 256, (nb, hkv, 18 * D), dtype=torch.uint8, device="cuda")
    before = cache.clone()
    k = W.normal_values((2, hkv, D), "bf16", 1, "cuda")
    bad = torch.tensor([nb * 16, 2 ** 40], device="cuda")
    B.reshape_and_cache_int4(k, k.clone(), cache, bad)
    assert B.device_status(clear=True) == 0x4 and torch.equal(cache, before)
    ko, vo = torch.full_like(k, 5), torch.full_like(k, 5)
    B.gather_cache_int4(ko, vo, cache, bad)
    assert B.device_status(clear=True) == 0x4 and not ko.any() and not vo.any()
    B.copy_blocks_int4(cache, torch.tensor([[0, nb], [-1, 2], [-2, 1]], device="cuda"))
    assert B.device_status(clear=True) == 0x8 and torch.equal(cache, before)


def test_copy_blocks_with_padding():
    cache = torch.randint(0, 256, (24, 8, 18 * 128), dtype=torch.uint8, device="cuda")
    before = cache.clone()
    pairs = [[0, 5], [3, 7], [3, 9], [20, 1]]
    B.copy_blocks_int4(cache, torch.tensor(pairs + [[-1, -1]] * 3, device="cuda"))
    for src, dst in pairs:
        before[dst] = before[src]
    assert torch.equal(cache, before) and B.device_status(clear=True) == 0


# ---- decode ----------------------------------------------------------------------------
LENS = [1, 0, 15, 16, 17, 63, 64, 65, 250]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv", [(2, 2), (4, 2), (3, 1), (8, 2), (5, 1), (6, 1), (7, 1), (16, 2)])
def test_decode(dtype, D, hq, hkv):
    c = Case(LENS, hq, hkv, D, dtype, 3)
    c.check(c.run())
    assert B.device_status(clear=True) == 0


MANY = [1, 300, 0, 16, 511, 33, 0, 0, 64, 31, 32, 2, 700, 15] + [5, 40] * 20


@pytest.mark.parametrize("dtype,hq,hkv,D", [("bf16", 12, 12, 128), ("bf16", 48, 12, 64), ("f16", 36, 12, 256),
                                            ("f16", 24, 24, 64), ("bf16", 80, 10, 128)])
def test_list_schedule(dtype, hq, hkv, D):
    # more items than CTAs of their own: shares that start and end anywhere, items over warps and CTAs
    c = Case(MANY, hq, hkv, D, dtype, 5, extra_cols=3)
    assert B.int4_workspace_size(len(MANY), hq, hkv, D, c.tables.shape[1]) > 0
    c.check(c.run())
    assert B.device_status(clear=True) == 0


@pytest.mark.parametrize("hq,hkv,D", [(1, 1, 128), (8, 1, 64), (3, 1, 256)])
def test_one_long_sequence_over_all_ctas(hq, hkv, D):
    c = Case([9001, 0, 40], hq, hkv, D, "bf16", 6)
    assert B.int4_workspace_size(3, hq, hkv, D, c.tables.shape[1]) > 0
    c.check(c.run())


@pytest.mark.parametrize("window", [1, 33, 100])
def test_list_schedule_with_a_window(window):
    c = Case(MANY, 12, 12, 64, "bf16", 8)
    c.check(c.run(sliding_window=window), window)


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 31, 100, 4096])
def test_windows(window):
    c = Case([1, 300, 0, 16, 117, 33], 4, 2, 128, "f16", 7)
    first = np.maximum(c.lens_np - window, 0) // 16
    t = c.tables_np.copy()
    for s, j in enumerate(first):
        t[s, :j] = -1                             # blocks before the window are never read
    c.tables = _cuda(t)
    c.check(c.run(sliding_window=window), window)
    assert B.device_status(clear=True) == 0


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D,hq,hkv", [(128, 2, 2), (64, 8, 1), (256, 4, 1)])
def test_rows_past_the_end_may_hold_anything(dtype, D, hq, hkv):
    c = Case([1, 7, 21, 40], hq, hkv, D, dtype, 11)
    kp, vp = c.kp.copy(), c.vp.copy()
    tiles = O4.tile_bytes(c.kc, kp, c.vc, vp, dtype)
    live = np.zeros(tiles.shape[0] * 16, bool)
    for s, L in enumerate(c.lens_np):
        for p in range(L):
            live[c.tables_np[s, p // 16] * 16 + p % 16] = True
    live = live.reshape(-1, 16)
    for slot in range(16):                        # NaN pairs and full codes in every dead row
        row = 8 * (slot // 8) + 2 * (slot % 4) + (slot // 4) % 2
        dead = ~live[:, slot]
        for base in (16 * D, 17 * D):
            tiles[dead, :, base + row * (D // 16):base + (row + 1) * (D // 16)] = 0xFF
    c.cache = _cuda(tiles)
    c.check(c.run())


def test_nan_in_a_live_row_shows():
    c = Case([20, 20], 2, 2, 64, "bf16", 12)
    c.vp[c.tables_np[1, 0], 1, 3] = np.nan
    c.cache = _cuda(O4.tile_bytes(c.kc, np.nan_to_num(c.kp), c.vc, np.nan_to_num(c.vp, nan=0), "bf16"))
    tile = c.cache[int(c.tables_np[1, 0]), 1]
    row = 2 * 3
    tile[17 * 64 + row * 4:17 * 64 + row * 4 + 4] = 0xFF
    out = c.run()
    assert torch.isfinite(out[0]).all() and torch.isfinite(out[1, 0]).all() and torch.isnan(out[1, 1]).all()


@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 1)])
@pytest.mark.parametrize("dtype,magnitude", [("bf16", 1e30), ("bf16", 1e-30), ("f16", 3e4), ("f16", 1e-6)])
def test_extreme_value_scales(hq, hkv, dtype, magnitude):
    def v(nb):
        rng = np.random.default_rng(13)
        x = rng.normal(size=(nb, hkv, 16, 128)) * magnitude * np.exp2(rng.integers(-6, 1, size=(nb, hkv, 16, 1)))
        return O4.round_to(np.clip(x, -6.5e4, 6.5e4) if dtype == "f16" else x, dtype)
    c = Case([1, 200, 64], hq, hkv, 128, dtype, 14, v=v)
    c.check(c.run())


@pytest.mark.parametrize("factor", [2.0 ** 12, 2.0 ** -12])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 1)])
def test_peaked_and_flat_softmax(factor, hq, hkv):
    c = Case([200, 333], hq, hkv, 128, "bf16", 15)
    c.q = (c.q.float() * factor).to(c.q.dtype)
    c.scale = 128 ** -0.5 / 32
    c.check(c.run())


def test_growing_scores_move_the_running_maximum():
    # every later token scores higher: the reference maximum moves again and again
    D, L = 128, 600
    def k(nb):
        x = np.zeros((nb, 1, 16, D))
        for p in range(L):
            x[tables[p // 16], 0, p % 16, :] = p / 8
        x[..., 1::2] = 0
        return O4.round_to(x, "bf16")
    nb = W.pool_size(np.array([L]), 1.2) + 1
    tables, _ = W.scattered_tables(np.array([L]), nb, 16)
    tables = tables[0]
    c = Case([L], 2, 1, D, "bf16", 16, k=k)
    c.q = torch.ones_like(c.q)
    c.q[:, 1] = -1
    c.scale = 0.02
    c.check(c.run())


def test_bad_ids_and_lengths_are_flagged():
    c = Case([40, 40, 40], 2, 1, 128, "bf16", 17)
    t, n = c.tables_np.copy(), c.lens_np.copy()
    t[0, 1], n[2] = 10 ** 6, 17 * 16
    c.tables, c.lens = _cuda(t), _cuda(n)
    out = c.run()
    assert B.device_status(clear=True) & 0x3 == 0x3
    c.lens_np = c.lens_np[1:2]
    c.tables_np, c.q = c.tables_np[1:2], c.q[1:2].clone()
    c.check(out[1:2])
    c.lens = _cuda(np.array([40, -3, 40], np.int32))
    c.tables = _cuda(W.scattered_tables(np.array([40, 40, 40]), W.pool_size([40] * 3, 1.2) + 1, 17)[0])
    c.q = torch.cat([c.q] * 3)
    assert not c.run()[1].any() and B.device_status(clear=True) == 0x2


def test_a_pool_past_four_gigabytes():
    D, hkv, L = 128, 8, 100
    nb = (1 << 32) // (hkv * 18 * D) + 5000
    small = Case([L], 8, hkv, D, "f16", 18)
    ids = small.tables_np[0, :7].copy()
    cache = torch.empty((nb, hkv, 18 * D), dtype=torch.uint8, device="cuda")
    far = nb - 1 - np.arange(7, dtype=np.int32) * 3
    for a, b in zip(ids.tolist(), far.tolist()):
        cache[b] = small.cache[a]
    near = small.run()
    small.cache, small.tables = cache, _cuda(far[None])
    assert torch.equal(small.run(), near)
    slots = torch.tensor([int(far[0]) * 16 + 4], device="cuda")
    k = W.normal_values((1, hkv, D), "f16", 2, "cuda")
    B.reshape_and_cache_int4(k, k.clone(), cache, slots)
    ko, vo = torch.empty_like(k), torch.empty_like(k)
    B.gather_cache_int4(ko, vo, cache, slots)
    assert torch.equal(ko, vo) and (ko - k).abs().max() < 0.5
    B.copy_blocks_int4(cache, torch.tensor([[int(far[0]), int(far[0]) - 1]], device="cuda"))
    assert torch.equal(cache[int(far[0])], cache[int(far[0]) - 1])


def test_calls_are_reproducible():
    for lens, hq, hkv in (([300, 1000, 77], 8, 2), (MANY, 24, 12)):
        c = Case(lens, hq, hkv, 128, "bf16", 20)
        first = c.run()
        for _ in range(3):
            assert torch.equal(c.run(), first)


def test_a_workspace_of_the_callers():
    c = Case(MANY, 12, 12, 64, "bf16", 21)
    ws = torch.full((B.int4_workspace_size(len(MANY), 12, 12, 64, c.tables.shape[1]) + 64,), 0xFF, dtype=torch.uint8,
                    device="cuda")
    c.check(c.run(workspace=ws))
    assert (ws[-64:] == 0xFF).all()
    with pytest.raises(B.PagedKVError, match="workspace"):
        c.run(workspace=ws[:-65])


@pytest.mark.parametrize("D,hq,hkv", [(64, 8, 1), (128, 2, 2), (256, 4, 2)])
def test_fp16_outputs_are_near_their_own_rounding(D, hq, hkv):
    """Relative rms error of fp16 outputs. A rounding to fp16 is off by at most 2^-11 relative, uniformly: rms at
    most a = 2^-11 / sqrt(3), about 0.72 a over mantissas from 1 to 2. The output has one; every weight p s has one,
    which its value's p s (c - 7.5) takes on, the value less its group's midrange: for 64 normal values of rms v that
    is at most 1.1 v. Together 0.72 a sqrt(1 + 1.1^2) = 1.07 a at most; sqrt(2) a is allowed. (With codes that are
    not centred it would be p s c, of rms 2.6 v for a minimum 2.4 v below the mean: 2 a.)"""
    c = Case([100, 240, 33], hq, hkv, D, "f16", 40)
    want, _ = O4.decode(W.to_numpy_storage(c.q, "f16"), c.kc, c.kp, c.vc, c.vp, c.tables_np, c.lens_np, c.scale, "f16", 0)
    err = np.sqrt(((H.to_f64(c.run()) - want) ** 2).mean() / (want ** 2).mean())
    assert err <= 2.0 ** 0.5 * 2.0 ** -11 / 3 ** 0.5, err
