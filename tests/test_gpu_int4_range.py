"""The 4-bit decode over the whole range of its types: values next to the largest and the smallest of bf16, groups of
very different size in one row, single rows that dwarf the rest. The bound is test_gpu_int4's (the oracle's for the
weights, one rounding of the output) and two absolute terms that only the ends show:
 * outputs that fp32 and bf16 hold as subnormals only: half of bf16's smallest step, 2^-134, and one fp32 step (2^-149)
   for each of the sum's terms and roundings;
 * weights times scales that fp16 holds as subnormals only. The kernel rounds p s 2^(7 - E) to fp16, with p <= 2^8 the
   weight before it is divided by the sum l of all and 2^E <= 2 s_max a bound of the attended scales of the 64 dims.
   Below 2^-14 that rounding is off by 2^-25 at most, p s so by 2^(E - 32) <= 2^-31 s_max, times a code of at most 15
   for each of the sequence's L tokens; l >= 1, as a weight next to the reference maximum is 1 or more (and what is
   rescaled by powers of two or moves to another maximum only shrinks): 15 L 2^-31 s_max."""

import numpy as np
import pytest
import torch

import helpers as H
import oracle.int4 as O4
from paged_kv_cache_217_gb300 import binding as B
from paged_kv_cache_217_gb300 import workloads as W
from test_gpu_int4 import HALF_STEP, MANY, TINY, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    H.ensure_built()
    B.device_status(clear=True)
    yield


def _check(c, out):
    want, bound = O4.decode(W.to_numpy_storage(c.q, c.dtype), c.kc, c.kp, c.vc, c.vp, c.tables_np, c.lens_np, c.scale,
                            c.dtype, 0)
    got = H.to_f64(out)
    assert np.isfinite(got).all()
    tiny = TINY[c.dtype] if c.dtype == "f16" else 2.0 ** -134 + (2 * c.lens_np.max() + 8) * 2.0 ** -149
    S, hq, D = want.shape
    coarse = np.zeros((S, c.hkv, D // 64))
    for i, n in enumerate(c.lens_np.tolist()):
        if n:
            rows = c.vp[c.tables_np[i, :-(-n // 16)]][..., 0]            # [blocks, hkv, 16, D / 64]
            rows = rows.transpose(0, 2, 1, 3).reshape(-1, c.hkv, D // 64)[:n]
            coarse[i] = 15 * n * 2.0 ** -31 * rows.max(0)
    coarse = np.repeat(np.repeat(coarse, 64, 2), hq // c.hkv, 1)
    allowed = bound + HALF_STEP[c.dtype] * (np.abs(want) + bound) + tiny + coarse
    worst = np.max((np.abs(got - want) - allowed) / allowed)
    assert worst <= 0, f"over the bound by {worst:.3g} of it"
    assert B.device_status(clear=True) == 0


def _magnitude(m, D, hkv, dtype="bf16", steps=6):
    """V rows of uniform values up to m (a number, or one per group), over 2^steps from row to row."""
    def v(nb):
        rng = np.random.default_rng(13)
        x = rng.uniform(-1, 1, size=(nb, hkv, 16, D)) * np.exp2(rng.integers(-steps, 1, size=(nb, hkv, 16, 1)))
        return O4.round_to(x * np.repeat(np.broadcast_to(m, D // 64), 64), dtype)
    return v


ENDS = [3.3e38, 1e37, 2e34, 1e33, 2.0 ** 80, 2.0 ** 75, 1e-33, 1e-36, 2.0 ** -124, 2.0 ** -130]


@pytest.mark.parametrize("magnitude", ENDS)
@pytest.mark.parametrize("hq,hkv,D", [(1, 1, 128), (8, 1, 128), (4, 2, 64), (8, 1, 64), (2, 2, 256), (5, 1, 256)])
def test_ends_of_bf16(magnitude, hq, hkv, D):
    c = Case([1, 200, 64, 33], hq, hkv, D, "bf16", 14, v=_magnitude(magnitude, D, hkv))
    _check(c, c.run())


@pytest.mark.parametrize("magnitude", [3.3e38, 1.0, 1e-36])
@pytest.mark.parametrize("hq,hkv,D", [(12, 12, 128), (40, 8, 64), (36, 12, 256)])
def test_ends_of_bf16_over_warps_and_ctas(magnitude, hq, hkv, D):
    c = Case(MANY, hq, hkv, D, "bf16", 15, v=_magnitude(magnitude, D, hkv), extra_cols=3)
    assert B.int4_workspace_size(len(MANY), hq, hkv, D, c.tables.shape[1]) > 0
    _check(c, c.run())
    one = Case([9001, 40], 4, 1, D, "bf16", 16, v=_magnitude(magnitude, D, 1))
    assert B.int4_workspace_size(2, 4, 1, D, one.tables.shape[1]) > 0
    _check(one, one.run())


@pytest.mark.parametrize("dtype,magnitudes", [("bf16", [1e6, 1e-6]), ("bf16", [1e-30, 3e38, 1.0, 1e-36]),
                                              ("bf16", [1e20, 1e-10, 1e3, 1e38]), ("f16", [3e4, 1e-3]),
                                              ("f16", [1e-2, 6e4, 1.0, 1e-4])])
@pytest.mark.parametrize("hq,hkv", [(2, 2), (8, 1)])
def test_groups_of_very_different_size(dtype, magnitudes, hq, hkv):
    D = 64 * len(magnitudes)
    c = Case([1, 200, 64, 700], hq, hkv, D, dtype, 17, v=_magnitude(np.array(magnitudes), D, hkv, dtype, steps=2))
    _check(c, c.run())


@pytest.mark.parametrize("what", ["offset", "scale", "both"])
@pytest.mark.parametrize("at", [0, 40, 333, 699])
@pytest.mark.parametrize("hq,hkv,D", [(2, 2, 128), (8, 1, 64)])
def test_one_row_that_dwarfs_the_rest(what, at, hq, hkv, D):
    """One row next to the type's largest value, in one warp's piece of the sequence; 700 others of size 1."""
    c = Case([700, 20], hq, hkv, D, "bf16", 18)
    kc, kp, vc, vp = c.kc, c.kp, c.vc.copy(), c.vp.copy()
    block, slot = c.tables_np[0, at // 16], at % 16
    if what != "scale":
        vp[block, :, slot, :, 1] = O4.round_to(np.float32(-3.2e38 if what == "both" else 3.2e38), "bf16")
    if what != "offset":
        vp[block, :, slot, :, 0] = O4.round_to(np.float32(4.2e37 if what == "both" else 2.0e37), "bf16")
    c.vp = vp
    if what == "offset":
        vc[block, :, slot] = 0
        c.vc = vc
    c.cache = torch.from_numpy(O4.tile_bytes(kc, kp, c.vc, vp, "bf16")).cuda()
    _check(c, c.run())


def test_growing_scores_over_the_largest_values():
    """The running maximum moves again and again while the sums are kept small."""
    D, L = 128, 600
    nb = W.pool_size(np.array([L]), 1.2) + 1
    table = W.scattered_tables(np.array([L]), nb, 16)[0][0]

    def k(n):
        x = np.zeros((n, 1, 16, D))
        for p in range(L):
            x[table[p // 16], 0, p % 16, :] = p / 8
        x[..., 1::2] = 0
        return O4.round_to(x, "bf16")
    c = Case([L], 2, 1, D, "bf16", 16, k=k, v=_magnitude(3.3e38, D, 1))
    c.q = torch.ones_like(c.q)
    c.q[:, 1] = -1
    c.scale = 0.02
    _check(c, c.run())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_rows_of_any_size_are_written_as_defined(dtype, D):
    """Every byte of the tiles, for rows of every power of two of the type, groups of ties and of one value."""
    nb, hkv = 80, 2
    rng = np.random.default_rng(D)
    low, high = {"f16": (-24, 15), "bf16": (-133, 127)}[dtype]
    size = np.exp2(rng.uniform(low, high, size=(nb * 16, hkv, D // 64, 1)))
    x = rng.uniform(-1, 1, size=(nb * 16, hkv, D // 64, 64)) * size
    x[::7] = np.rint(x[::7] / size[::7] * 15) * size[::7] / 8          # steps and halves of steps
    x[::11] = x[::11, :, :, :1]
    x[::13] += 40 * size[::13]                                         # far from zero
    limit = 65504.0 if dtype == "f16" else 3.38e38
    x = O4.round_to(np.clip(x, -limit, limit), dtype).reshape(nb * 16, hkv, D) + 0.0
    k, v = x, x[::-1]
    cache = torch.zeros((nb, hkv, 18 * D), dtype=torch.uint8, device="cuda")
    slots = rng.permutation(nb * 16)
    B.reshape_and_cache_int4(*(torch.from_numpy(np.ascontiguousarray(a[slots]).astype(np.float32)).cuda().to(
        H.torch_dtype(dtype)) for a in (k, v)), cache, torch.from_numpy(slots).cuda())
    dense = []
    for a in (k, v):
        dense += [t.reshape(nb, 16, hkv, *t.shape[2:]).swapaxes(1, 2) for t in O4.quantize(a, dtype)]
    assert np.array_equal(cache.cpu().numpy(), O4.tile_bytes(*dense, dtype))
    assert B.device_status(clear=True) == 0
