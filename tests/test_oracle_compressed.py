"""Pins of the 4-bit and latent oracles: worked examples and closed forms (CPU)."""

import numpy as np
import pytest

import oracle.int4 as O4
import oracle.latent as OL


def test_group_of_sixteen_steps_is_exact():
    # 0, 1, .. 15 repeated: z = 0, s = 1, every code exact
    x = np.tile(np.arange(16.0), 4)
    c, p = O4.quantize(x, "bf16")
    assert p.tolist() == [[1.0, 0.0]] and c.tolist() == list(range(16)) * 4
    assert np.array_equal(O4.dequantize(c, p), x)


def test_ties_constant_and_non_finite_groups():
    x = np.zeros(192)
    x[:4] = [-1.0, 14.0, 1.5, 2.5]          # s = 1: (x - z) = 2.5 and 3.5 are ties
    x[64:128] = 3.0                          # constant: s = 0, codes 0
    x[130] = np.inf
    c, p = O4.quantize(x, "f16")
    assert c[:4].tolist() == [0, 15, 2, 4] and c[4] == 1
    assert p[1].tolist() == [0.0, 3.0] and not c[64:128].any()
    assert np.isnan(p[2]).all() and np.isnan(O4.dequantize(c, p)[128:]).all()


@pytest.mark.parametrize("dtype,half_step", [("f16", 2.0 ** -12), ("bf16", 2.0 ** -9)])
def test_error_bound(dtype, half_step):
    x = O4.round_to(np.random.default_rng(0).normal(size=(200, 128)) * 3, dtype)
    c, p = O4.quantize(x, dtype)
    err = np.abs(O4.dequantize(c, p) - x).reshape(200, 2, 64)
    # half a step, and for the top code what rounding s takes away; fp32 steps add 2^-20 of the range
    assert np.all(err <= p[..., 0:1] * (0.5 + 15 * half_step + 2.0 ** -16))


def test_widest_ranges_stay_finite():
    big = O4.round_to(np.float32(3.3e38), "bf16")
    x = np.full(64, -big)
    x[1] = big
    c, p = O4.quantize(x, "bf16")
    assert np.isfinite(p).all() and c[:2].tolist() == [0, 15]


@pytest.mark.parametrize("D", [64, 128, 256])
def test_tile_places_every_byte_once(D):
    codes = np.arange(16 * D).reshape(16, D)
    k = [(codes >> b & 1).astype(np.uint8) for b in range(12)]
    pairs = np.zeros((16, D // 64, 2))
    seen = np.zeros((18 * D, 2, 12), int)
    for b in range(12):
        tile = O4.tile_bytes(k[b], pairs, np.zeros_like(k[b]), pairs, "f16")
        seen[:, 0, b], seen[:, 1, b] = tile & 15, tile >> 4
    ids = (seen * (1 << np.arange(12))).sum(-1)[:8 * D].reshape(-1)
    assert sorted(ids.tolist()) == list(range(16 * D))


def test_absorbed_form_equals_expanded_form():
    rng = np.random.default_rng(1)
    H, N, V, L = 3, 128, 128, 21
    qn, qr = rng.normal(size=(H, N)), rng.normal(size=(H, 64))
    U, W = rng.normal(size=(H, N, 512)) / 16, rng.normal(size=(H, V, 512)) / 16
    cache = rng.normal(size=(3, 16, 576)).astype(np.float16)
    table = np.array([[2, 0]])
    q = np.concatenate((np.einsum("hnc,hn->hc", U, qn), qr), 1).astype(np.float16)[None]
    qf = q.astype(np.float64)
    out, _ = OL.decode(q, cache, table, [L], 192 ** -0.5, "f16")
    rows = OL.rows_of(cache.astype(np.float64), table[0], L)
    # the absorbed query was rounded to fp16: compare with keys of exactly that query (U = identity maps)
    want = OL.expanded(qf[0, :, :512], qf[0, :, 512:], rows[:, :512], rows[:, 512:],
                       np.tile(np.eye(512), (H, 1, 1)), W, 192 ** -0.5)
    assert np.allclose(np.einsum("hvc,hc->hv", W, out[0]), want, rtol=1e-12, atol=1e-12)
    loose = OL.expanded(qn, qr, rows[:, :512], rows[:, 512:], U, W, 192 ** -0.5)
    assert np.abs(want - loose).max() < 0.05 * np.abs(loose).max()
