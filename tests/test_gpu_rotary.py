"""The rotated cache write (GPU): bit-exact to its fp32 definition, within the oracle's rounding, and the pools
around it untouched."""

import numpy as np
import pytest
import torch

import helpers as H
import oracle.prompt as OP
from paged_kv_cache_217_gb300 import binding as B

pytestmark = pytest.mark.gpu

HALF_STEP = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    H.ensure_built()
    B.device_status(clear=True)
    yield


def table(rot, positions=600):
    angle = torch.outer(torch.arange(positions, dtype=torch.float64),
                        10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot))
    return torch.cat((angle.cos(), angle.sin()), 1).float().cuda()


def turned(x, positions, cos_sin, interleaved):
    """The definition, operation by operation in fp32."""
    rot = cos_sin.shape[1]
    c, s = cos_sin[positions.long()][:, None].chunk(2, -1)
    f = x.float()
    a, b = (f[..., 0:rot:2], f[..., 1:rot:2]) if interleaved else (f[..., :rot // 2], f[..., rot // 2:rot])
    y = (a * c - b * s, b * c + a * s)
    y = torch.stack(y, -1).flatten(-2) if interleaved else torch.cat(y, -1)
    return torch.cat((y, f[..., rot:]), -1).to(x.dtype)


class Case:
    def __init__(self, T, hq, hkv, d, dtype, seed=0, sliced=False):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        dt = H.torch_dtype(dtype)
        x = torch.randn((T, hq + 2 * hkv, d), generator=gen, device="cuda").to(dt)
        self.q, self.k, self.v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
        if not sliced:
            self.q, self.k, self.v = (t.contiguous() for t in (self.q, self.k, self.v))
        nb = -(-T // 16) + 2
        self.slots = torch.randperm(nb * 16, generator=gen, device="cuda")[:T]
        self.positions = torch.randint(0, 600, (T,), generator=gen, device="cuda", dtype=torch.int32)
        self.pools = [torch.randn((nb, hkv, 16, d), generator=gen, device="cuda").to(dt) for _ in range(2)]

    def run(self, cos_sin, interleaved=False):
        self.q_out = torch.full(self.q.shape, float("nan"), dtype=self.q.dtype, device="cuda")
        kp, vp = (p.clone() for p in self.pools)
        B.rotary_and_cache(self.q_out, self.q, self.k, self.v, self.positions, cos_sin, kp, vp, self.slots, interleaved)
        torch.cuda.synchronize()
        return kp, vp

    def want(self, cos_sin, interleaved=False):
        kp, vp = (p.clone() for p in self.pools)
        live = (self.slots >= 0) & (self.positions >= 0)
        at, safe = self.slots[live], self.positions.clamp(min=0)
        kp[at // 16, :, at % 16] = turned(self.k, safe, cos_sin, interleaved)[live]
        vp[at // 16, :, at % 16] = self.v[live]
        return turned(self.q, safe, cos_sin, interleaved), kp, vp


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("hq,hkv,d,rot", [(4, 4, 64, 64), (8, 2, 128, 128), (5, 1, 128, 32), (3, 3, 256, 256), (7, 1, 256, 80),
                                          (40, 40, 128, 128), (1, 1, 64, 16)])
def test_bits(hq, hkv, d, rot, interleaved, dtype):
    for T in (1, 37):
        c = Case(T, hq, hkv, d, dtype, seed=T, sliced=T > 1)
        cs = table(rot)
        kp, vp = c.run(cs, interleaved)
        q, k, v = c.want(cs, interleaved)
        assert torch.equal(c.q_out, q) and torch.equal(kp, k) and torch.equal(vp, v)
        exact = OP.rotate(H.to_f64(c.q), c.positions.cpu().numpy(), cs.double().cpu().numpy(), interleaved)
        # two products and a sum in fp32 (each off by 2^-24 of the larger product), one rounding
        size = np.abs(H.to_f64(c.q)).max(-1, keepdims=True)
        allowed = HALF_STEP[dtype] * np.abs(exact) + 2.0 ** -21 * size + 2.0 ** -25
        assert (np.abs(H.to_f64(c.q_out) - exact) <= allowed).all()
    assert B.device_status(clear=True) == 0


def test_many_tokens():
    c = Case(3001, 8, 2, 128, "bf16", seed=3, sliced=True)
    cs = table(128)
    c.slots[::5] = -1
    kp, vp = c.run(cs)
    q, k, v = c.want(cs)
    assert torch.equal(c.q_out, q) and torch.equal(kp, k) and torch.equal(vp, v)


def test_skipped_slots_and_padding():
    """A slot < 0 keeps K and V out of the cache, a position < 0 leaves the whole token out."""
    c = Case(40, 4, 2, 128, "f16", seed=4)
    c.slots[3::7] = -1
    c.positions[5::6] = -1
    cs = table(64)
    kp, vp = c.run(cs)
    q, k, v = c.want(cs)
    pad = c.positions < 0
    assert c.q_out[pad].isnan().all() and torch.equal(c.q_out[~pad], q[~pad])
    assert torch.equal(kp, k) and torch.equal(vp, v)
    assert B.device_status(clear=True) == 0


def test_in_place_and_without_queries():
    c = Case(21, 4, 2, 128, "bf16", seed=5, sliced=True)
    cs = table(128)
    q, k, v = c.want(cs)
    kp, vp = (p.clone() for p in c.pools)
    B.rotary_and_cache(c.q, c.q, c.k, c.v, c.positions, cs, kp, vp, c.slots)
    assert torch.equal(c.q, q) and torch.equal(kp, k) and torch.equal(vp, v)
    kp, vp = (p.clone() for p in c.pools)
    B.rotary_and_cache(None, None, c.k, c.v, c.positions, cs, kp, vp, c.slots)
    assert torch.equal(kp, k) and torch.equal(vp, v)


def test_bad_positions_and_slots_are_flagged():
    c = Case(9, 2, 2, 64, "f16", seed=6)
    cs = table(64)
    c.positions[4] = 600
    kp, _ = c.run(cs)
    assert B.device_status(clear=True) == 0x80
    c.positions[4] = 599
    assert torch.equal(c.run(cs)[0], kp)
    c.slots[2] = c.pools[0].shape[0] * 16
    c.run(cs)
    assert B.device_status(clear=True) == 0x4


def test_values_at_the_types_ends():
    c = Case(4, 2, 1, 64, "f16", seed=7)
    c.q[0].fill_(65504.0)
    c.k[1].fill_(float("inf"))
    c.k[2].fill_(float("nan"))
    cs = table(64)
    kp, vp = c.run(cs)
    q, k, v = c.want(cs)
    assert torch.equal(c.q_out, q) and torch.equal(kp.nan_to_num(nan=7.0), k.nan_to_num(nan=7.0)) and torch.equal(vp, v)
