"""Refusals of the 4-bit cache, latent attention and device table calls, without a GPU: every check that runs
on the host before anything would be launched, in the C ABI and in the binding."""

import pytest
import torch

from paged_kv_cache_217_gb300 import binding as B

FAKE = 0x10000  # a 16-byte aligned address; never dereferenced because every call below fails its checks


def _call(name, spec, kw):
    args = dict(spec)
    assert set(kw) <= set(args)
    args.update(kw)
    st = getattr(B.lib(), name)(*args.values(), None)
    return st, B.lib().pkv_last_error_string().decode()


DECODE = dict(out=FAKE, q=FAKE, cache=FAKE, bt=FAKE, cl=FAKE, S=4, hq=8, hkv=4, D=128, mb=4, nb=64, scale=0.1, dt=0,
              window=0, ws=FAKE, wsb=1 << 24)


@pytest.mark.parametrize("kw,status", [
    (dict(S=-1), 1), (dict(hq=6, hkv=4), 1), (dict(hq=0), 1), (dict(hq=36, hkv=4), 2), (dict(D=96), 2),
    (dict(dt=2), 2), (dict(mb=0), 1), (dict(nb=0), 1), (dict(S=65536), 2), (dict(scale=float("nan")), 1),
    (dict(out=None), 1), (dict(q=FAKE + 2), 1), (dict(cache=FAKE + 8), 1), (dict(bt=FAKE + 2), 1), (dict(cl=FAKE + 1), 1),
    (dict(mb=1 << 27), 1), (dict(nb=1 << 30), 2), (dict(S=200, ws=None), 5), (dict(S=200, wsb=16), 5),
    (dict(S=200, ws=FAKE + 8), 5),
])
def test_decode_int4_refusals(kw, status):
    st, msg = _call("pkv_paged_attention_decode_int4", DECODE, kw)
    assert st == status and msg


WRITE = dict(k=FAKE, v=FAKE, dt=0, cache=FAKE, slots=FAKE, T=4, hkv=4, D=128, nb=64)


@pytest.mark.parametrize("name", ["pkv_reshape_and_cache_int4", "pkv_gather_cache_int4"])
@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), 1), (dict(hkv=0), 1), (dict(nb=0), 1), (dict(D=80), 2), (dict(dt=7), 2), (dict(k=None), 1),
    (dict(v=FAKE + 4), 1), (dict(cache=FAKE + 4), 1), (dict(slots=FAKE + 4), 1), (dict(T=2 ** 31 - 1, hkv=9), 2),
    (dict(T=1, hkv=2 ** 24), 2),
])
def test_cache_int4_refusals(name, kw, status):
    st, msg = _call(name, WRITE, kw)
    assert st == status and msg


@pytest.mark.parametrize("name,spec,kw,status", [
    ("pkv_copy_blocks_int4", dict(c=FAKE, p=FAKE, n=1, hkv=2, D=128, nb=4), dict(n=-1), 1),
    ("pkv_copy_blocks_int4", dict(c=FAKE, p=FAKE, n=1, hkv=2, D=128, nb=4), dict(n=65536), 2),
    ("pkv_copy_blocks_int4", dict(c=FAKE, p=FAKE, n=1, hkv=2, D=128, nb=4), dict(hkv=0), 1),
    ("pkv_copy_blocks_int4", dict(c=FAKE, p=FAKE, n=1, hkv=2, D=128, nb=4), dict(D=32), 2),
    ("pkv_copy_blocks_int4", dict(c=FAKE, p=FAKE, n=1, hkv=2, D=128, nb=4), dict(p=FAKE + 4), 1),
    ("pkv_copy_blocks_latent", dict(c=FAKE, p=FAKE, n=1, nb=4), dict(c=None), 1),
    ("pkv_copy_blocks_latent", dict(c=FAKE, p=FAKE, n=1, nb=4), dict(nb=0), 1),
    ("pkv_copy_blocks_latent", dict(c=FAKE, p=FAKE, n=1, nb=4), dict(c=FAKE + 8), 1),
])
def test_copy_refusals(name, spec, kw, status):
    st, msg = _call(name, spec, kw)
    assert st == status and msg


LATENT = dict(out=FAKE, q=FAKE, cache=FAKE, bt=FAKE, cl=FAKE, S=4, heads=16, mb=4, nb=64, scale=0.1, dt=1, ws=FAKE,
              wsb=1 << 30)


@pytest.mark.parametrize("kw,status", [
    (dict(S=-1), 1), (dict(heads=0), 1), (dict(heads=1025), 2), (dict(dt=3), 2), (dict(mb=0), 1), (dict(nb=0), 1),
    (dict(mb=1 << 27), 1), (dict(S=65536), 2), (dict(nb=1 << 27), 2), (dict(scale=float("inf")), 1), (dict(q=None), 1),
    (dict(out=FAKE + 8), 1), (dict(cache=FAKE + 2), 1), (dict(bt=FAKE + 2), 1),
])
def test_latent_refusals(kw, status):
    st, msg = _call("pkv_paged_latent_decode", LATENT, kw)
    assert st == status and msg


def test_latent_workspace():
    assert B.latent_workspace_size(0, 16, 4) == 0
    need = B.latent_workspace_size(4, 16, 4)
    if need:
        assert _call("pkv_paged_latent_decode", LATENT, dict(ws=None))[0] == 5
        assert _call("pkv_paged_latent_decode", LATENT, dict(wsb=need - 1))[0] == 5
        assert _call("pkv_paged_latent_decode", LATENT, dict(ws=FAKE + 8))[0] == 5


LATENT_WRITE = dict(latent=FAKE, rope=FAKE, ls=512, rs=64, dt=0, cache=FAKE, slots=FAKE, T=3, nb=4)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), 1), (dict(nb=0), 1), (dict(dt=9), 2), (dict(rope=None), 1), (dict(ls=-8), 1), (dict(rs=68), 1),
    (dict(latent=FAKE + 8), 1), (dict(slots=FAKE + 4), 1),
])
def test_latent_write_refusals(kw, status):
    st, msg = _call("pkv_latent_cache_write", LATENT_WRITE, kw)
    assert st == status and msg


EXTEND = dict(bt=FAKE, cl=FAKE, new=FAKE, S=4, mb=4, stack=FAKE, count=FAKE, nb=64, ref=None, nl=FAKE, nc=FAKE,
              slots=FAKE, n=16, pairs=None, info=None, ws=None, wsb=0)


@pytest.mark.parametrize("kw,status", [
    (dict(S=-1), 1), (dict(n=-1), 1), (dict(S=65536), 2), (dict(mb=0), 1), (dict(nb=0), 1), (dict(mb=1 << 27), 1),
    (dict(bt=None), 1), (dict(slots=None), 1), (dict(nl=None), 1), (dict(ref=FAKE), 1), (dict(pairs=FAKE), 1),
    (dict(slots=FAKE + 4), 1), (dict(info=FAKE + 2), 1), (dict(n=100000), 5), (dict(S=2000), 5),
    (dict(S=2000, ws=FAKE + 4, wsb=1 << 20), 5),
])
def test_extend_refusals(kw, status):
    st, msg = _call("pkv_extend_block_tables", EXTEND, kw)
    assert st == status and msg


RELEASE = dict(bt=FAKE, cl=FAKE, fin=FAKE, S=4, mb=4, stack=FAKE, count=FAKE, nb=64, ref=None, ws=FAKE, wsb=16)


@pytest.mark.parametrize("kw,status", [
    (dict(S=-1), 1), (dict(S=65536), 2), (dict(mb=0), 1), (dict(nb=0), 1), (dict(fin=None), 1), (dict(ref=FAKE + 2), 1),
    (dict(ws=None), 5), (dict(wsb=8), 5), (dict(nb=1 << 20), 5), (dict(mb=1 << 27), 1),
])
def test_release_refusals(kw, status):
    st, msg = _call("pkv_release_sequences", RELEASE, kw)
    assert st == status and msg


def test_empty_calls_do_nothing():
    assert _call("pkv_paged_attention_decode_int4", DECODE, dict(S=0, out=None))[0] == 0
    assert _call("pkv_reshape_and_cache_int4", WRITE, dict(T=0, k=None))[0] == 0
    assert _call("pkv_paged_latent_decode", LATENT, dict(S=0, out=None))[0] == 0
    assert _call("pkv_latent_cache_write", LATENT_WRITE, dict(T=0, rope=None))[0] == 0
    assert _call("pkv_extend_block_tables", EXTEND, dict(S=0, n=0, bt=None))[0] == 0
    assert _call("pkv_release_sequences", RELEASE, dict(S=0, bt=None))[0] == 0


def test_sizes():
    assert [B.int4_tile_bytes(d) for d in (64, 128, 256, 96)] == [1152, 2304, 4608, 0]
    assert B.int4_workspace_size(4, 32, 8, 128, 128) == 0       # 32 items of at most 64 tile pairs: a CTA each
    assert B.int4_workspace_size(256, 32, 8, 128, 64) >= 2 * 304 * 4 * 128 * 4
    assert B.int4_workspace_size(4, 32, 8, 128, 4096, 512) == 0  # the window bounds the tiles
    assert B.int4_workspace_size(4, 32, 8, 96, 4096) == 0        # no such head_dim
    assert B.lib().pkv_extend_workspace_size(64, 64) == 0
    assert B.lib().pkv_extend_workspace_size(2000, 64) >= 4 * 6 * 2000
    assert B.lib().pkv_release_workspace_size(129) == 32


def test_the_binding_refuses_what_the_kernels_do_not_take():
    k = torch.zeros(2, 3, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        B.reshape_and_cache_int4(k, k, torch.zeros(2, 3, 18 * 64, dtype=torch.uint8), torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="CUDA"):
        B.paged_latent_decode(torch.zeros(1, 2, 512), torch.zeros(1, 2, 576), torch.zeros(3, 16, 576),
                              torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), 1.0)
