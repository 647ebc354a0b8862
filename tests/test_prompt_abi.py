"""Refusals of the prompt, prefix and rotating calls, without a GPU: every check that runs on the host before
anything would be launched, in the C ABI and in the binding."""

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


PROMPT = dict(out=FAKE, q=FAKE, k=FAKE, v=FAKE, bt=FAKE, cl=FAKE, qs=FAKE, T=40, S=4, hq=8, hkv=4, D=128, mb=4, nb=64,
              scale=0.1, dt=0, causal=1, window=0, ws=FAKE, wsb=1 << 30)
PREFIX = dict(out=FAKE, q=FAKE, k=FAKE, v=FAKE, bt=FAKE, cl=FAKE, gs=FAKE, pb=FAKE, n=2, S=4, hq=8, hkv=4, D=128, mb=4,
              nb=64, scale=0.1, dt=0, ws=FAKE, wsb=1 << 30)
BOTH = [
    (dict(S=-1), 1), (dict(hq=6, hkv=4), 1), (dict(hq=0), 1), (dict(hkv=0), 1), (dict(hq=129, hkv=1), 2), (dict(D=96), 2),
    (dict(dt=2), 2), (dict(mb=0), 1), (dict(nb=0), 1), (dict(S=65536), 2), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(scale=3.4e38), 1), (dict(out=None), 1), (dict(q=None), 1), (dict(q=FAKE + 2), 1),
    (dict(k=FAKE + 8), 1), (dict(v=FAKE + 8), 1), (dict(bt=FAKE + 2), 1), (dict(cl=FAKE + 1), 1), (dict(cl=None), 1),
    (dict(mb=1 << 27), 1), (dict(nb=1 << 28), 2),
]


@pytest.mark.parametrize("kw,status", BOTH + [(dict(T=-1), 1), (dict(qs=None), 1), (dict(qs=FAKE + 2), 1),
                                              (dict(T=2 ** 29), 2), (dict(causal=0, window=5), 2)])
def test_prompt_refusals(kw, status):
    st, msg = _call("pkv_paged_prompt_attention", PROMPT, kw)
    assert st == status and msg


@pytest.mark.parametrize("kw,status", BOTH + [(dict(n=-1), 1), (dict(n=5), 1), (dict(gs=None), 1), (dict(pb=None), 1),
                                              (dict(gs=FAKE + 2), 1), (dict(pb=FAKE + 2), 1)])
def test_prefix_refusals(kw, status):
    st, msg = _call("pkv_paged_prefix_decode", PREFIX, kw)
    assert st == status and msg


@pytest.mark.parametrize("name,spec,kw", [("pkv_paged_prompt_attention", PROMPT, dict(S=0)),
                                          ("pkv_paged_prompt_attention", PROMPT, dict(T=0)),
                                          ("pkv_paged_prefix_decode", PREFIX, dict(S=0))])
def test_empty_calls(name, spec, kw):
    assert _call(name, spec, kw)[0] == 0


ROTARY = dict(qo=FAKE, q=FAKE, k=FAKE, v=FAKE, qos=1024, qs=1024, ks=512, vs=512, pos=FAKE, cs=FAKE, mp=100, rot=128, il=0,
              kp=FAKE, vp=FAKE, slots=FAKE, T=4, hq=8, hkv=4, D=128, nb=64, dt=0)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), 1), (dict(hq=-1), 1), (dict(hkv=0), 1), (dict(nb=0), 1), (dict(mp=0), 1), (dict(D=80), 2), (dict(rot=0), 2),
    (dict(rot=144), 2), (dict(rot=24), 2), (dict(dt=7), 2), (dict(k=None), 1), (dict(q=None), 1), (dict(qo=None), 1),
    (dict(pos=None), 1), (dict(cs=None), 1), (dict(kp=None), 1), (dict(slots=None), 1), (dict(qs=1020), 1), (dict(ks=-8), 1),
    (dict(vs=4), 1), (dict(qos=1000), 1), (dict(qos=-1024), 1), (dict(q=FAKE + 2), 1), (dict(cs=FAKE + 8), 1),
    (dict(pos=FAKE + 2), 1), (dict(slots=FAKE + 4), 1), (dict(vp=FAKE + 8), 1), (dict(hq=4097), 2),
])
def test_rotary_refusals(kw, status):
    st, msg = _call("pkv_rotary_and_cache", ROTARY, kw)
    assert st == status and msg


def test_binding_refuses_before_it_calls():
    q = torch.zeros(3, 4, 64, dtype=torch.float16)
    pool = torch.zeros(2, 2, 16, 64, dtype=torch.float16)
    i32 = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        B.paged_prompt_attention(q, q, pool, pool, i32.view(3, 1), i32, i32, 0.1)
    with pytest.raises(ValueError, match="CUDA"):
        B.paged_prefix_decode(q, q, pool, pool, i32.view(3, 1), i32, i32, i32, 0.1)
    with pytest.raises(ValueError, match="CUDA"):
        B.rotary_and_cache(q, q, q, q, i32, torch.zeros(4, 64), pool, pool, i32.long())
