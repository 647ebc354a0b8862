"""The README's decode loop, run as it is printed there: sequences end one after the other, and their places take no
more blocks."""

import os
import re

import numpy as np
import pytest
import torch

import helpers as H
import oracle.int4 as O4
import paged_kv_cache_217_gb300 as pkv
from paged_kv_cache_217_gb300 import binding as B
from paged_kv_cache_217_gb300 import workloads as W

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    H.ensure_built()
    B.device_status(clear=True)
    yield


def _loop():
    with open(os.path.join(ROOT, "README.md")) as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    (code,) = [b for b in blocks if "extend_block_tables" in b]
    return compile(code, "README.md", "exec")


@pytest.mark.parametrize("captured", [False, True])
def test_the_decode_loop(captured):
    code = _loop()
    prompts, width, nb, hq, hkv, head_dim, steps = [5, 16, 33, 15, 64, 1], 8, 60, 8, 2, 64, 40
    S, ends = len(prompts), {3: [0, 4], 20: [2], 33: [5, 1]}
    host = B.BlockManager(nb, np.random.default_rng(0).permutation(nb).astype(np.int32))
    for s, n in enumerate(prompts):
        host.add_seq(s, n)
    host.free_seq(3)
    host.fork(1, 3)                               # place 3 shares place 1's block
    prompts[3] = prompts[1]
    i32 = lambda a: torch.as_tensor(np.asarray(a), dtype=torch.int32).cuda()  # noqa: E731
    tables, lens = (i32(a) for a in host.block_tables(range(S), width))
    free = host.free_stack()
    ns = dict(torch=torch, pkv=pkv, head_dim=head_dim, tables=tables, lens=lens, new_tokens=i32(np.ones(S)),
              free_stack=i32(np.concatenate((free, np.zeros(nb - len(free), np.int32)))), free_count=i32([len(free)]),
              refcounts=i32([host.refcount(b) for b in range(nb)]), finished=i32(np.zeros(S)),
              slots=torch.empty(S, dtype=torch.int64, device="cuda"),
              pairs=torch.empty((S, 2), dtype=torch.int64, device="cuda"),
              kv4=torch.empty((nb, hkv, 18 * head_dim), dtype=torch.uint8, device="cuda"))
    new = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    ns.update(k_new=new(S, hkv, head_dim), v_new=new(S, hkv, head_dim), q=new(S, hq, head_dim), out=new(S, hq, head_dim))
    # the prompts' rows, and each sequence's rows as the oracle keeps them
    rows = [[[], []] for _ in range(S)]
    for s in (0, 1, 2, 4, 5):
        k, v = (W.normal_values((prompts[s], hkv, head_dim), "bf16", 10 * s + i, "cuda") for i in (0, 1))
        at = tables[s, torch.arange(prompts[s], device="cuda") // 16].long() * 16 + torch.arange(prompts[s], device="cuda") % 16
        pkv.reshape_and_cache_int4(k, v, ns["kv4"], at)
        rows[s] = [list(H.to_f64(k)), list(H.to_f64(v))]
    rows[3] = [list(r) for r in rows[1]]
    live = set(range(S))
    if captured:
        before = {n: t.clone() for n, t in ns.items() if isinstance(t, torch.Tensor)}
        exec(code, ns)                            # (warm-up: library state, torch's own)
        for n, t in before.items():
            ns[n].copy_(t)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            exec(code, ns)
    for step in range(steps):
        for i, n in enumerate(("k_new", "v_new", "q")):
            ns[n].copy_(W.normal_values(tuple(ns[n].shape), "bf16", 1000 + 10 * step + i, "cuda"))
        for s in live:
            rows[s][0].append(H.to_f64(ns["k_new"])[s])
            rows[s][1].append(H.to_f64(ns["v_new"])[s])
            host.append_slot(s)
        ns["finished"].copy_(i32([s in ends.get(step, []) for s in range(S)]))
        graph.replay() if captured else exec(code, ns)
        torch.cuda.synchronize()
        # attention of every place over its own rows, zeros for empty ones
        got = H.to_f64(ns["out"])
        for s in range(S):
            if s not in live:
                assert not got[s].any()
                continue
            n = len(rows[s][0])
            parts = []
            for r in rows[s]:
                c, p = O4.quantize(np.array(r), "bf16")
                pad = -n % 16
                c, p = np.pad(c, ((0, pad), (0, 0), (0, 0))), np.pad(p, ((0, pad), (0, 0), (0, 0), (0, 0)))
                parts += [a.reshape(-1, 16, *a.shape[1:]).swapaxes(1, 2) for a in (c, p)]
            want, bound = O4.decode(W.to_numpy_storage(ns["q"][s:s + 1], "bf16"), *parts, np.arange(-(-n // 16))[None], [n],
                                    head_dim ** -0.5, "bf16")
            assert np.all(np.abs(got[s] - want[0]) <= bound[0] + 2.0 ** -8 * (np.abs(want[0]) + bound[0]))
        for s in ends.get(step, []):
            host.free_seq(s)
            live.remove(s)
        want_tables, want_lens = host.block_tables(sorted(live), width)
        assert lens.cpu().numpy()[sorted(live)].tolist() == want_lens.tolist()
        assert int(ns["free_count"]) == len(host.free_stack())
        empty = [s for s in range(S) if s not in live]
        assert not lens[empty].any() and (tables[empty] == -1).all()
    assert ns["new_tokens"].cpu().tolist() == [int(s in live) for s in range(S)]
    assert B.device_status(clear=True) == 0
