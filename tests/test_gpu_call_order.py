"""Calls that follow one another with no wait between, or are made by two host threads at once, give what each gives
alone."""

import threading

import numpy as np
import pytest
import torch

import helpers as H
from paged_kv_cache_217_gb300 import binding as B
from paged_kv_cache_217_gb300 import workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    H.ensure_built()
    B.device_status(clear=True)
    yield


def _i32(a):
    return torch.as_tensor(np.asarray(a), dtype=torch.int32).cuda()


@pytest.mark.parametrize("S,partition", [(7, 0), (160, 0), (1000, 0), (160, B.SHARED_PREFIX)])
def test_a_plan_sees_the_tables_made_right_before_it(S, partition):
    """extend_block_tables and the launch plan in turn, 40 times without a wait: every plan equals, byte for byte,
    the one made of a copy of its step's tables and lengths with nothing else in flight."""
    hq, hkv, D, width = 8, 2, 64, 10
    rng = np.random.default_rng(S)
    tab = torch.full((S, width), -1, dtype=torch.int32, device="cuda")
    lens, count = _i32(np.zeros(S)), _i32([S * width])
    stack = _i32(rng.permutation(S * width))
    slots = torch.empty(3 * S, dtype=torch.int64, device="cuda")
    need = B.workspace_size(S, hq, hkv, D, width, partition)
    assert need > 0 and need % 16 == 0
    steps = 40
    new = [_i32(rng.integers(0, 4, S)) for _ in range(steps)]
    plans = torch.zeros((steps, need), dtype=torch.uint8, device="cuda")
    held = torch.empty((steps, S), dtype=torch.int32, device="cuda"), torch.empty((steps, S, width), dtype=torch.int32,
                                                                                  device="cuda")
    torch.cuda.synchronize()
    for i in range(steps):
        B.extend_block_tables(tab, lens, new[i], stack, count, slots)
        B.paged_attention_plan(lens, tab, hq, hkv, D, partition, workspace=plans[i])
        held[0][i].copy_(lens)
        held[1][i].copy_(tab)
    torch.cuda.synchronize()
    assert (held[0].cpu().numpy() == np.cumsum([n.cpu().numpy() for n in new], 0)).all()
    for i in range(steps):
        alone = torch.zeros(need, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        B.paged_attention_plan(held[0][i], held[1][i], hq, hkv, D, partition, workspace=alone)
        torch.cuda.synchronize()
        assert torch.equal(alone, plans[i])
    assert B.device_status(clear=True) == 0


def test_a_plan_replaces_the_one_before_it():
    S, hq, hkv, D, width = 500, 8, 2, 64, 40
    rng = np.random.default_rng(0)
    lens = [_i32(rng.integers(1, 16 * width, S)) for _ in range(2)]
    tab = _i32(rng.permutation(S * width).reshape(S, width))
    ws = torch.zeros(B.workspace_size(S, hq, hkv, D, width), dtype=torch.uint8, device="cuda")
    for _ in range(20):
        for n in lens:
            torch.cuda.synchronize()
            ws.zero_()
            B.paged_attention_plan(n, tab, hq, hkv, D, workspace=ws)
            torch.cuda.synchronize()
            alone = ws.clone()
            B.paged_attention_plan(lens[0] if n is lens[1] else lens[1], tab, hq, hkv, D, workspace=ws)
            B.paged_attention_plan(n, tab, hq, hkv, D, workspace=ws)
            torch.cuda.synchronize()
            assert torch.equal(ws, alone)


def _from_threads(jobs, rounds):
    """Each job `rounds` times from a thread of its own, all started together; its results in order."""
    start, results, errors = threading.Barrier(len(jobs)), [[] for _ in jobs], []

    def work(i):
        try:
            start.wait()
            for _ in range(rounds):
                results[i].append(jobs[i]())
        except BaseException as e:  # noqa: BLE001 (handed to the test)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    if errors:
        raise errors[0]
    return results


def test_a_thread_whose_first_call_is_a_decode():
    """The calls that encode tensor maps, from threads that have made no CUDA call before."""
    q, pool = W.normal_values((3, 8, 64), "f16", 1, "cuda"), W.normal_values((4, 2, 16, 64), "f16", 2, "cuda")
    ql, rows = W.normal_values((3, 16, 576), "f16", 3, "cuda"), W.normal_values((4, 16, 576), "f16", 4, "cuda")
    tab, lens = _i32([[0], [2], [3]]), _i32([5, 16, 1])
    out, ws = torch.zeros((2, 3, 8, 64), dtype=q.dtype, device="cuda"), torch.zeros(1 << 22, dtype=torch.uint8, device="cuda")
    outl = torch.zeros((2, 3, 16, 512), dtype=q.dtype, device="cuda")
    calls = [lambda i: B.paged_attention_decode(out[i], q, pool, pool, tab, lens, 0.1, workspace=ws),
             lambda i: B.paged_latent_decode(outl[i], ql, rows, tab, lens, 0.1, workspace=ws)]
    for call in calls:                            # (every tensor is there: the thread's first CUDA call is the decode's)
        call(0)
        _from_threads([lambda: call(1)], 1)
    torch.cuda.synchronize()
    assert torch.equal(out[0], out[1]) and torch.equal(outl[0], outl[1]) and out.any() and outl.any()
    assert B.device_status(clear=True) == 0
