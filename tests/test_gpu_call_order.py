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


def _decodes(seed, S, hq, hkv, heads, most, dtype="f16"):
    """(list-schedule 4-bit decode, latent decode, 16-bit split decode) of one batch, as calls without arguments."""
    rng = np.random.default_rng(seed)
    lens_np = rng.integers(1, most, S).astype(np.int32)
    nb = W.pool_size(lens_np, 1.2) + 1
    tab, lens = _i32(W.scattered_tables(lens_np, nb, seed)[0]), _i32(lens_np)
    D = 64
    pool = torch.empty((nb, hkv, 18 * D), dtype=torch.uint8, device="cuda")
    k, v = (W.normal_values((nb * 16, hkv, D), dtype, seed + i, "cuda") for i in (1, 2))
    B.reshape_and_cache_int4(k, v, pool, torch.arange(nb * 16, device="cuda"))
    rows = W.normal_values((nb, 16, 576), dtype, seed + 3, "cuda")
    q, ql = W.normal_values((S, hq, D), dtype, seed + 4, "cuda"), W.normal_values((S, heads, 576), dtype, seed + 5, "cuda")
    kp, vp = (W.normal_values((nb, hkv, 16, D), dtype, seed + i, "cuda") for i in (6, 7))
    assert B.int4_workspace_size(S, hq, hkv, D, tab.shape[1]) > 0
    return (lambda: B.paged_attention_decode_int4(torch.empty_like(q), q, pool, tab, lens, 0.1),
            lambda: B.paged_latent_decode(torch.empty((S, heads, 512), dtype=ql.dtype, device="cuda"), ql, rows, tab,
                                          lens, 0.07),
            lambda: B.paged_attention_decode(torch.empty_like(q), q, kp, vp, tab, lens, 0.1, partition_size=128))


def _tables(seed, S, n):
    """An extend of S prompts by two kernels, the release of every other one and the state after both."""
    rng = np.random.default_rng(seed)
    new, gone = _i32(rng.integers(1, 2 * n, S)), _i32(rng.integers(0, 2, S))
    width, total = (2 * n + 15) // 16, int(new.sum())
    nb = S * width
    order = _i32(rng.permutation(nb))
    assert B.lib().pkv_extend_workspace_size(S, total) > 0

    def run():
        tab = torch.full((S, width), -1, dtype=torch.int32, device="cuda")
        lens, stack = torch.zeros(S, dtype=torch.int32, device="cuda"), order.clone()
        count = torch.full((1,), nb, dtype=torch.int32, device="cuda")
        slots = torch.empty(total, dtype=torch.int64, device="cuda")
        B.extend_block_tables(tab, lens, new, stack, count, slots)
        full = tab.clone()
        B.release_sequences(tab, lens, gone, stack, count)
        return torch.cat([full.flatten(), tab.flatten(), lens, stack, count]), slots
    return run


def _plan_and_decode(seed, S):
    """A plan into the stream's workspace, which nothing uses, then a 16-bit decode that makes its own there."""
    rng = np.random.default_rng(seed)
    lens_np = rng.integers(1, 200, S).astype(np.int32)
    nb = W.pool_size(lens_np, 1.2) + 1
    tab, lens = _i32(W.scattered_tables(lens_np, nb, seed)[0]), _i32(lens_np)
    q = W.normal_values((S, 8, 64), "bf16", seed, "cuda")
    kp, vp = (W.normal_values((nb, 2, 16, 64), "bf16", seed + i, "cuda") for i in (1, 2))

    def run():
        B.paged_attention_plan(lens, tab, 8, 2, 64)
        return B.paged_attention_decode(torch.empty_like(q), q, kp, vp, tab, lens, 0.125)
    return run


def _same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b)) if isinstance(a, tuple) else torch.equal(a, b)


@pytest.mark.parametrize("stream", ["default", "own"])
def test_threads_that_share_a_stream(stream):
    """Calls of several kernels that pass state through the stream's workspace, each from a thread of its own: the same
    bits as alone."""
    jobs = [*_decodes(1, 30, 24, 12, 16, 700), *_decodes(50, 41, 20, 20, 128, 1500), _tables(7, 900, 12),
            _tables(8, 2000, 4), _plan_and_decode(9, 200), _plan_and_decode(10, 150)]
    alone = [job() for job in jobs]
    torch.cuda.synchronize()
    st = torch.cuda.default_stream() if stream == "default" else torch.cuda.Stream()

    def on_stream(job):
        def run():
            with torch.cuda.stream(st):
                return job()
        return run
    for round_ in range(3):
        for want, got in zip(alone, _from_threads([on_stream(j) for j in jobs], 40)):
            assert all(_same(want, g) for g in got)
    assert B.device_status(clear=True) == 0


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
