"""The 4-bit cache, latent attention and the device block tables run together, as a decode loop uses them:
tables and slots from the requests' lengths, copy-on-write copies, cache write, attention -- eagerly against
the host block manager and the oracles, captured into CUDA graphs, and on several streams."""

import numpy as np
import pytest
import torch

import helpers as H
import oracle.int4 as O4
import oracle.latent as OL
from paged_kv_cache_217_gb300 import binding as B
from paged_kv_cache_217_gb300 import workloads as W

pytestmark = pytest.mark.gpu

HALF_STEP = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    H.ensure_built()
    B.device_status(clear=True)
    yield


class Loop:
    """A batch that starts from prompts (some shared by two samples) and appends a token per sequence and step."""

    def __init__(self, prompts, width=8, nb=200, seed=0):
        self.S = 2 * len(prompts)
        order = np.random.default_rng(seed).permutation(nb).astype(np.int32)
        self.host = B.BlockManager(nb, order)
        for i, n in enumerate(prompts):
            self.host.add_seq(2 * i, n)
            self.host.fork(2 * i, 2 * i + 1)
        tables, lens = self.host.block_tables(range(self.S), width)
        stack = np.zeros(nb, np.int32)
        free = self.host.free_stack()
        stack[:len(free)] = free
        dev = lambda a, t: torch.as_tensor(np.asarray(a), dtype=t).cuda()  # noqa: E731
        self.width, self.nb = width, nb
        self.tables, self.lens = dev(tables, torch.int32), dev(lens, torch.int32)
        self.stack, self.count = dev(stack, torch.int32), dev([len(free)], torch.int32)
        self.ref = dev([self.host.refcount(b) for b in range(nb)], torch.int32)
        self.one = torch.ones(self.S, dtype=torch.int32, device="cuda")
        self.slots = torch.empty(self.S, dtype=torch.int64, device="cuda")
        self.pairs = torch.empty((self.S, 2), dtype=torch.int64, device="cuda")

    def extend(self):
        B.extend_block_tables(self.tables, self.lens, self.one, self.stack, self.count, self.slots, refcounts=self.ref,
                              cow_pairs=self.pairs)

    def host_step(self):
        """The same step by the host manager: its slots and pairs must be the device's."""
        slots, pairs = self.host.append_slots(range(self.S))
        assert self.slots.cpu().tolist() == slots.tolist()
        got = self.pairs.cpu().numpy()
        assert got[:len(pairs)].tolist() == pairs.tolist() and (got[len(pairs):] == -1).all()
        tables, lens = self.host.block_tables(range(self.S), self.width)
        assert np.array_equal(self.tables.cpu().numpy(), tables) and np.array_equal(self.lens.cpu().numpy(), lens)
        return tables, lens


class Int4Loop(Loop):
    def __init__(self, prompts, hq=8, hkv=2, D=64, dtype="bf16", **kw):
        super().__init__(prompts, **kw)
        self.dtype, self.scale, self.D, self.hkv, self.hq = dtype, D ** -0.5, D, hkv, hq
        self.cache = torch.zeros((self.nb, hkv, 18 * D), dtype=torch.uint8, device="cuda")
        k, v = (W.normal_values((self.nb * 16, hkv, D), dtype, s, "cuda") for s in (1, 2))
        B.reshape_and_cache_int4(k, v, self.cache, torch.arange(self.nb * 16, device="cuda"))
        # the oracle's copy: codes and pairs by block
        self.rows = [list(O4.quantize(H.to_f64(x), dtype)) for x in (k, v)]
        self.rows = [[a.reshape(self.nb, 16, *a.shape[1:]).swapaxes(1, 2).copy() for a in r] for r in self.rows]
        self.k, self.v = (torch.empty((self.S, hkv, D), dtype=k.dtype, device="cuda") for _ in range(2))
        self.q = torch.empty((self.S, hq, D), dtype=k.dtype, device="cuda")
        self.out = torch.empty_like(self.q)

    def feed(self, step):
        for i, x in enumerate((self.k, self.v, self.q)):
            x.copy_(W.normal_values(tuple(x.shape), self.dtype, 100 * step + i, "cuda"))

    def step(self):
        self.extend()
        B.copy_blocks_int4(self.cache, self.pairs)
        B.reshape_and_cache_int4(self.k, self.v, self.cache, self.slots)
        B.paged_attention_decode_int4(self.out, self.q, self.cache, self.tables, self.lens, self.scale)

    def check(self):
        pairs, slots = self.pairs.cpu().numpy(), self.slots.cpu().numpy()
        tables, lens = self.host_step()
        for rows, x in zip(self.rows, (self.k, self.v)):
            new = O4.quantize(H.to_f64(x), self.dtype)
            for a, n in zip(rows, new):
                for src, dst in pairs.tolist():
                    if src >= 0:
                        a[dst] = a[src]
                for s, slot in enumerate(slots.tolist()):
                    a[slot // 16, :, slot % 16] = n[s]
        (kc, kp), (vc, vp) = self.rows
        want, bound = O4.decode(W.to_numpy_storage(self.q, self.dtype), kc, kp, vc, vp, tables, lens, self.scale,
                                self.dtype)
        got = H.to_f64(self.out)
        assert np.all(np.abs(got - want) <= bound + HALF_STEP[self.dtype] * (np.abs(want) + bound))


class LatentLoop(Loop):
    def __init__(self, prompts, heads=16, dtype="bf16", **kw):
        super().__init__(prompts, **kw)
        self.dtype, self.scale = dtype, 192 ** -0.5
        self.cache = W.normal_values((self.nb, 16, 576), dtype, 1, "cuda")
        self.mirror = W.to_numpy_storage(self.cache, dtype).copy()
        self.proj = torch.empty((self.S, 576), dtype=self.cache.dtype, device="cuda")
        self.q = torch.empty((self.S, heads, 576), dtype=self.cache.dtype, device="cuda")
        self.out = torch.empty((self.S, heads, 512), dtype=self.cache.dtype, device="cuda")

    def feed(self, step):
        for i, x in enumerate((self.proj, self.q)):
            x.copy_(W.normal_values(tuple(x.shape), self.dtype, 100 * step + i, "cuda"))

    def step(self):
        self.extend()
        B.copy_blocks_latent(self.cache, self.pairs)
        B.latent_cache_write(self.proj[:, :512], self.proj[:, 512:], self.cache, self.slots)
        B.paged_latent_decode(self.out, self.q, self.cache, self.tables, self.lens, self.scale)

    def check(self):
        pairs, slots = self.pairs.cpu().numpy(), self.slots.cpu().numpy()
        tables, lens = self.host_step()
        for src, dst in pairs.tolist():
            if src >= 0:
                self.mirror[dst] = self.mirror[src]
        p = W.to_numpy_storage(self.proj, self.dtype)
        self.mirror = OL.cache_write(p[:, :512], p[:, 512:], self.mirror, slots)
        assert np.array_equal(W.to_numpy_storage(self.cache, self.dtype).view(np.uint16), self.mirror.view(np.uint16))
        want, bound = OL.decode(W.to_numpy_storage(self.q, self.dtype), self.mirror, tables, lens, self.scale,
                                self.dtype)
        got = H.to_f64(self.out)
        assert np.all(np.abs(got - want) <= bound + HALF_STEP[self.dtype] * (np.abs(want) + bound))


LOOPS = [lambda: Int4Loop([5, 16, 33, 70]), lambda: Int4Loop([40, 1] * 9, hq=12, hkv=12, nb=400),
         lambda: LatentLoop([5, 16, 33, 70])]


@pytest.mark.parametrize("make", LOOPS)
def test_a_decode_loop(make):
    loop = make()
    for step in range(4):
        loop.feed(step)
        loop.step()
        loop.check()
    assert B.device_status(clear=True) == 0


@pytest.mark.parametrize("make", LOOPS)
def test_a_captured_decode_loop(make):
    loop = make()
    stream = torch.cuda.Stream()
    state = [t.clone() for t in (loop.tables, loop.lens, loop.stack, loop.count, loop.ref, loop.cache)]
    with torch.cuda.stream(stream):
        loop.feed(0)
        loop.step()                              # (warm-up: function attributes, library state)
        for t, x in zip((loop.tables, loop.lens, loop.stack, loop.count, loop.ref, loop.cache), state):
            t.copy_(x)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            loop.step()
    torch.cuda.synchronize()
    for t, x in zip((loop.tables, loop.lens, loop.stack, loop.count, loop.ref, loop.cache), state):
        assert torch.equal(t, x)                 # a capture runs nothing
    for step in range(3):
        loop.feed(step)
        graph.replay()
        torch.cuda.synchronize()
        loop.check()
    assert B.device_status(clear=True) == 0


def test_two_graphs_of_two_batches_replayed_at_once():
    loops = [Int4Loop([300, 40] * 4, hq=12, hkv=12, width=24, nb=800, seed=3), LatentLoop([300, 7], width=24, seed=4),
             Int4Loop([90, 3, 250], width=24, seed=5)]
    graphs, streams = [], [torch.cuda.Stream() for _ in loops]
    for loop, stream in zip(loops, streams):
        loop.feed(1)
        torch.cuda.synchronize()
        loop.step()
        loop.check()
        loop.feed(2)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            loop.step()
        graphs.append(graph)
    torch.cuda.synchronize()
    for graph, stream in zip(graphs, streams):   # each has a workspace of its own
        with torch.cuda.stream(stream):
            graph.replay()
    torch.cuda.synchronize()
    for loop in loops:
        loop.check()


def test_calls_on_several_streams_at_once():
    S, hq, hkv, D = 24, 24, 12, 128
    lens = np.random.default_rng(0).integers(1, 900, S).astype(np.int32)
    tables, _ = W.scattered_tables(lens, W.pool_size(lens, 1.2), 1)
    nb = W.pool_size(lens, 1.2)
    cache = torch.empty((nb, hkv, 18 * D), dtype=torch.uint8, device="cuda")
    k, v = (W.normal_values((nb * 16, hkv, D), "f16", s, "cuda") for s in (1, 2))
    B.reshape_and_cache_int4(k, v, cache, torch.arange(nb * 16, device="cuda"))
    rows = W.normal_values((nb, 16, 576), "f16", 3, "cuda")
    tab, ln = torch.from_numpy(tables).cuda(), torch.from_numpy(lens).cuda()
    q = [W.normal_values((S, hq, D), "f16", 10 + i, "cuda") for i in range(3)]
    ql = [W.normal_values((S, 20, 576), "f16", 20 + i, "cuda") for i in range(3)]
    run = lambda i: (B.paged_attention_decode_int4(torch.empty_like(q[i]), q[i], cache, tab, ln, 0.1),  # noqa: E731
                     B.paged_latent_decode(torch.empty((S, 20, 512), dtype=q[i].dtype, device="cuda"), ql[i], rows,
                                           tab, ln, 0.07))
    alone = [run(i) for i in range(3)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(5):
        outs = []
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                outs.append(run(i))
        torch.cuda.synchronize()
        for a, b in zip(alone, outs):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert B.device_status(clear=True) == 0


def test_binding_refusals():
    q = torch.zeros((2, 4, 64), dtype=torch.float16, device="cuda")
    cache = torch.zeros((3, 2, 18 * 64), dtype=torch.uint8, device="cuda")
    tab, lens = torch.zeros((2, 1), dtype=torch.int32, device="cuda"), torch.ones(2, dtype=torch.int32, device="cuda")
    slots = torch.zeros(2, dtype=torch.int64, device="cuda")
    ok = lambda **kw: B.paged_attention_decode_int4(**{**dict(out=torch.empty_like(q), q=q, kv_cache=cache,  # noqa: E731
                                                              block_tables=tab, context_lens=lens, scale=1.0), **kw})
    ok()
    for kw, err in ((dict(out=q.float()), TypeError), (dict(kv_cache=cache.int()), TypeError),
                    (dict(block_tables=tab.long()), TypeError), (dict(context_lens=lens[:1]), ValueError),
                    (dict(kv_cache=cache[:, :, :-18].contiguous()), ValueError), (dict(q=q.float(), out=q.float()), TypeError),
                    (dict(q=q.transpose(0, 1)), ValueError), (dict(context_lens=lens.cpu()), ValueError),
                    (dict(scale=float("nan")), B.PagedKVError)):
        with pytest.raises(err):
            ok(**kw)
    k = torch.zeros((2, 2, 64), dtype=torch.float16, device="cuda")
    for args, err in (((k, k, cache, slots.int()), TypeError), ((k, k[:1], cache, slots), ValueError),
                      ((k, k.bfloat16(), cache, slots), ValueError), ((k, k, cache[:, :1].contiguous(), slots), ValueError),
                      ((k.float(), k.float(), cache, slots), TypeError)):
        for fn in (B.reshape_and_cache_int4, B.gather_cache_int4):
            with pytest.raises(err):
                fn(*args)
    rows = torch.zeros((3, 16, 576), dtype=torch.float16, device="cuda")
    lat, rope = torch.zeros((2, 512), dtype=torch.float16, device="cuda"), torch.zeros((2, 64), dtype=torch.float16, device="cuda")
    for args, err in (((lat, rope, rows, slots.int()), TypeError), ((lat.bfloat16(), rope, rows, slots), TypeError),
                      ((lat[:1], rope, rows, slots), ValueError), ((lat.t().contiguous().t(), rope, rows, slots), ValueError),
                      ((lat, torch.zeros((2, 68), dtype=torch.float16, device="cuda")[:, 4:], rows, slots), B.PagedKVError),
                      ((lat, rope, rows[:, :, :512].contiguous(), slots), ValueError)):
        with pytest.raises(err):
            B.latent_cache_write(*args)
    ql = torch.zeros((2, 4, 576), dtype=torch.float16, device="cuda")
    with pytest.raises(ValueError):
        B.paged_latent_decode(torch.empty((2, 4, 576), dtype=ql.dtype, device="cuda"), ql, rows, tab, lens, 1.0)
    with pytest.raises(TypeError):
        B.paged_latent_decode(torch.empty((2, 4, 512), dtype=ql.dtype, device="cuda"), ql, rows.bfloat16(), tab, lens, 1.0)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    with pytest.raises(ValueError):
        B.extend_block_tables(tab, lens, i32(2), i32(5), i32(1), slots, refcounts=i32(5))
    with pytest.raises(TypeError):
        B.extend_block_tables(tab, lens, i32(2), i32(5), i32(1), slots.int())
    with pytest.raises(ValueError):
        B.release_sequences(tab, lens, i32(2), i32(5), i32(1), refcounts=i32(4))
    assert B.device_status(clear=True) == 0


def test_workspaces_elsewhere_are_refused():
    S, mb = 40, 130
    tab, lens = torch.zeros((S, mb), dtype=torch.int32, device="cuda"), torch.zeros(S, dtype=torch.int32, device="cuda")
    q4 = torch.zeros((S, 12, 64), dtype=torch.float16, device="cuda")
    ql = torch.zeros((S, 16, 576), dtype=torch.float16, device="cuda")
    i32 = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    calls = [
        lambda ws: B.paged_attention_decode_int4(torch.empty_like(q4), q4, torch.zeros((4, 12, 1152), dtype=torch.uint8,
                                                 device="cuda"), tab, lens, 1.0, workspace=ws),
        lambda ws: B.paged_latent_decode(torch.empty((S, 16, 512), dtype=ql.dtype, device="cuda"), ql,
                                         torch.zeros((4, 16, 576), dtype=ql.dtype, device="cuda"), tab, lens, 1.0,
                                         workspace=ws),
        lambda ws: B.extend_block_tables(tab, lens, i32(S), i32(4), i32(1), torch.zeros(5000, dtype=torch.int64,
                                         device="cuda"), workspace=ws),
        lambda ws: B.release_sequences(tab, lens, i32(S), i32(4), i32(1), workspace=ws)]
    size = 64 << 20
    for call in calls:
        call(torch.empty(size, dtype=torch.uint8, device="cuda"))
        for bad in (torch.empty(size, dtype=torch.uint8), torch.empty(2 * size, dtype=torch.uint8, device="cuda")[::2]):
            with pytest.raises(ValueError):
                call(bad)
        with pytest.raises(B.PagedKVError):
            call(torch.empty(size, dtype=torch.uint8, device="cuda")[8:])
    assert B.device_status(clear=True) == 0


@pytest.mark.parametrize("S", [6, 160])
def test_device_tables_feed_the_launch_plan(S):
    """extend_block_tables, then the 16-bit step's plan, cache write and planned decode, with no wait between:
    the same bits as over the host manager's tables."""
    hq, hkv, D, width, nb = 4, 2, 64, 8, 1200
    rng = np.random.default_rng(S)
    host = B.BlockManager(nb, rng.permutation(nb).astype(np.int32))
    prompts = rng.integers(1, 90, S)
    for s, n in enumerate(prompts):
        host.add_seq(s, int(n))
    tables, lens = host.block_tables(range(S), width)
    free = host.free_stack()
    stack = np.zeros(nb, np.int32)
    stack[:len(free)] = free
    dev = lambda a: torch.as_tensor(np.asarray(a), dtype=torch.int32).cuda()  # noqa: E731
    tab, ln, stk, cnt, one = dev(tables), dev(lens), dev(stack), dev([len(free)]), dev(np.ones(S))
    slots = torch.empty(S, dtype=torch.int64, device="cuda")
    kp, vp = (W.normal_values((nb, hkv, 16, D), "bf16", s, "cuda") for s in (1, 2))
    k, v = (W.normal_values((8, S, hkv, D), "bf16", s, "cuda") for s in (3, 4))
    q = W.normal_values((8, S, hq, D), "bf16", 5, "cuda")
    outs = torch.empty_like(q)
    kp2, vp2 = kp.clone(), vp.clone()
    torch.cuda.synchronize()
    for i in range(8):
        B.extend_block_tables(tab, ln, one, stk, cnt, slots)
        B.paged_attention_plan(ln, tab, hq, hkv, D)
        B.reshape_and_cache(k[i], v[i], kp, vp, slots)
        B.paged_attention_decode(outs[i], q[i], kp, vp, tab, ln, 0.125, planned=True)
    torch.cuda.synchronize()
    for i in range(8):
        host_slots, pairs = host.append_slots(range(S))
        assert len(pairs) == 0
        tables, lens = host.block_tables(range(S), width)
        B.reshape_and_cache(k[i], v[i], kp2, vp2, torch.from_numpy(host_slots).cuda())
        t2, l2, out = dev(tables), dev(lens), torch.empty_like(q[i])
        B.paged_attention_plan(l2, t2, hq, hkv, D)
        torch.cuda.synchronize()
        B.paged_attention_decode(out, q[i], kp2, vp2, t2, l2, 0.125, planned=True)
        assert torch.equal(out, outs[i])
    assert torch.equal(kp, kp2) and torch.equal(vp, vp2) and B.device_status(clear=True) == 0
