"""Block tables and slot maps made on the device against the oracle block manager: the same blocks, slots,
copy-on-write pairs and reference counts as its appends in batch order; all-or-nothing failures; release."""

import numpy as np
import pytest
import torch

import helpers as H
from oracle.block_manager import OracleBlockManager
from paged_kv_cache_217_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    H.ensure_built()
    B.device_status(clear=True)
    yield


class Device:
    """Device state of a batch of S sequences over a pool."""

    def __init__(self, S, width, nb, order=None, shared=False):
        order = np.arange(nb, dtype=np.int32) if order is None else np.asarray(order, np.int32)
        self.tables = torch.full((S, width), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(S, dtype=torch.int32, device="cuda")
        self.stack = torch.from_numpy(order.copy()).cuda()
        self.count = torch.tensor([nb], dtype=torch.int32, device="cuda")
        self.ref = torch.zeros(nb, dtype=torch.int32, device="cuda") if shared else None
        self.pairs = torch.full((S, 2), -9, dtype=torch.int64, device="cuda") if shared else None
        self.info = torch.zeros(4, dtype=torch.int32, device="cuda")

    def extend(self, new, capacity=None, **kw):
        new = torch.as_tensor(np.asarray(new, np.int32)).cuda()
        n = int(new.clamp(min=0).sum()) if capacity is None else capacity
        slots = torch.full((n,), -5, dtype=torch.int64, device="cuda")
        B.extend_block_tables(self.tables, self.lens, new, self.stack, self.count, slots, refcounts=self.ref,
                              cow_pairs=self.pairs, info=self.info, **kw)
        return slots.cpu().numpy()

    def release(self, finished):
        B.release_sequences(self.tables, self.lens, torch.as_tensor(np.asarray(finished, np.int32)).cuda(), self.stack,
                            self.count, refcounts=self.ref)

    def state(self):
        return [t.cpu().numpy().copy() for t in (self.tables, self.lens, self.stack, self.count, self.ref)
                if t is not None]


def _oracle_extend(bm, new):
    """append_slot new[s] times for each sequence in order -> slots, pairs."""
    slots, pairs = [], []
    for s, n in enumerate(new):
        for _ in range(n):
            slot, src, dst = bm.append_slot(s)
            slots.append(slot)
            if src >= 0:
                pairs.append((src, dst))
    return slots, pairs


def _same(dev, bm, S):
    tables, lens = dev.tables.cpu().numpy(), dev.lens.cpu().numpy()
    for s in range(S):
        want = bm.block_table(s)
        assert lens[s] == bm.length(s)
        assert tables[s, :len(want)].tolist() == want and (tables[s, len(want):] == -1).all()
    n = int(dev.count)
    assert dev.stack.cpu().numpy()[:n].tolist() == bm.free
    if dev.ref is not None:
        assert dev.ref.cpu().numpy().tolist() == bm.refcount


@pytest.mark.parametrize("S,most,steps,pad", [(1, 1, 40, 0), (5, 3, 12, 7), (64, 40, 6, 0), (1024, 5, 4, 1),
                                             (1025, 3, 3, 2), (3000, 2, 3, 0), (7, 900, 3, 5)])
@pytest.mark.parametrize("shared", [False, True])
def test_extend_follows_the_block_manager(S, most, steps, pad, shared):
    rng = np.random.default_rng(S + most)
    width = (most * steps + 15) // 16 + 1
    nb = S * width
    order = rng.permutation(nb)
    dev = Device(S, width, nb, order, shared)
    bm = OracleBlockManager(nb, initial_free_order=order)
    for s in range(S):
        bm.add_seq(s, 0)
    for _ in range(steps):
        new = rng.integers(0, most, size=S, endpoint=True)
        slots = dev.extend(new, int(new.sum()) + pad)
        want, pairs = _oracle_extend(bm, new.tolist())
        assert slots[:len(want)].tolist() == want and (slots[len(want):] == -1).all()
        assert not pairs
        _same(dev, bm, S)
        assert dev.info.cpu().tolist()[:2] == [0, len(want)]
    assert B.device_status(clear=True) == 0


@pytest.mark.parametrize("prompts,n,S_extra", [(3, 4, 0), (1, 40, 3), (40, 30, 11), (700, 2, 0)])
def test_copy_on_write(prompts, n, S_extra):
    rng = np.random.default_rng(prompts * 100 + n)
    S = prompts * n + S_extra
    order = rng.permutation(prompts * 6 + S * 4)
    bm = OracleBlockManager(len(order), initial_free_order=order)
    place = rng.permutation(S)                    # siblings anywhere in the batch
    plen = rng.integers(1, 70, prompts)
    root = {}
    for i in range(S):
        s = int(place[i])
        if i < prompts * n:
            if i % prompts in root:
                bm.fork(root[i % prompts], s)
            else:
                bm.add_seq(s, int(plen[i % prompts]))
                root[i % prompts] = s
        else:
            bm.add_seq(s, int(rng.integers(0, 30)))
    dev = Device(S, 8, len(order), shared=True)
    for s in range(S):
        t = bm.block_table(s)
        dev.tables[s, :len(t)] = torch.tensor(t, dtype=torch.int32)
        dev.lens[s] = bm.length(s)
    dev.stack[:len(bm.free)] = torch.tensor(bm.free, dtype=torch.int32)
    dev.count[0] = len(bm.free)
    dev.ref.copy_(torch.tensor(bm.refcount, dtype=torch.int32))
    for step in range(4):
        new = rng.integers(0, 3, size=S, endpoint=True) if step else np.ones(S, int)
        slots = dev.extend(new, int(new.sum()) + 3)
        want, pairs = _oracle_extend(bm, new.tolist())
        assert slots[:len(want)].tolist() == want
        got = dev.pairs.cpu().numpy()
        assert got[:len(pairs)].tolist() == [list(p) for p in pairs] and (got[len(pairs):] == -1).all()
        if step == 0:
            assert (len(pairs) > 0) == any(p % 16 for p in plen)
        _same(dev, bm, S)
    # release some, then all: the same blocks come back, pushed in ascending order
    gone = rng.random(S) < 0.5
    before = int(dev.count)
    dev.release(gone)
    for s in np.nonzero(gone)[0].tolist():
        bm.free_seq(s)
    back = dev.stack.cpu().numpy()[before:int(dev.count)]
    assert back.tolist() == sorted(set(bm.free) - set(dev.stack.cpu().numpy()[:before].tolist()))
    assert dev.ref.cpu().numpy().tolist() == bm.refcount
    assert (dev.tables[torch.from_numpy(gone).cuda()] == -1).all() and not dev.lens[torch.from_numpy(gone).cuda()].any()
    dev.release(np.ones(S, int))
    assert int(dev.count) == len(order) and not dev.ref.any()
    assert sorted(dev.stack.cpu().numpy().tolist()) == list(range(len(order)))
    assert B.device_status(clear=True) == 0


@pytest.mark.parametrize("S", [6, 1500])
@pytest.mark.parametrize("why,flag", [("blocks", 0x40), ("width", 0x2), ("negative", 0x2), ("length", 0x2),
                                      ("slots", 0x4), ("count", 0x1)])
def test_a_failed_call_changes_nothing(S, why, flag):
    nb, width = S * 3, 4
    dev = Device(S, width, nb, shared=True)
    dev.extend(np.full(S, 20))
    new, capacity = np.full(S, 10), S * 10
    if why == "blocks":
        new[:] = 40
        capacity = S * 40
    elif why == "width":
        new[S // 2] = 45
        capacity += 100
    elif why == "negative":
        new[S - 1] = -1
    elif why == "length":
        dev.lens[S - 1] = -4
    elif why == "slots":
        capacity -= 1
    else:
        dev.count[0] = nb + 1
    before = dev.state()
    slots = dev.extend(new, capacity)
    for a, b in zip(before, dev.state()):
        assert np.array_equal(a, b)
    assert (slots == -1).all() and (dev.pairs == -1).all()
    assert B.device_status(clear=True) == flag and dev.info.cpu().tolist() == [flag, 0, 0, 0]


def test_totals_past_32_bits_fail_cleanly():
    dev = Device(3000, 70000, 5)                  # 3e9 new tokens
    slots = dev.extend(np.full(3000, 1_000_000), capacity=8)
    assert (slots == -1).all() and int(dev.count) == 5 and B.device_status(clear=True) == 0x44


def test_separate_outputs_make_the_call_repeatable():
    dev = Device(40, 9, 400)
    dev.extend(np.arange(40) % 19)
    lens, count = torch.empty_like(dev.lens), torch.empty_like(dev.count)
    new = np.arange(40)[::-1] % 23
    a = dev.extend(new, new_lens=lens, new_free_count=count)
    tables = dev.tables.clone()
    b = dev.extend(new, new_lens=lens, new_free_count=count)
    assert np.array_equal(a, b) and torch.equal(tables, dev.tables)
    assert torch.equal(lens.cpu(), dev.lens.cpu() + torch.from_numpy(new.astype(np.int32).copy()))
    assert len(set(a.tolist())) == len(a)


def test_bad_entries_are_flagged():
    dev = Device(2, 3, 8)
    dev.extend([5, 20])
    dev.tables[0, 0] = 99                         # its tokens get no slot
    dev.stack[int(dev.count) - 1] = -4            # the next block taken is none
    slots = dev.extend([2, 14])
    assert slots[:2].tolist() == [-1, -1] and (slots[2:14] >= 0).all() and (slots[14:] == -1).all()
    assert B.device_status(clear=True) == 0x1
    dev.release([1, 1])
    assert B.device_status(clear=True) == 0x1     # the id outside the pool


def test_release_without_refcounts_and_after_a_window():
    dev = Device(3, 6, 30)
    dev.extend([40, 96, 17])
    free = int(dev.count)
    dev.tables[1, :3] = -1                        # released by a sliding window before
    dev.release([0, 1, 0])
    assert int(dev.count) == free + 3 and dev.lens.cpu().tolist() == [40, 0, 17]
    assert B.device_status(clear=True) == 0
    dev.tables[2, 0] = dev.tables[0, 0]           # one block in two tables, no counts
    dev.release([1, 0, 1])
    ids = dev.stack.cpu().numpy()[:int(dev.count)]
    assert len(set(ids.tolist())) == len(ids) and B.device_status(clear=True) == 0x1


def test_unaligned_slot_maps_and_no_sequences():
    dev = Device(3, 4, 20)
    new = torch.tensor([5, 0, 30], dtype=torch.int32, device="cuda")
    buf = torch.full((60,), -7, dtype=torch.int64, device="cuda")
    B.extend_block_tables(dev.tables, dev.lens, new, dev.stack, dev.count, buf[1:38])
    got = buf.cpu().numpy()
    assert got[0] == -7 and (got[1:36] >= 0).all() and got[36:38].tolist() == [-1, -1] and (got[38:] == -7).all()
    empty = Device(0, 4, 20)
    assert (empty.extend([], 9) == -1).all() and int(empty.count) == 20
    assert B.device_status(clear=True) == 0
