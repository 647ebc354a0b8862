"""extend_block_tables of no sequences: the free count and info are results of the call all the same."""

import pytest
import torch

import helpers as H
from paged_kv_cache_217_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    H.ensure_built()
    B.device_status(clear=True)
    yield


@pytest.mark.parametrize("n", [0, 9, 5000])
@pytest.mark.parametrize("width", [0, 4])
@pytest.mark.parametrize("shared", [False, True])
def test_no_sequences_write_the_count_and_info(n, width, shared):
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    count, after, info = torch.full((1,), 13, dtype=torch.int32, device="cuda"), i32(1) - 7, i32(4) - 7
    slots = torch.full((n,), -5, dtype=torch.int64, device="cuda")
    kw = dict(refcounts=i32(20), cow_pairs=torch.zeros((0, 2), dtype=torch.int64, device="cuda")) if shared else {}
    B.extend_block_tables(i32(0, width), i32(0), i32(0), i32(20), count, slots, info=info, new_free_count=after, **kw)
    assert int(after) == 13 and int(count) == 13 and info.tolist() == [0, 0, 0, 0] and (slots == -1).all()
    B.extend_block_tables(i32(0, width), i32(0), i32(0), i32(20), count, slots, **kw)
    assert int(count) == 13 and B.device_status(clear=True) == 0
    count.fill_(21)                               # more free blocks than the pool has
    B.extend_block_tables(i32(0, width), i32(0), i32(0), i32(20), count, slots, info=info, new_free_count=after, **kw)
    assert info.tolist() == [1, 0, 0, 0] and int(after) == 21 and B.device_status(clear=True) == 1
