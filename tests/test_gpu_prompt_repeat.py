"""The same inputs give the same bits, whatever ran before on the SMs and left in their shared memory."""

import pytest
import torch

import test_gpu_prompt as P
from test_gpu_prompt import _built  # noqa: F401

pytestmark = pytest.mark.gpu


def before(d, size):
    """A call whose queries of that size fill the query tiles of every SM."""
    c = P.Case([300] * 80, [300] * 80, 16, 1, d, "bf16", seed=70)
    c.q.mul_(size)
    c.run()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new", [[1] * 7, [5, 1, 3, 14], [1, 2, 200, 15]])
@pytest.mark.parametrize("hq,hkv", [(8, 1), (3, 1), (7, 1), (6, 2)])
def test_bits_after_other_calls(hq, hkv, new, d):
    c = P.Case([2000, 700, 5000, 901, 64, 130, 333][:len(new)], new, hq, hkv, d, "bf16", seed=71)
    group, blocks = torch.tensor([0, 3], dtype=torch.int32, device="cuda"), torch.tensor([40], dtype=torch.int32, device="cuda")
    p = P.prefix_case([2000, 700, 5000, 901], hq, hkv, d, "bf16", [0, 3], [40], seed=72)
    p.groups, p.blocks = group, blocks
    first = None
    for size in (0.0, 300.0, 20.0, 1.0):
        before(d, size)
        out = c.run()
        before(d, size)
        behind = P.prefix_run(p)
        first = (out, behind) if first is None else first
        assert torch.equal(out, first[0]) and torch.equal(behind, first[1])
    c.check(first[0], heads=[hq - 1], wanted=set(range(0, sum(new), 5)))
