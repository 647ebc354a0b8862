"""A weighted mean of equal values is that value: the sum that outputs are divided by is that of the weights as the
products take them.

The products of a weight and a value are exact in fp32, and at most 125 steps of 16 positions and as many additions
follow, each off by 2^-22 of its result at most: under 2^-14 in all, while half a step of either type is 2^-12 of a
value or more. So the quotient rounds to the value itself."""

import numpy as np
import pytest
import torch

import helpers as H
import test_gpu_prompt as P
from test_gpu_prompt import _built  # noqa: F401

pytestmark = pytest.mark.gpu


def constant(c, dtype):
    """V of one value a channel, the last ones of a binade among them, where half a step is smallest."""
    last = 2.0 - {"f16": 2.0 ** -10, "bf16": 2.0 ** -7}[dtype]
    row = torch.randn(c.v.shape[-1], generator=torch.Generator().manual_seed(90)).to(c.v.dtype)
    row[::4], row[1::4] = last, -last / 8
    c.v[:] = row.cuda()
    return row.cuda()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hkv,d", [(4, 4, 64), (4, 1, 128), (6, 2, 256)])
@pytest.mark.parametrize("size", [0.5, 3.0])
def test_equal_values(size, hq, hkv, d, dtype):
    c = P.Case([1900, 700, 64, 65, 333, 1, 17], [9, 300, 64, 1, 130, 1, 2], hq, hkv, d, dtype, seed=90)
    row = constant(c, dtype)
    c.q.mul_(size)
    for causal, window in ((True, 0), (True, 70), (False, 0)):
        assert (c.run(causal, window) == row).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("seqs", [30, 240])
@pytest.mark.parametrize("hq,hkv,d", [(2, 2, 64), (8, 2, 128), (4, 2, 256)])
def test_equal_values_behind_prefixes(hq, hkv, d, seqs, dtype):
    lens = np.random.default_rng(91).integers(160, 900, seqs)
    c = P.prefix_case(lens, hq, hkv, d, dtype, [0, seqs - 2], [10], seed=91)
    row = constant(c, dtype)
    c.q.mul_(2)
    assert (P.prefix_run(c) == row).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_one_weight_above_the_reference(dtype):
    """A score that exceeds the first one by less than what moves the reference has a weight that is rounded, and all
    but alone: each sequence another one."""
    seqs = 400
    c = P.Case([129] * seqs, [1] * seqs, 1, 1, 64, dtype, seed=92, scale=1.0)
    row = constant(c, dtype)
    tables = c.tables.long()
    c.q.zero_()
    c.q[..., 0] = 1
    c.k.zero_()
    c.k[..., 0] = -100
    c.k[tables[:, 0], 0, 0, 0] = 0
    c.k[tables[:, 8], 0, 0, 0] = torch.linspace(4.9, 5.5, seqs, device="cuda").to(H.torch_dtype(dtype))
    assert (c.run() == row).all()
