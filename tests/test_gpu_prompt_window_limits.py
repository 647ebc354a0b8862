"""Windows that are no limit, with more query tokens than tokens: no position is lost to the window's size."""

import numpy as np
import pytest
import torch

import test_gpu_prompt as P
from paged_kv_cache_217_gb300 import binding as B
from test_gpu_prompt import _built  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 2, 2 ** 30, 2 ** 31, 2 ** 32 + 1, 2 ** 40])
@pytest.mark.parametrize("hq,hkv,d", [(4, 4, 64), (4, 1, 128), (6, 2, 256)])
def test_windows_without_limit(window, hq, hkv, d):
    c = P.Case([60, 700, 3, 0, 200], [64, 300, 400, 9, 900], hq, hkv, d, "bf16", seed=60)
    out = c.run(window=window)
    assert torch.equal(out, c.run())
    c.check(out, heads=[hq - 1], wanted=set(range(0, 1673, 9)) | {3, 4, 63, 363, 760, 761, 763})


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 33 + 3])
def test_windows_without_limit_among_single_tokens(window):
    lens = np.random.default_rng(61).integers(0, 120, 240)
    new = np.ones(240, int)
    new[[3, 50]] = [90, 20]
    c = P.Case(lens, new, 4, 2, 64, "f16", seed=61)
    out = c.run(window=window)
    assert torch.equal(out, c.run())
    c.check(out, heads=[3])
    assert B.device_status(clear=True) == 0
