"""Orderings inside the kernels that no run can be relied on to show: read from the sources, on the CPU."""

import os
import re

import pytest

from paged_kv_cache_217_gb300 import build

SOURCES = sorted(f for f in os.listdir(build.CSRC) if f.endswith((".cu", ".cuh")))


def _source(name):
    """A source's text without comments."""
    with open(os.path.join(build.CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def _block_end(text, start):
    """Index behind the brace that closes the one at `start`."""
    depth = 0
    for i in range(start, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return i + 1
    raise AssertionError("unbalanced braces")


@pytest.mark.parametrize("name", [n for n in SOURCES if "mbar_init_fence();" in _source(n)])
def test_a_warp_waits_for_the_lane_that_initialised_its_barriers(name):
    """A lane's shared-memory writes are ordered for its warp by __syncwarp only (shuffles and votes order no memory):
    it is the first statement after a block that lane 0 alone initialises barriers in."""
    text = _source(name)
    blocks = [m for m in re.finditer(r"if \(lane == 0\) \{", text)]
    for m in blocks:
        end = _block_end(text, m.end() - 1)
        if "mbar_init(" in text[m.start():end]:
            assert text[end:].lstrip().startswith("__syncwarp();"), text[m.start():end + 120]
