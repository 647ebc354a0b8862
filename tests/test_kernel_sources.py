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


# Kernels that programmatic dependent launches start while their predecessor still runs, or right behind it: only
# griddepcontrol.wait makes the predecessor's stores visible. (launch_dependents itself needs no wait, a prefetch
# brings no value, and barriers and tensor memory are the CTA's own.)
GLOBAL = re.compile(r"__ldg\(|__ldcg\(|\b(lens|tables|header|order|rows|counters|groups|chunks|others)\[|"
                    r"\ba\.(context_lens|block_tables|q|desc|part_ml|part_o|refcounts|free_stack|free_count)\b|\*ra\b")


def _kernels(text):
    for m in re.finditer(r"__global__[^;{]*?\b(\w+)\s*\(([^{;]*)\)\s*\{", text):
        yield m.group(1), text[m.end():_block_end(text, m.end() - 1)]


@pytest.mark.parametrize("name", [n for n in SOURCES if "griddepcontrol.wait" in _source(n)])
def test_kernels_that_wait_do_so_before_they_touch_memory(name):
    found = 0
    for kernel, body in _kernels(_source(name)):
        at = body.find("griddepcontrol.wait")
        if at < 0:
            continue
        found += 1
        first = GLOBAL.search(body)
        assert first is None or first.start() > at, f"{kernel}: {body[first.start():first.start() + 60]!r} before the wait"
    assert found or name == "decode.cuh"          # (there the wait is a function of its own)


@pytest.mark.parametrize("launch", ["launch_decode_sk_f16", "launch_decode_f16", "launch_decode_int8", "launch_decode_int4",
                                    "launch_latent_decode", "launch_extend_block_tables", "launch_release_sequences"])
def test_launches_that_share_a_workspace_are_enqueued_together(launch):
    """Between the start of the function (or the block) that makes them and the launch the stream's lock is taken,
    and before it nothing is enqueued."""
    text = _source("api.cu")
    for m in re.finditer(rf"pkv::{launch}\(", text):
        body = text[text.rfind("\n}\n", 0, m.start()):m.start()]
        at = body.rfind("const EnqueueLock lock(stream);")
        enqueued = [body.find(w) for w in ("cudaMemsetAsync(", "launch_prefix_plan_ws(context_lens", "launch_seq_order(")]
        assert at >= 0 and body[at:].count("EnqueueLock") == 1
        first = min([e for e in enqueued if e >= 0], default=len(body))
        assert body.find("const EnqueueLock lock(stream);") < first


@pytest.mark.parametrize("launch", ["launch_prefix_plan_ws(context_lens", "pkv::launch_seq_order("])
def test_plans_are_enqueued_under_the_lock(launch):
    """Every plan that is written into a workspace: a decode's own, and pkv_paged_attention_plan's."""
    text = _source("api.cu")
    at = [m.start() for m in re.finditer(re.escape(launch), text)]
    assert len(at) == 3
    for i in at:
        body = text[text.rfind("\n}\n", 0, i):i]
        assert body.count("EnqueueLock lock(") == 1 or (body.count("EnqueueLock lock(") == 2 and "if (balanced) {" in body)
