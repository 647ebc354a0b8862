"""What must hold of the prompt calls' host code: everything is enqueued under the lock of the stream, and the
workspace that a size call names is enough for any call of the sizes."""

import re
from pathlib import Path

import pytest

from paged_kv_cache_217_gb300 import binding as B

CSRC = Path(B.__file__).parent / "csrc"


@pytest.mark.parametrize("name", ["prompt_impl"])
def test_launches_are_under_the_lock(name):
    text = (CSRC / "api.cu").read_text()
    body = re.search(r"\n(extern \"C\" )?pkv_status_t " + name + r"\(.*?\n}\n", text, re.S).group(0)
    first = min(m.start() for m in re.finditer(r"pkv::launch_|cudaMemsetAsync", body))
    assert 0 <= body.find("const EnqueueLock lock(stream);") < first


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 2), (40, 40), (32, 8), (64, 1)])
def test_workspace_sizes(hq, hkv, d):
    for tokens, seqs in ((1, 1), (7, 3), (1000, 30), (128, 128), (4096, 500)):
        n = B.prompt_workspace_size(tokens, seqs, hq, hkv, d, 64)
        assert n > 0 and n % 16 == 0
        p = B.prefix_workspace_size(seqs, min(seqs, 3), hq, hkv, d, 64)
        assert p > 0 and p % 16 == 0
