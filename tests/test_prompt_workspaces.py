"""The workspace that a size call names is what the calls ask for, on both sides of the rule that brings in a decode
grid, without a GPU: every call below is refused for its workspace, and its message names the bytes."""

import itertools
import re

import pytest

from paged_kv_cache_217_gb300 import binding as B
from test_prompt_abi import PREFIX, PROMPT, _call

WORKSPACE = 5
LARGE = 2 ** 28                              # blocks x KV heads beyond what a decode grid's offsets take


def needed(name, spec, **sizes):
    status, message = _call(name, spec, dict(sizes, ws=None, wsb=0))
    assert status == WORKSPACE, message
    n = int(re.search(r"of (\d+) bytes", message).group(1))
    for have in (0, n - 16, n - 1):
        assert _call(name, spec, dict(sizes, wsb=have))[0] == WORKSPACE
    assert _call(name, spec, dict(sizes, ws=0x10008))[0] == WORKSPACE      # 8-byte aligned
    return n


HEADS = [(1, 1), (8, 2), (40, 40), (32, 8), (64, 1)]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv", HEADS)
def test_prompts(hq, hkv, d):
    for (tokens, seqs), mb in itertools.product([(1, 1), (7, 3), (1000, 30), (128, 128), (470, 460), (4096, 500)], [1, 4, 700]):
        named = B.prompt_workspace_size(tokens, seqs, hq, hkv, d, mb)
        sizes = dict(T=tokens, S=seqs, hq=hq, hkv=hkv, D=d, mb=mb)
        assert max(needed("pkv_paged_prompt_attention", PROMPT, nb=nb, **sizes) for nb in (64, LARGE // hkv)) == named


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv", HEADS)
def test_prefixes(hq, hkv, d):
    for (seqs, groups), mb in itertools.product([(1, 0), (1, 1), (3, 2), (60, 1), (128, 128), (460, 0), (500, 7)], [1, 4, 700]):
        named = B.prefix_workspace_size(seqs, groups, hq, hkv, d, mb)
        sizes = dict(S=seqs, n=groups, hq=hq, hkv=hkv, D=d, mb=mb)
        assert max(needed("pkv_paged_prefix_decode", PREFIX, nb=nb, **sizes) for nb in (64, LARGE // hkv)) == named
