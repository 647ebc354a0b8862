"""Which memory the binding's own workspaces take (CPU, against a stand-in for torch's device calls)."""

import contextlib

import pytest
import torch

from paged_kv_cache_217_gb300 import binding as B


@pytest.fixture
def devices(monkeypatch):
    """Two devices, 0 the current one, whose streams have handles 10 and 11; `capturing` holds those under capture."""
    now, capturing, made = [0], set(), []

    @contextlib.contextmanager
    def device(d):
        before, now[0] = now[0], d.index
        yield
        now[0] = before

    def empty(n, dtype, device):
        made.append((now[0], device.index))
        return torch.zeros(n, dtype=dtype)
    monkeypatch.setattr(B, "_handles", (lambda: now[0], lambda index: 10 + index))
    monkeypatch.setattr(B, "_scratches", {})
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: now[0] in capturing)
    monkeypatch.setattr(torch, "empty", empty)
    return capturing, made


def test_eager_calls_of_a_stream_share_a_workspace_that_grows(devices):
    first, second = B._scratch(torch.device("cuda", 0), 100), B._scratch(torch.device("cuda", 0), 1000)
    assert first is second and first.numel() >= 1000
    more = B._scratch(torch.device("cuda", 0), first.numel() + 1)
    assert more is not first and B._scratch(torch.device("cuda", 0), 1) is more
    assert B._scratch(torch.device("cuda", 1), 1) is not more
    assert B._scratch(torch.device("cuda", 0), 0) is None


@pytest.mark.parametrize("index", [0, 1])
def test_a_captured_call_has_memory_of_its_own_on_any_device(devices, index):
    capturing, made = devices
    eager = [B._scratch(torch.device("cuda", i), 64) for i in range(2)]
    capturing.add(index)                          # (the other device's stream, current or not, is not)
    a, b = (B._scratch(torch.device("cuda", index), 64) for _ in range(2))
    assert a is not b and a is not eager[index] and a.numel() == 64
    assert made[-1] == (index, index)             # made while its device is the current one
    assert B._scratch(torch.device("cuda", 1 - index), 64) is eager[1 - index]
