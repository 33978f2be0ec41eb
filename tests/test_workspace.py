"""The binding's shared workspace: who keeps it, on host buffers (no GPU)."""
import weakref

import pytest
import torch

from helpers import ensure_built

DEV = torch.device("cuda", 0)


@pytest.fixture
def lib(monkeypatch):
    ensure_built()
    from int4_weight_only_gb300 import _lib
    zeros = torch.zeros
    monkeypatch.setattr(_lib, "_ws", {})
    monkeypatch.setattr(torch, "zeros", lambda n, dtype, device: zeros(n, dtype=dtype))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    return _lib


def test_an_outgrown_buffer_is_kept(lib):
    """A captured graph has its address."""
    first = lib._workspace(DEV, 1000)
    ref, n = weakref.ref(first), first.numel()
    del first
    second = lib._workspace(DEV, n + 1)
    assert second.numel() > n and ref() is not None
    assert lib._workspace(DEV, n) is second


def test_the_first_buffer_serves_attention(lib):
    """152 SMs x 2 parts x 16 heads x (128 + 2) floats behind the counters."""
    first = lib._workspace(DEV, 1000)
    assert lib._workspace(DEV, 65536 + 152 * 2 * 16 * 130 * 4) is first


def test_a_buffer_made_during_a_capture_is_not_shared(lib, monkeypatch):
    """Its zero fill has only been recorded, and its memory is the graph's."""
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    assert lib._workspace(DEV, 1000).numel() >= 1000 and not lib._ws
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    eager = lib._workspace(DEV, 1000)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    assert lib._workspace(DEV, 1000) is eager
    assert lib._workspace(DEV, eager.numel() + 1) is not eager and lib._workspace(DEV, 1000) is eager
