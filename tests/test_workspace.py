"""The binding's shared workspace: who keeps it, on host buffers (no GPU)."""
import contextlib
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
    streams = [None]                    # the current one and, innermost last, those entered
    filled = []                    # the stream of each zero fill

    @contextlib.contextmanager
    def stream(s):
        streams.append(s if s is not None else streams[-1])
        yield
        streams.pop()

    def fill(n, dtype, device):
        filled.append(streams[-1])
        return zeros(n, dtype=dtype)
    monkeypatch.setattr(_lib, "_ws", {})
    monkeypatch.setattr(_lib, "filled", filled, raising=False)
    monkeypatch.setattr(torch, "zeros", fill)
    monkeypatch.setattr(torch.cuda, "stream", stream)
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


def test_the_fill_is_on_the_calls_own_stream(lib):
    """Elsewhere it could come after the kernel."""
    calls = []

    def fn(ptr, nbytes, raw):
        calls.append(nbytes)
        return 0 if nbytes >= 1000 else lib.W4_ERR_WORKSPACE
    lib._call_with_workspace(fn, "fn", (), (7,), DEV, None, lambda: 1000, "side")
    assert lib.filled == ["side"] and calls[0] == 0 and calls[1] >= 1000
    lib._workspace(DEV, 2 * calls[1])
    assert lib.filled == ["side", None]
