"""The binding's shared workspace under captured graphs and other streams."""
import pytest
import torch

import workloads as WL
from block_helpers import Paged, randn_bf16
from helpers import ensure_built

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


@pytest.fixture
def lib(monkeypatch):
    """The binding's module as it is before the process's first call."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ensure_built()
    from int4_weight_only_gb300 import _lib
    monkeypatch.setattr(_lib, "_ws", {})
    monkeypatch.setenv("W4_GEMV_SPLIT", "4")
    return _lib


def linear():
    """A linear whose K is split over CTAs, which meet in the workspace."""
    N, K, G = 3584, 18944, 128
    packed, scales, _ = WL.make_random_format(N, K, G, True, 3)
    args = (WL.make_activations(K, 1, 4).cuda(), packed.cuda(), scales.cuda(), None, None, N, K, G)
    return args, torch.empty(1, N, dtype=torch.bfloat16, device="cuda")


def attention(lens=(6000, 20)):
    cache = Paged(list(lens), 4, 128, 16)
    cache.fill_random()
    q = randn_bf16(len(lens), 28, 128, seed=1).cuda()
    return (q, cache.k, cache.v, cache.kv_len, cache.table, max(lens))


def test_a_graph_of_linears_outlives_the_first_attention_call(lib):
    args, y = linear()
    want = lib.w4a16_linear(*args).clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.w4a16_linear(*args, y=y)
    lib.w4_attn_decode(*attention())
    lib._workspace(DEV, 2 * lib._ws[0].numel())         # a call that needs more than the buffer has
    taken = [torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda") for n in (1 << 20, 4 << 20, 8 << 20) * 3]
    for _ in range(3):
        y.fill_(0)
        g.replay()
        assert torch.equal(y, want)
    assert all((t == 0xA5).all() for t in taken) and lib.w4_get_device_error() == 0


def test_a_first_call_inside_a_capture(lib):
    """The first calls without a workspace of their own are captured; eager calls after it, before
    the graph ever runs, find counters at zero."""
    args, y = linear()
    att = attention()
    out = torch.empty_like(att[0])
    own = torch.zeros(4 << 20, dtype=torch.uint8, device="cuda")
    lib.w4a16_linear(*args, workspace=own)
    lib.w4_attn_decode(*att, workspace=own)
    assert not lib._ws
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.w4a16_linear(*args, y=y)
        lib.w4_attn_decode(*att, out=out)
    torch.cuda.synchronize()
    want, want_o = lib.w4a16_linear(*args).clone(), lib.w4_attn_decode(*att).clone()
    for _ in range(3):
        y.fill_(0)
        out.fill_(0)
        g.replay()
        assert torch.equal(y, want) and torch.equal(out, want_o)
    assert torch.equal(lib.w4a16_linear(*args), want) and torch.equal(lib.w4_attn_decode(*att), want_o)
    assert lib.w4_get_device_error() == 0


def test_a_first_call_on_another_stream(lib):
    """The current stream is busy: the first call on another one does not wait for it, and
    its counters are cleared all the same."""
    args, y = linear()
    att = attention()
    own = torch.zeros(4 << 20, dtype=torch.uint8, device="cuda")
    want, want_o = lib.w4a16_linear(*args, workspace=own).clone(), lib.w4_attn_decode(*att, workspace=own).clone()
    side = torch.cuda.Stream()
    for first in ("linear", "attention"):
        lib._ws.clear()
        y.fill_(0)
        out = torch.zeros_like(want_o)
        torch.cuda.synchronize()
        done = torch.cuda.Event()
        torch.cuda._sleep(200_000_000)
        done.record()
        if first == "linear":
            lib.w4a16_linear(*args, y=y, stream=side)
        lib.w4_attn_decode(*att, out=out, stream=side)
        side.synchronize()
        assert not done.query()
        assert torch.equal(out, want_o) and (first != "linear" or torch.equal(y, want))
        torch.cuda.synchronize()
        assert not lib._ws[0][:65536].any()
