"""The decoder block of examples/decoder_block.py: prompts, chunks and single
tokens through all operators together.

The same tokens must give the same hidden states however they are fed (whole
prompts, chunks behind a cached prefix, one token at a time, a captured graph):
the paths differ only in bf16 roundings of intermediate results.  One block adds
two residual branches of size about 1; each passes six bf16 roundings (2^-8 each,
independent) on its way, so outputs of size 1 agree to 2^-8 * sqrt(12) in the
root mean square and to 6 times that at worst over a few thousand values."""
import os
import sys

import pytest
import torch

from helpers import ROOT, ensure_built

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(ROOT, "examples"))

RMS = 2.0 ** -8 * 12 ** 0.5


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ensure_built()
    import decoder_block
    return decoder_block


def agree(a, b):
    d = (a.float() - b.float())
    size = b.float().square().mean().sqrt().item()
    assert d.square().mean().sqrt().item() <= RMS * size
    assert d.abs().max().item() <= 6 * RMS * max(size, b.float().abs().max().item())


CONFIGS = [dict(hidden=256, q_heads=4, kv_heads=2, head_dim=64, ffn=512, page_size=16),
           dict(hidden=384, q_heads=7, kv_heads=1, head_dim=128, ffn=256, page_size=32, window=40, sinks=3,
                rope="yarn", factor=4.0, orig_len=64)]


@pytest.mark.parametrize("cfg", CONFIGS)
def test_one_token_at_a_time_matches_the_prompt(ex, cfg):
    c = ex.Config(**cfg)
    block = ex.Block(c, layers=1, seed=1)
    lens = [70, 33, 1]
    h = [torch.randn(n, c.hidden, generator=torch.Generator().manual_seed(n)).bfloat16().cuda() for n in lens]
    goff = torch.tensor([0, 70, 103, 104], dtype=torch.int32, device="cuda")
    whole = ex.Cache(c, 1, 3, 80)
    whole.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
    want = block.forward(torch.cat(h), whole, goff, 70)
    # token by token; a sequence that has ended is an unused row of the batch
    single = ex.Cache(c, 1, 3, 80)
    for t in range(70):
        single.kv_len.copy_(torch.tensor([t + 1 if t < n else 0 for n in lens], dtype=torch.int32))
        x = torch.stack([s[t] if t < len(s) else s[0] for s in h])
        out = block.forward(x, single)
        for b, n in enumerate(lens):
            if t == n - 1 or t in (0, 17, 41) and t < n:
                row = int(goff[b]) + t
                agree(out[b:b + 1], want[row:row + 1])
    # a chunk of 37 behind the first 33
    chunk = ex.Cache(c, 1, 1, 80)
    for lo, hi in ((0, 33), (33, 70)):
        chunk.kv_len.fill_(hi)
        got = block.forward(h[0][lo:hi].contiguous(), chunk, torch.tensor([0, hi - lo], dtype=torch.int32,
                                                                         device="cuda"), hi - lo)
        agree(got, want[lo:hi])
    from int4_weight_only_gb300 import w4_get_device_error
    assert w4_get_device_error() == 0


def test_captured_step(ex):
    """A captured decode step replays with growing lengths as the eager one."""
    c = ex.Config(**CONFIGS[0])
    block = ex.Block(c, layers=2, seed=2)
    x = torch.randn(5, c.hidden, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    eager, graph = ex.Cache(c, 2, 5, 40), ex.Cache(c, 2, 5, 40)

    def step(cache):
        cache.kv_len.add_(1)
        return block.forward(x, cache)
    want = [step(eager).clone() for _ in range(35)]
    step(graph)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        out = step(graph)
    for t in range(1, 35):
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[t]), t
