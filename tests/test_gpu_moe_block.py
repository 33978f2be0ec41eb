"""The serving step of examples/moe_block.py: page plans, shared attention and routed experts together.

Attention with and without sharing differs by the rounding of the shared keys' weights to bf16 and of results
that are rounded from them; one block adds two residual branches of size about 1, each passing a handful of bf16
roundings (2^-8 each, independent), so hidden states of size 1 agree to 2^-8 * sqrt(12) in the root mean square,
as in the plain decoder block's test.  A router's choice may flip where two scores lie within such a difference:
rows where it did are left out, and are few."""
import os
import sys

import pytest
import torch

from helpers import ROOT, ensure_built

pytestmark = pytest.mark.gpu
sys.path.insert(0, ROOT)
sys.path.insert(0, os.path.join(ROOT, "examples"))
RMS = 2.0 ** -8 * 12 ** 0.5


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ensure_built()
    from examples import moe_block
    return moe_block


CONFIGS = [dict(hidden=256, q_heads=8, kv_heads=2, head_dim=64, experts=16, topk=4, width=128, expert_groups=4,
                top_groups=2, page_size=16),
           dict(hidden=384, q_heads=7, kv_heads=1, head_dim=128, experts=12, topk=2, width=64, expert_groups=1,
                top_groups=1, score="softmax", scale=1.0, page_size=32)]


def serve(ex, cfg, n, own, steps, shared, graph=False):
    """A prompt of n tokens run once, `own` more for each request, then decode steps; returns the steps' outputs."""
    c = ex.Config(**cfg)
    block = ex.Block(c, layers=1, seed=1)
    batch, max_len = len(own), n + max(own) + steps + 2
    cache = ex.Cache(c, 1, batch, max_len, batch * (max(own) + steps) // c.page_size + n // c.page_size + 3 * batch + 2)
    g = torch.Generator().manual_seed(n)

    def rand(t):
        return torch.randn(t, c.hidden, generator=g).bfloat16().cuda()
    ex.prompt(block, cache, rand(n), slice(0, 1))
    cache.share(n)
    for b, m in enumerate(own):
        if m:
            ex.prompt(block, cache, rand(m), slice(b, b + 1))
    x = torch.empty(batch, c.hidden, dtype=torch.bfloat16, device="cuda")
    active = torch.ones(batch, dtype=torch.int32, device="cuda")

    def step():
        kv_len, goff = cache.plan(active, batch)
        # without an offset each row of the batch is one token: rows of requests outside the step are unused
        return block.forward(x, cache, kv_len, shared=shared)
    outs, replay = [], None
    for i in range(steps):
        x.copy_(rand(batch))
        if graph and i == 0:
            keep = [t.clone() for t in (cache.lens, cache.used, cache.table, cache.k[0], cache.v[0])]
            step()
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            replay = torch.cuda.CUDAGraph()
            with torch.cuda.graph(replay, stream=side):
                out = step()
            for t, k in zip((cache.lens, cache.used, cache.table, cache.k[0], cache.v[0]), keep):
                t.copy_(k)
        if graph:
            replay.replay()
            outs.append(out.clone())
        else:
            outs.append(step())
    import int4_weight_only_gb300 as w4
    assert w4.w4_get_device_error() == 0
    assert cache.lens.tolist() == [n + m + steps for m in own]
    return torch.stack(outs)


@pytest.mark.parametrize("cfg", CONFIGS)
@pytest.mark.parametrize("n", [64, 150, 700])
def test_shared_and_unshared_steps_agree(ex, cfg, n):
    own = [0, 5, 33, 1, 0, 17]
    a = serve(ex, cfg, n, own, 20, True)
    b = serve(ex, cfg, n, own, 20, False)
    d = (a.float() - b.float()).square().mean(-1).sqrt()
    size = b.float().square().mean(-1).sqrt()
    same = d <= 4 * RMS * size                        # else another expert
    assert same.float().mean() > 0.9
    assert (d[same].square().mean().sqrt() <= RMS * size[same].square().mean().sqrt()).item()


@pytest.mark.parametrize("cfg", CONFIGS)
def test_captured_steps_are_the_eager_ones(ex, cfg):
    own = [3, 0, 14, 40]
    a = serve(ex, cfg, 100, own, 40, True)
    b = serve(ex, cfg, 100, own, 40, True, graph=True)
    assert torch.equal(a, b)


def test_script_runs(ex, monkeypatch, capsys):
    monkeypatch.setattr(sys, "argv", ["moe_block.py", "--layers", "1", "--batch", "5", "--prompt", "200", "--steps", "4"])
    ex.main()
    assert capsys.readouterr().out.count("finite: True") == 2
