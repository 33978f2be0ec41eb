"""A decoder block on libw4: INT4 linears with the operators between them.

    x -> qkv (w4a16_linear) -> rotary + cache write (w4_rope_append)
      -> attention (w4_attn_prefill for prompts, w4_attn_decode for one token)
      -> o (w4a16_linear) -> + residual, norm (w4_block_norm)
      -> gate|up + SiLU (w4a16_linear_swiglu, or w4a16_linear for many tokens)
      -> down (w4a16_linear) -> + residual, the next block's norm (w4_block_norm)

Run as a script it prefills a ragged batch of prompts at the 7B sizes of
workloads.py (hidden 3584, 28 query and 4 key-value heads of 128, feed-forward
18944; random weights), decodes some tokens through a captured CUDA graph and
prints the times:

    python examples/decoder_block.py [--layers 2] [--batch 8] [--prompt 512] [--steps 32]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import int4_weight_only_gb300 as w4  # noqa: E402


class Config:
    def __init__(self, hidden=3584, q_heads=28, kv_heads=4, head_dim=128, ffn=18944, group=128, base=1e6,
                 page_size=64, window=0, sinks=0, rope="plain", factor=1.0, orig_len=32768):
        self.hidden, self.q_heads, self.kv_heads, self.head_dim, self.ffn = hidden, q_heads, kv_heads, head_dim, ffn
        self.group, self.base, self.page_size = group, base, page_size
        self.window, self.sinks = window, sinks
        self.rope, self.factor, self.orig_len = rope, factor, orig_len


class Linear:
    """One quantized layer."""

    def __init__(self, W, group):
        self.N, self.K, self.group = W.shape[0], W.shape[1], group
        self.packed, self.scales, _ = w4.w4_pack_rtn(W.contiguous(), group, True)

    def __call__(self, x):
        return w4.w4a16_linear(x, self.packed, self.scales, None, None, self.N, self.K, self.group)


class Layer:
    def __init__(self, c, gen):
        def W(n, k):
            return torch.randn(n, k, generator=gen, device="cuda") * 0.02
        d = c.head_dim
        self.qkv = Linear(W((c.q_heads + 2 * c.kv_heads) * d, c.hidden), c.group)
        self.o = Linear(W(c.hidden, c.q_heads * d), c.group)
        gate, up = W(c.ffn, c.hidden), W(c.ffn, c.hidden)
        self.gate_up = Linear(w4.pair_gate_up(gate, up), c.group)
        self.gate, self.up = Linear(gate, c.group), Linear(up, c.group)
        self.down = Linear(W(c.hidden, c.ffn), c.group)
        self.norm_in = (1 + 0.1 * torch.randn(c.hidden, generator=gen, device="cuda")).bfloat16()
        self.norm_mid = (1 + 0.1 * torch.randn(c.hidden, generator=gen, device="cuda")).bfloat16()


class Cache:
    """A page pool per layer, one page table for all of them.  Pages are handed
    out in order; a server would keep a free list."""

    def __init__(self, c, layers, batch, max_len):
        cols = -(-max_len // c.page_size)
        self.max_len = max_len
        shape = (batch * cols, c.kv_heads, c.page_size, c.head_dim)
        self.k = [torch.empty(shape, dtype=torch.bfloat16, device="cuda") for _ in range(layers)]
        self.v = [torch.empty(shape, dtype=torch.bfloat16, device="cuda") for _ in range(layers)]
        self.table = torch.arange(batch * cols, dtype=torch.int32, device="cuda").view(batch, cols)
        self.kv_len = torch.zeros(batch, dtype=torch.int32, device="cuda")


class Block:
    def __init__(self, c, layers=1, seed=0):
        gen = torch.Generator("cuda").manual_seed(seed)
        self.c = c
        self.layers = [Layer(c, gen) for _ in range(layers)]
        self.norm_out = torch.ones(c.hidden, dtype=torch.bfloat16, device="cuda")
        inv, self.mscale = w4.w4_rope_freqs(c.head_dim, c.base, c.rope, c.factor, c.orig_len)
        self.inv_freq = inv.cuda()

    def forward(self, h, cache, goff=None, max_q=1):
        """h [T, hidden] bf16, the new tokens of every sequence (kv_len already
        counts them); goff None: one token a sequence.  Returns the final norm."""
        c, d = self.c, self.c.head_dim
        T = h.shape[0]
        r, x = w4.w4_block_norm(None, h, self.layers[0].norm_in)
        for i, layer in enumerate(self.layers):
            qkv = layer.qkv(x).view(T, c.q_heads + 2 * c.kv_heads, d)
            q, k, v = qkv.split([c.q_heads, c.kv_heads, c.kv_heads], dim=1)
            q = w4.w4_rope_append(q, k, v, cache.k[i], cache.v[i], cache.kv_len, cache.table, self.inv_freq,
                                  goff=goff, mscale=self.mscale)
            if goff is None:
                a = w4.w4_attn_decode(q, cache.k[i], cache.v[i], cache.kv_len, cache.table, cache.max_len,
                                      window=c.window, sinks=c.sinks)
            else:
                a = w4.w4_attn_prefill(q, cache.k[i], cache.v[i], goff, cache.kv_len, cache.table, max_q,
                                       cache.max_len, window=c.window, sinks=c.sinks)
            r, x = w4.w4_block_norm(layer.o(a.view(T, -1)), r, layer.norm_mid)
            if T <= 16:
                g = layer.gate_up
                f = w4.w4a16_linear_swiglu(x, g.packed, g.scales, None, None, c.ffn, c.hidden, c.group)
            else:
                f = torch.nn.functional.silu(layer.gate(x)) * layer.up(x)
            after = self.layers[i + 1].norm_in if i + 1 < len(self.layers) else self.norm_out
            r, x = w4.w4_block_norm(layer.down(f), r, after)
        return x


def timed(fn, n):
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(n):
        fn()
    b.record()
    b.synchronize()
    return a.elapsed_time(b) / n


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--batch", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=512)
    ap.add_argument("--steps", type=int, default=32)
    args = ap.parse_args()
    c = Config()
    block = Block(c, args.layers)
    cache = Cache(c, args.layers, args.batch, args.prompt + args.steps + 1)
    lens = [max(1, args.prompt - 37 * b) for b in range(args.batch)]
    goff = torch.tensor([0] + lens, dtype=torch.int32).cumsum(0).int().cuda()
    cache.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
    h = torch.randn(sum(lens), c.hidden, device="cuda").bfloat16()
    block.forward(h, cache, goff, max(lens))
    ms = timed(lambda: block.forward(h, cache, goff, max(lens)), 5)
    print(f"prefill: {sum(lens)} tokens, {args.layers} layers: {ms:.3f} ms")
    x = torch.randn(args.batch, c.hidden, device="cuda").bfloat16()

    def step():
        cache.kv_len.add_(1)
        return block.forward(x, cache)
    step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = step()
    ms = timed(graph.replay, max(args.steps - 2, 1))
    if w4.w4_get_device_error():
        raise SystemExit("device error")
    print(f"decode: batch {args.batch}, {args.layers} layers: {ms * 1e3:.1f} us a step, finite: "
          f"{bool(torch.isfinite(out).all())}")


if __name__ == "__main__":
    main()
