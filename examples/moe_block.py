"""A serving step of decoder blocks with routed experts, over a paged cache in which requests share a prompt.

    w4_kv_plan: pages, lengths, offsets of the step from the requests' lengths
    x -> qkv -> w4_rope_append -> w4_attn_shared (one token each) or w4_attn_prefill (prompts) -> o
      -> + residual, norm -> router -> w4_moe_route -> w4_moe_gather
      -> gate|up, SiLU, down of every expert (w4a16_grouped_linear) -> w4_moe_combine -> + residual, norm

Requests begin with the same prompt, which is run once; its whole pages are entered into every request's table.
Everything that changes from step to step (lengths, pages, groups) stays on the device, so that a decode step is
one captured graph.  Run as a script it serves a batch behind a long prompt at the expert sizes of workloads.py
(128 experts, 8 of them a token, hidden 2048, width 1024; random weights) and prints the times with and without
sharing:

    python examples/moe_block.py [--layers 2] [--batch 32] [--prompt 8192] [--steps 32]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import int4_weight_only_gb300 as w4  # noqa: E402
from examples.decoder_block import Linear, timed  # noqa: E402


class Config:
    def __init__(self, hidden=2048, q_heads=16, kv_heads=4, head_dim=128, experts=128, topk=8, width=1024, group=32,
                 expert_groups=8, top_groups=4, score="sigmoid", scale=2.5, base=1e6, page_size=64):
        self.hidden, self.q_heads, self.kv_heads, self.head_dim = hidden, q_heads, kv_heads, head_dim
        self.experts, self.topk, self.width, self.group = experts, topk, width, group
        self.expert_groups, self.top_groups, self.score, self.scale = expert_groups, top_groups, score, scale
        self.base, self.page_size = base, page_size


class Experts:
    """The experts' matrices, quantized and stacked, and the router before them."""

    def __init__(self, c, gen):
        self.c = c

        def W(n, k):
            return torch.randn(n, k, generator=gen, device="cuda") * 0.02
        self.gate_up = w4.w4_pack_rtn(W(c.experts * 2 * c.width, c.hidden), c.group, True)[:2]
        self.down = w4.w4_pack_rtn(W(c.experts * c.hidden, c.width), c.group, True)[:2]
        self.router = (torch.randn(c.experts, c.hidden, generator=gen, device="cuda") * 0.05).bfloat16()
        self.bias = torch.randn(c.experts, generator=gen, device="cuda") * 0.02

    def __call__(self, x):
        c = self.c
        w, _, row, goff = w4.w4_moe_route((x @ self.router.t()).float(), c.topk, bias=self.bias, score=c.score,
                                          groups=c.expert_groups, top_groups=c.top_groups, group_best=2, scale=c.scale)
        # few rows an expert: the decode kernel in tiles of 16; many: the tensor cores
        tile = 16 if row.numel() < 16 * c.experts else 256
        xs = w4.w4_moe_gather(x, row)
        g = w4.w4a16_grouped_linear(xs, goff, *self.gate_up, None, None, c.experts, 2 * c.width, c.hidden, c.group, tile)
        h = torch.nn.functional.silu(g[:, :c.width]) * g[:, c.width:]
        y = w4.w4a16_grouped_linear(h, goff, *self.down, None, None, c.experts, c.hidden, c.width, c.group, tile)
        return w4.w4_moe_combine(y, row, w)


class Layer:
    def __init__(self, c, gen):
        def W(n, k):
            return torch.randn(n, k, generator=gen, device="cuda") * 0.02
        self.qkv = Linear(W((c.q_heads + 2 * c.kv_heads) * c.head_dim, c.hidden), c.group)
        self.o = Linear(W(c.hidden, c.q_heads * c.head_dim), c.group)
        self.experts = Experts(c, gen)
        self.norm_in = (1 + 0.1 * torch.randn(c.hidden, generator=gen, device="cuda")).bfloat16()
        self.norm_mid = (1 + 0.1 * torch.randn(c.hidden, generator=gen, device="cuda")).bfloat16()


class Cache:
    """A page pool per layer, one table, and the free list, all on the device."""

    def __init__(self, c, layers, batch, max_len, pages):
        self.c, self.max_len, self.pages = c, max_len, pages
        shape = (pages, c.kv_heads, c.page_size, c.head_dim)
        self.k = [torch.empty(shape, dtype=torch.bfloat16, device="cuda") for _ in range(layers)]
        self.v = [torch.empty(shape, dtype=torch.bfloat16, device="cuda") for _ in range(layers)]
        i32 = dict(dtype=torch.int32, device="cuda")
        self.table = torch.zeros(batch, -(-max_len // c.page_size), **i32)
        self.lens = torch.zeros(batch, **i32)
        self.free = torch.arange(pages, **i32)
        self.used = torch.zeros(1, **i32)
        # one group over the whole batch until a prompt is shared
        self.group = torch.tensor([0, batch], **i32)
        self.shared = torch.zeros(1, **i32)

    def plan(self, new, T, rows=slice(None)):
        """The step's (kv_len, goff), with `new` tokens for the requests `rows` of the batch."""
        kv_len, goff, _, _ = w4.w4_kv_plan(self.lens[rows], new, self.free, self.used, self.table[rows], self.c.page_size,
                                           self.pages, T, lens_out=self.lens[rows], used_out=self.used)
        return kv_len, goff

    def share(self, n):
        """The first n tokens of request 0 become everybody's: whole pages by their numbers, the page in which they end
        by a copy of it.  (Pages are handed out so that each request's next one is its own.)"""
        c, whole = self.c, n // self.c.page_size
        batch = self.table.shape[0]
        self.table[1:, :whole] = self.table[0, :whole]
        self.lens[1:] = whole * c.page_size
        if n % c.page_size:
            left = torch.full((batch - 1,), n % c.page_size, dtype=torch.int32, device="cuda")
            self.plan(left, int(left.sum()), slice(1, None))
            for pool in self.k + self.v:
                pool[self.table[1:, whole].long()] = pool[self.table[0, whole].long()].clone()
        self.shared.fill_(n)


class Block:
    def __init__(self, c, layers=1, seed=0):
        gen = torch.Generator("cuda").manual_seed(seed)
        self.c = c
        self.layers = [Layer(c, gen) for _ in range(layers)]
        self.norm_out = torch.ones(c.hidden, dtype=torch.bfloat16, device="cuda")
        inv, self.mscale = w4.w4_rope_freqs(c.head_dim, c.base)
        self.inv_freq = inv.cuda()

    def forward(self, h, cache, kv_len, goff=None, max_q=1, rows=slice(None), shared=True):
        """h [T, hidden] bf16, the new tokens of the requests `rows`, already planned; goff None: one token each."""
        c, d, T = self.c, self.c.head_dim, h.shape[0]
        table = cache.table[rows]
        r, x = w4.w4_block_norm(None, h, self.layers[0].norm_in)
        for i, layer in enumerate(self.layers):
            k_cache, v_cache = cache.k[i], cache.v[i]
            q, k, v = layer.qkv(x).view(T, c.q_heads + 2 * c.kv_heads, d).split([c.q_heads, c.kv_heads, c.kv_heads], dim=1)
            q = w4.w4_rope_append(q, k, v, k_cache, v_cache, kv_len, table, self.inv_freq, goff=goff, mscale=self.mscale)
            if goff is not None:
                a = w4.w4_attn_prefill(q, k_cache, v_cache, goff, kv_len, table, max_q, cache.max_len)
            elif shared:
                a = w4.w4_attn_shared(q, k_cache, v_cache, kv_len, table, cache.group, cache.shared, cache.max_len)
            else:
                a = w4.w4_attn_decode(q, k_cache, v_cache, kv_len, table, cache.max_len)
            r, x = w4.w4_block_norm(layer.o(a.view(T, -1)), r, layer.norm_mid)
            after = self.layers[i + 1].norm_in if i + 1 < len(self.layers) else self.norm_out
            r, x = w4.w4_block_norm(layer.experts(x), r, after)
        return x


def prompt(block, cache, h, rows):
    """Runs h [T, hidden] as new tokens of one request (a slice of one row of the batch)."""
    T = h.shape[0]
    new = torch.tensor([T], dtype=torch.int32, device="cuda")
    kv_len, goff = cache.plan(new, T, rows)
    return block.forward(h, cache, kv_len, goff, T, rows)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--batch", type=int, default=32)
    ap.add_argument("--prompt", type=int, default=8192)
    ap.add_argument("--steps", type=int, default=32)
    args = ap.parse_args()
    c = Config()
    block = Block(c, args.layers)
    max_len = args.prompt + 2 * args.steps + 64
    cache = Cache(c, args.layers, args.batch, max_len, -(-args.prompt // c.page_size) + args.batch * 6)
    prompt(block, cache, torch.randn(args.prompt, c.hidden, device="cuda").bfloat16(), slice(0, 1))
    cache.share(args.prompt)
    x = torch.randn(args.batch, c.hidden, device="cuda").bfloat16()
    one = torch.ones(args.batch, dtype=torch.int32, device="cuda")
    for shared in (True, False):
        def step():
            kv_len, _ = cache.plan(one, args.batch)
            return block.forward(x, cache, kv_len, shared=shared)
        step()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = step()
        ms = timed(graph.replay, max(args.steps - 2, 1))
        print(f"decode: batch {args.batch} behind {args.prompt} tokens, {args.layers} layers, "
              f"{'shared' if shared else 'each its own'}: {ms * 1e3:.1f} us a step, finite: "
              f"{bool(torch.isfinite(out).all())}")
    if w4.w4_get_device_error():
        raise SystemExit("device error")


if __name__ == "__main__":
    main()
