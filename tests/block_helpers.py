"""Paged caches and comparisons for the decoder-block tests."""
import numpy as np
import torch

U = 2.0 ** -8                 # half a unit in the last place of bf16 (8 significant bits), relative


def to64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def within(y, ref, bound, what=""):
    """|y - ref| <= bound elementwise; NaN and infinities must agree."""
    y = to64(y) if isinstance(y, torch.Tensor) else y
    assert y.shape == ref.shape, (what, y.shape, ref.shape)
    fin = np.isfinite(ref)
    assert np.array_equal(np.isfinite(y), fin), f"{what}: non-finite values differ"
    over = np.abs(y - np.where(fin, ref, 0))[fin] - np.broadcast_to(bound, ref.shape)[fin]
    assert over.size == 0 or over.max() <= 0, f"{what}: {over.max():.3e} over the bound ({(over > 0).sum()} values)"


class Paged:
    """A pool filled with `fill` (NaN), pages handed out in a shuffled order.

    layout: "hnd" [pages, heads, slots, D], "nhd" [pages, slots, heads, D],
    "mixed" keys and values interleaved in one buffer with unused columns."""

    def __init__(self, lens, heads, D, page_size, layout="hnd", seed=0, fill=float("nan"), extra_cols=2,
                 device="cuda"):
        self.lens, self.heads, self.D, self.ps = list(lens), heads, D, page_size
        self.g = torch.Generator().manual_seed(seed)
        cols = max([-(-n // page_size) for n in lens] + [1]) + extra_cols
        need = sum(-(-n // page_size) for n in lens)
        pages = need + 3
        order = torch.randperm(pages, generator=self.g).tolist()
        # entries past a sequence's pages are out of range: they must not be read
        self.table_cpu = torch.full((len(lens), cols), 1 << 30, dtype=torch.int32)
        for b, n in enumerate(lens):
            for j in range(-(-n // page_size)):
                self.table_cpu[b, j] = order.pop()
        kw = dict(dtype=torch.bfloat16, device=device)
        if layout == "hnd":
            self.k = torch.full((pages, heads, page_size, D), fill, **kw)
            self.v = torch.full_like(self.k, fill)
        elif layout == "nhd":
            self.k = torch.full((pages, page_size, heads, D), fill, **kw).transpose(1, 2)
            self.v = torch.full((pages, page_size, heads, D), fill, **kw).transpose(1, 2)
        else:
            both = torch.full((pages, page_size, heads, 2, D + 8), fill, **kw)
            self.k = both[..., 0, :D].transpose(1, 2)
            self.v = both[..., 1, :D].transpose(1, 2)
        self.table = self.table_cpu.to(device)
        self.kv_len = torch.tensor(lens, dtype=torch.int32, device=device)

    def cells(self, b, n=None):
        j = torch.arange(self.lens[b] if n is None else n)
        return self.table_cpu[b].long()[j // self.ps], j % self.ps

    def put(self, b, k, v):
        """Write keys and values [n, heads, D] (CPU) as the sequence's first n."""
        pg, sl = self.cells(b, k.shape[0])
        dev = self.k.device
        self.k[pg.to(dev), :, sl.to(dev)] = k.to(dev, torch.bfloat16)
        self.v[pg.to(dev), :, sl.to(dev)] = v.to(dev, torch.bfloat16)

    def get(self, b, pool):
        pg, sl = self.cells(b)
        dev = self.k.device
        return pool[pg.to(dev), :, sl.to(dev)]

    def fill_random(self, scale=1.0):
        """Random keys and values for every sequence; returns them in float64."""
        out = []
        for b, n in enumerate(self.lens):
            k = (torch.randn(n, self.heads, self.D, generator=self.g) * scale).bfloat16()
            v = torch.randn(n, self.heads, self.D, generator=self.g).bfloat16()
            self.put(b, k, v)
            out.append((to64(k), to64(v)))
        return out


def randn_bf16(*shape, seed, scale=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale).bfloat16()
