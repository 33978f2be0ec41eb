"""Pages that hold no key that a token sees may be handed back: their table
entries, out of range here, are not looked at, in either form of attention."""
import numpy as np
import pytest
import torch

from block_helpers import Paged
from helpers import ensure_built
from oracle import block_oracle as BO
from test_gpu_attn import decode, prefill

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w4():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ensure_built()


def without_hidden_pages(qs, lens, heads, D, ps, window, sinks):
    cache = Paged(lens, heads, D, ps, seed=ps + window)
    kv = cache.fill_random()
    gone = 0
    for b, (n, m) in enumerate(zip(qs, lens)):
        seen = BO.visible(np.arange(m - n, m), m, window, sinks).any(0)
        for j in range(-(-m // ps)):
            if not seen[j * ps:(j + 1) * ps].any():
                cache.table_cpu[b, j] = -1
                gone += 1
    assert gone
    cache.table = cache.table_cpu.cuda()
    return cache, kv


RULES = [(16, 100, 0), (16, 100, 5), (32, 300, 4), (64, 129, 20), (16, 40, 200), (32, 700, 0), (16, 800, 9), (128, 90, 1)]


@pytest.mark.parametrize("ps,window,sinks", RULES)
@pytest.mark.parametrize("qs,lens", [([70], [2000]), ([3, 150], [1500, 1111]), ([1], [900]),
                                     ([40] * 90, [1000 + 13 * i for i in range(90)])])
def test_prefill(w4, qs, lens, ps, window, sinks):
    """A few items, whose steps the CTAs of a cluster share, and many, each on one CTA."""
    cache, kv = without_hidden_pages(qs, lens, 2, 64, ps, window, sinks)
    rows = None if len(qs) < 9 else [0, 1, 20, 39]
    prefill(w4, qs, lens, 4, 2, 64, ps, window, sinks, cache=cache, kv=kv, rows=rows)


@pytest.mark.parametrize("ps,window,sinks", RULES)
def test_decode(w4, ps, window, sinks):
    lens = [2000, 900, 517, 1800]
    cache, kv = without_hidden_pages([1] * 4, lens, 2, 64, ps, window, sinks)
    decode(w4, lens, 4, 2, 64, ps, window, sinks, cache=cache, kv=kv)
