"""Infinities among the values that a token sees: o = sum_j w_j v_j with w_j > 0
is the infinity (infinities of both signs: NaN), in both forms of attention and
wherever a sequence is cut."""
import numpy as np
import pytest
import torch

from block_helpers import Paged, randn_bf16, to64
from helpers import ensure_built
from oracle import block_oracle as BO
from test_gpu_attn import check

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(scope="module")
def w4():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ensure_built()


def same(o, want, what):
    """The finite values within the attention bound, the others equal."""
    ref, _, mag = want
    y, fin = to64(o), np.isfinite(ref)
    assert np.array_equal(y[~fin], ref[~fin], equal_nan=True), what
    check(o, None, (ref, None, np.where(np.isfinite(mag), mag, 0)), what)


def poisoned(lens, heads, D, where, seed=0):
    """A cache of random keys and values with `where` (slot from the end: value)
    in column 3 of every head; the keys that have such a value get close scores."""
    cache = Paged(lens, heads, D, 16, seed=seed)
    kv = []
    for b, (k, v) in enumerate(cache.fill_random()):
        for back, x in where.items():
            if back <= len(v):
                v[len(v) - back, :, 3] = x
        cache.put(b, torch.tensor(k).bfloat16(), torch.tensor(v).bfloat16())
        kv.append((k, v))
    return cache, kv


WHERE = [{1: INF}, {1: -INF}, {1: INF, 2: INF}, {1: INF, 2: -INF}, {40: INF}, {40: -INF, 90: -INF}, {7: INF, 60: -INF}]


@pytest.mark.parametrize("where", WHERE)
@pytest.mark.parametrize("Hq,Hkv,D", [(28, 4, 128), (6, 2, 64), (17, 1, 128), (40, 1, 64)])
def test_decode(w4, Hq, Hkv, D, where):
    """One key (its weight is exactly 1), short sequences, and one that many CTAs share."""
    lens = [1, 2, 50, 100, 3000]
    cache, kv = poisoned(lens, Hkv, D, where, Hq)
    q = randn_bf16(len(lens), Hq, D, seed=1).cuda()
    o = w4.w4_attn_decode(q, cache.k, cache.v, cache.kv_len, cache.table, max(lens))
    assert w4.w4_get_device_error() == 0
    for b, n in enumerate(lens):
        same(o[b:b + 1], BO.attention(to64(q[b:b + 1]), *kv[b], [n - 1], D ** -0.5), f"{where} length {n}")


@pytest.mark.parametrize("where", WHERE)
@pytest.mark.parametrize("Hq,Hkv,D", [(28, 4, 128), (6, 2, 64), (40, 1, 64)])
def test_prefill(w4, Hq, Hkv, D, where):
    qs, lens = [1, 50, 100, 70], [1, 50, 120, 700]
    cache, kv = poisoned(lens, Hkv, D, where, Hq)
    q = randn_bf16(sum(qs), Hq, D, seed=1).cuda()
    off = np.concatenate([[0], np.cumsum(qs)])
    o = w4.w4_attn_prefill(q, cache.k, cache.v, torch.tensor(off, dtype=torch.int32, device="cuda"), cache.kv_len,
                           cache.table, max(qs), max(lens))
    assert w4.w4_get_device_error() == 0
    for b, (n, m) in enumerate(zip(qs, lens)):
        t = slice(int(off[b]), int(off[b + 1]))
        same(o[t], BO.attention(to64(q[t]), *kv[b], m - n + np.arange(n), D ** -0.5), f"{where} {n} of {m}")
