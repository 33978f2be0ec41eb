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


def test_scores_of_minus_infinity(w4):
    """They weigh nothing; a token that sees no other score gets zeros, as one that sees no key."""
    n, D = 300, 64
    cache = Paged([n, n], 1, D, 16)
    kv = cache.fill_random()
    for b, hidden in ((0, slice(0, 290)), (1, slice(0, n))):
        k, v = kv[b]
        k[hidden, :, 0] = -INF
        cache.put(b, torch.tensor(k).bfloat16(), torch.tensor(v).bfloat16())
    q = randn_bf16(80, 4, D, seed=1).abs().cuda()
    off = torch.tensor([0, 40, 80], dtype=torch.int32, device="cuda")
    lse = torch.zeros(80, 4, device="cuda")
    o = w4.w4_attn_prefill(q, cache.k, cache.v, off, cache.kv_len, cache.table, 40, n, lse=lse)
    lse1 = torch.zeros(2, 4, device="cuda")
    o1 = w4.w4_attn_decode(q[[39, 79]], cache.k, cache.v, cache.kv_len, cache.table, n, lse=lse1)
    assert w4.w4_get_device_error() == 0
    for y, z in ((o[:30], lse[:30]), (o[40:], lse[40:]), (o1[1:], lse1[1:])):
        assert not y.any() and (z == -INF).all()
    k, v = kv[0][0][290:], kv[0][1][290:]
    check(o[30:40], lse[30:40], BO.attention(to64(q[30:40]), k, v, np.arange(10), D ** -0.5), "prompt")
    check(o1[:1], lse1[:1], BO.attention(to64(q[39:40]), k, v, [9], D ** -0.5), "one token")
