"""Hidden values that are not finite have no influence, whatever else a CTA
works on and however many keys are cached."""
import numpy as np
import pytest
import torch

from block_helpers import Paged, randn_bf16, to64
from helpers import ensure_built
from oracle import block_oracle as BO
from test_gpu_attn import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w4():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ensure_built()


def poison(cache, kv, b, slots, bad, heads=slice(None)):
    k, v = kv[b]
    v = v.copy()
    v[slots, heads] = bad
    cache.put(b, torch.tensor(k).bfloat16(), torch.tensor(v).bfloat16())
    kv[b] = (k, v)


def compare(o, q, kv, off, qs, lens, b, rows, window=0, sinks=0):
    """Rows of sequence b: finite values within the bound, the others equal."""
    n, m, D = qs[b], lens[b], q.shape[2]
    at = np.array([r % n for r in rows])
    t = torch.as_tensor(at + int(off[b])).cuda()
    ref, _, mag = BO.attention(to64(q[t]), *kv[b], m - n + at, D ** -0.5, window, sinks)
    y, fin = to64(o[t]), np.isfinite(ref)
    assert np.array_equal(y[~fin], ref[~fin], equal_nan=True), f"sequence {b}"
    check(o[t], None, (ref, None, np.where(np.isfinite(mag), mag, 0)), f"sequence {b}")


def run(w4, cache, q, qs, lens, **kw):
    off = np.concatenate([[0], np.cumsum(qs)])
    o = w4.w4_attn_prefill(q, cache.k, cache.v, torch.tensor(off, dtype=torch.int32, device="cuda"), cache.kv_len,
                           cache.table, max(qs), max(lens), **kw)
    assert w4.w4_get_device_error() == 0
    return o, off


def test_long_prefix_in_a_batch(w4):
    """The last value behind a long prefix is hidden from all rows but the last: the items that
    share a CTA with it are computed, within a wait limit that is many times the call's time."""
    qs, lens, H, D = [60] + [36] * 149, [20000] + [40] * 149, 4, 128
    cache = Paged(lens, H, D, 64)
    kv = cache.fill_random()
    poison(cache, kv, 0, [19999], float("nan"))
    q = randn_bf16(sum(qs), 28, D, seed=1).cuda()
    w4.w4_set_wait_limit(20_000_000)
    try:
        o, off = run(w4, cache, q, qs, lens)
    finally:
        w4.w4_set_wait_limit(0)
    compare(o, q, kv, off, qs, lens, 0, [0, 30, -1])
    for b in range(1, 150):
        compare(o, q, kv, off, qs, lens, b, [0, 17, -1])


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("Hq,Hkv,D", [(28, 4, 128), (16, 16, 64), (17, 1, 64)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (90, 0), (200, 21)])
def test_slots_around_every_edge(w4, Hq, Hkv, D, window, sinks, bad):
    """Single values at the causal edge, the window's and the first tokens', each in one head and
    column; a few items and (the same sequences many times over) a list of them."""
    for copies in (1, 30):
        qs, lens = [70, 300, 9] * copies, [600, 300, 1000] * copies
        cache = Paged(lens, Hkv, D, 32, seed=Hq)
        kv = cache.fill_random()
        for b in (0, 1, 2):
            n, m = qs[b], lens[b]
            for i, j in enumerate((m - 1, m - 2, m - n, m - n // 2, max(m - max(window, 1), 0), max(m - n - window + 1, 0),
                                   20, 21, 0)):
                k, v = kv[b]
                v[j, i % Hkv, (7 * i) % D] = bad
            poison(cache, kv, b, [], 0)
        q = randn_bf16(sum(qs), Hq, D, seed=2).cuda()
        o, off = run(w4, cache, q, qs, lens, window=window, sinks=sinks)
        for b in (0, 1, 2, 3 * copies - 1):
            compare(o, q, kv, off, qs, lens, b, [0, 1, 4, 8, 34, 35, 36, 63, 64, 69, 149, 150, 299][: qs[b]], window, sinks)


def test_two_tile_and_one_tile_items_on_one_cta(w4):
    """Uneven sequences, so that CTAs go from items of two tiles to several of one; every other
    sequence ends in a value that is not finite.  The same bits at every call."""
    r = np.random.default_rng(5)
    qs = [int(x) for x in r.choice([1, 5, 18, 19, 36, 130, 700], 90)]
    lens = [n + int(x) for n, x in zip(qs, r.integers(0, 40, 90))]
    H, D = 4, 128
    cache = Paged(lens, H, D, 16)
    kv = cache.fill_random()
    for b in range(0, 90, 2):
        poison(cache, kv, b, [lens[b] - 1], float("nan"), b % H)
    q = randn_bf16(sum(qs), 28, D, seed=1).cuda()
    o, off = run(w4, cache, q, qs, lens)
    for b in range(0, 90, 5):
        compare(o, q, kv, off, qs, lens, b, [0, -1, qs[b] // 2])
    first = o.view(torch.int16).clone()
    for _ in range(20):
        assert torch.equal(run(w4, cache, q, qs, lens)[0].view(torch.int16), first)
