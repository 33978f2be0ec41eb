"""GPU parity of w4_attn_decode and w4_attn_prefill against the float64 oracle.

Bound of an output value, from w = softmax weights, A = sum_j w_j |v_j|:
one bf16 rounding of the result (2^-8 |o|), the weights' rounding to bf16 as
matrix operands (2^-8 A), and the fp32 scores: |q . k| sums to at most a few
hundred in D <= 128 terms, so a score is off by at most 2^-12 (log units) and
A by twice that (2^-11 A).  The log-sum-exp is off by the score error, 2^-12,
plus 2^-20 of its size."""
import numpy as np
import pytest
import torch

from block_helpers import Paged, U, randn_bf16, to64, within
from helpers import check_band, ensure_built, guarded_empty
from oracle import block_oracle as BO

pytestmark = pytest.mark.gpu

PAGE_ERR, ROWS_ERR = -13, -11


@pytest.fixture(scope="module")
def w4():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ensure_built()


def check(o, lse, want, what):
    ref, wl, mag = want
    within(o, ref, U * np.abs(ref) + (U + 2.0 ** -11) * mag, what)
    if lse is not None:
        wl32 = np.abs(np.where(np.isfinite(wl), wl, 0))
        within(lse.cpu().numpy().astype(np.float64), wl, 2.0 ** -12 + 2.0 ** -20 * wl32, what + " lse")


def decode(w4, lens, Hq, Hkv, D, ps=16, window=0, sinks=0, layout="hnd", scale=None, seed=0, k_scale=1.0, kv=None,
           cache=None, max_len=None, workspace=None):
    if cache is None:
        cache = Paged(lens, Hkv, D, ps, layout, seed)
        kv = cache.fill_random(k_scale)
    B = len(lens)
    ld = Hq * D + 24
    q = torch.zeros(B, ld, dtype=torch.bfloat16)
    q[:, 8:8 + Hq * D] = randn_bf16(B, Hq * D, seed=seed + 9)
    qd = q.cuda()[:, 8:8 + Hq * D].unflatten(1, (Hq, D))
    out, raw = guarded_empty((B, Hq, D), torch.bfloat16)
    lse, raw2 = guarded_empty((B, Hq), torch.float32)
    sc = D ** -0.5 if scale is None else scale
    w4.w4_attn_decode(qd, cache.k, cache.v, cache.kv_len, cache.table, max(lens) if max_len is None else max_len, sc,
                      window, sinks, out=out, lse=lse, workspace=workspace)
    check_band(raw, "out")
    check_band(raw2, "lse")
    assert w4.w4_get_device_error() == 0
    for b, n in enumerate(lens):
        want = BO.attention(to64(qd[b:b + 1]), *kv[b], [n - 1], sc, window, sinks)
        check(out[b:b + 1], lse[b:b + 1], want, f"decode {Hq}/{Hkv}x{D} page {ps} length {n} window {window}+{sinks}")
    return out


def prefill(w4, qs, lens, Hq, Hkv, D, ps=16, window=0, sinks=0, layout="hnd", scale=None, seed=0, k_scale=1.0,
            lead=0, pad=0, cache=None, kv=None, max_q=None, max_len=None, rows=None):
    """rows: the row numbers inside each sequence that are compared (None: all)."""
    if cache is None:
        cache = Paged(lens, Hkv, D, ps, layout, seed)
        kv = cache.fill_random(k_scale)
    T = lead + sum(qs) + pad
    q = torch.zeros(T, Hq * D + 24, dtype=torch.bfloat16)
    q[:, 8:8 + Hq * D] = randn_bf16(T, Hq * D, seed=seed + 9)
    qd = q.cuda()[:, 8:8 + Hq * D].unflatten(1, (Hq, D))
    off = np.concatenate([[0], np.cumsum(qs)]) + lead
    out, raw = guarded_empty((T, Hq, D), torch.bfloat16)
    lse, raw2 = guarded_empty((T, Hq), torch.float32)
    out.fill_(-3.0)
    lse.fill_(-3.0)
    sc = D ** -0.5 if scale is None else scale
    w4.w4_attn_prefill(qd, cache.k, cache.v, torch.tensor(off, dtype=torch.int32, device="cuda"), cache.kv_len,
                       cache.table, max(qs) if max_q is None else max_q, max(lens) if max_len is None else max_len, sc,
                       window, sinks, out=out, lse=lse)
    check_band(raw, "out")
    check_band(raw2, "lse")
    assert w4.w4_get_device_error() == 0
    assert (out[:lead] == -3.0).all() and (out[T - pad:] == -3.0).all()
    assert (lse[:lead] == -3.0).all() and (lse[T - pad:] == -3.0).all()
    for b, (n, m) in enumerate(zip(qs, lens)):
        at = np.arange(n) if rows is None else np.array([r for r in rows if r < n], int)
        t = torch.as_tensor(at + off[b])
        want = BO.attention(to64(qd[t.cuda()]), *kv[b], m - n + at, sc, window, sinks)
        check(out[t.cuda()], lse[t.cuda()], want, f"prefill {Hq}/{Hkv}x{D} page {ps} rows {n} length {m} {window}+{sinks}")
    return out


HEADS = [(28, 4, 128), (4, 4, 64), (8, 1, 128), (16, 1, 64), (9, 3, 64), (17, 1, 128), (40, 1, 64), (5, 5, 128)]
LENS = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200]


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
def test_decode_heads_and_lengths(w4, Hq, Hkv, D):
    decode(w4, LENS, Hq, Hkv, D, seed=Hq)


@pytest.mark.parametrize("layout", ["hnd", "nhd", "mixed"])
@pytest.mark.parametrize("ps", [16, 32, 128, 4096])
def test_decode_pools(w4, layout, ps):
    decode(w4, [1, 130, 300, 77], 6, 2, 64, ps, layout=layout)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 0), (17, 5), (64, 16), (100, 100), (1000, 3), (33, 40),
                                          (0, 7), (30, 1000)])
def test_decode_window(w4, window, sinks):
    decode(w4, [1, 20, 33, 64, 129, 300, 517], 4, 2, 64, window=window, sinks=sinks, seed=window)


def test_decode_unused_rows(w4):
    """Length 0: zero output, -inf log-sum-exp; also a whole unused batch."""
    out = decode(w4, [5, 0, 0, 40, 0], 7, 1, 128)
    assert not out[1].any()
    decode(w4, [0, 0], 4, 4, 64)


@pytest.mark.parametrize("lens", [[40000], [3, 20000, 1, 9000], [2500] * 3, list(range(0, 700, 3))])
def test_decode_splits(w4, lens):
    """Long sequences are cut over many CTAs, many short ones share CTAs; the
    bits do not change from call to call."""
    cache = Paged(lens, 2, 64, 64, seed=3)
    kv = cache.fill_random()
    a = decode(w4, lens, 6, 2, 64, 64, cache=cache, kv=kv)
    b = decode(w4, lens, 6, 2, 64, 64, cache=cache, kv=kv)
    assert torch.equal(a, b)


def test_decode_more_sequences_than_threads(w4):
    lens = [(37 * i) % 90 for i in range(300)]
    decode(w4, lens, 3, 1, 64, seed=4)


def test_workspace_is_left_ready(w4):
    """The caller's workspace: counters back at zero, any call order."""
    n = w4.w4_attn_decode_workspace_bytes(8, 2, 128)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    for lens in ([5000, 3], [4000, 4999, 1, 77], [64]):
        decode(w4, lens, 8, 2, 128, 32, workspace=ws)
        assert not ws[:65536].any()
    with pytest.raises(w4.W4Error):
        decode(w4, [64], 8, 2, 128, 32, workspace=ws[:65536])


def test_decode_sharp_and_flat_scores(w4):
    """One key dominates (others underflow), all scores equal, large scores."""
    decode(w4, [300, 50], 4, 2, 64, scale=4.0, k_scale=3.0)
    cache = Paged([200], 1, 64, 16)
    k = torch.zeros(200, 1, 64).bfloat16()
    v = randn_bf16(200, 1, 64, seed=2)
    cache.put(0, k, v)
    decode(w4, [200], 4, 1, 64, cache=cache, kv=[(to64(k), to64(v))])


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_decode_hidden_keys_have_no_influence(w4, bad):
    cache = Paged([300], 2, 64, 16)
    kv = cache.fill_random()
    k, v = (torch.tensor(x).bfloat16() for x in kv[0])
    k[20:180], v[20:180] = bad, bad
    cache.put(0, k, v)
    decode(w4, [300], 4, 2, 64, window=120, sinks=20, cache=cache, kv=[(to64(k), to64(v))])


def test_decode_visible_nan(w4):
    """A visible NaN reaches the heads that see it and no other."""
    cache = Paged([100, 100], 2, 64, 16)
    kv = cache.fill_random()
    v = torch.tensor(kv[0][1]).bfloat16()
    v[50, 1, 3] = float("nan")
    cache.put(0, torch.tensor(kv[0][0]).bfloat16(), v)
    q = randn_bf16(2, 4, 64, seed=1).cuda()
    o = w4.w4_attn_decode(q, cache.k, cache.v, cache.kv_len, cache.table, 100)
    bad = torch.isnan(o)
    assert bad[0, 2:, 3].all() and bad.sum() == 2


def test_decode_bad_device_data(w4):
    q = randn_bf16(2, 4, 64, seed=1).cuda()

    def call(c, max_len=64):
        o = w4.w4_attn_decode(q, c.k, c.v, c.kv_len, c.table, max_len)
        return o, w4.w4_get_device_error()
    c = Paged([40, 50], 2, 64, 16, fill=1.0)
    kv = c.fill_random()
    good, rc = call(c)
    assert rc == 0
    for bad in (-1, c.k.shape[0], -(1 << 31)):
        c.table[1, 2] = bad
        o, rc = call(c)
        assert rc == PAGE_ERR and torch.equal(o[0], good[0])
    c = Paged([40, 50], 2, 64, 16, fill=1.0)
    for n, lim in ((-1, 64), (49, 48), (1 << 30, 1 << 30)):
        c.kv_len[1] = n
        o, rc = call(c, lim)
        assert rc == PAGE_ERR
    assert len(kv) == 2


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
def test_prefill_heads(w4, Hq, Hkv, D):
    prefill(w4, [1, 3, 17, 40, 130], [1, 70, 17, 41, 130], Hq, Hkv, D, seed=Hq)


@pytest.mark.parametrize("Hq,Hkv,D", [(128, 1, 64), (64, 1, 128), (130, 2, 64), (1, 1, 128)])
def test_wide_and_single_groups(w4, Hq, Hkv, D):
    """Up to 128 query heads on one key-value head; a single head."""
    decode(w4, [1, 33, 150], Hq, Hkv, D, seed=Hq)
    prefill(w4, [3, 1, 5], [40, 1, 140], Hq, Hkv, D, seed=Hq)


@pytest.mark.parametrize("qs,lens", [([1], [1]), ([128], [128]), ([129], [129]), ([127], [255]), ([5], [1030]),
                                     ([300], [333]), ([64, 1, 200, 0, 31], [64, 500, 201, 60, 31])])
@pytest.mark.parametrize("D", [64, 128])
def test_prefill_lengths(w4, qs, lens, D):
    prefill(w4, qs, lens, 4, 2, D, 32, seed=D)


@pytest.mark.parametrize("layout", ["hnd", "nhd", "mixed"])
@pytest.mark.parametrize("ps", [16, 64, 128, 256, 4096])
def test_prefill_pools(w4, layout, ps):
    prefill(w4, [50, 90], [170, 90], 6, 2, 64, ps, layout=layout, lead=1, pad=2)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 0), (17, 5), (64, 16), (130, 130), (1000, 3), (33, 40),
                                          (0, 7), (128, 4)])
def test_prefill_window(w4, window, sinks):
    prefill(w4, [70, 260], [500, 260], 4, 2, 64, window=window, sinks=sinks, seed=window)


def test_prefill_rows_without_a_key(w4):
    """More rows than cached tokens: the first rows see nothing."""
    prefill(w4, [9, 140, 3], [4, 10, 0], 4, 2, 64, max_len=16)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_prefill_hidden_keys_have_no_influence(w4, bad):
    """Keys and values that a row does not see, in blocks it reads: hidden by
    the window from every row, and by the causal mask from the earlier ones."""
    cache = Paged([600], 2, 64, 16)
    kv = cache.fill_random()
    k, v = (torch.tensor(x).bfloat16() for x in kv[0])
    k[20:180], v[20:180] = bad, bad
    cache.put(0, k, v)
    prefill(w4, [200], [600], 4, 2, 64, window=220, sinks=20, cache=cache, kv=[(to64(k), to64(v))])
    # the last key is not finite: only the last row sees it
    cache = Paged([300, 40], 2, 128, 32)
    kv = cache.fill_random()
    k, v = (torch.tensor(x).bfloat16() for x in kv[0])
    v[299, :, 5] = bad
    cache.put(0, k, v)
    qs = [290, 40]
    q = randn_bf16(330, 6, 128, seed=9).cuda()
    goff = torch.tensor([0, 290, 330], dtype=torch.int32, device="cuda")
    lse = torch.empty(330, 6, device="cuda")
    out = w4.w4_attn_prefill(q, cache.k, cache.v, goff, cache.kv_len, cache.table, 290, 300, lse=lse)
    assert w4.w4_get_device_error() == 0
    kk, vv = to64(k), to64(v)
    check(out[:289], lse[:289], BO.attention(to64(q[:289]), kk, vv, np.arange(10, 299), 128 ** -0.5), "causal")
    check(out[290:], lse[290:], BO.attention(to64(q[290:]), *kv[1], np.arange(40), 128 ** -0.5), "other sequence")
    last = to64(out[289])
    assert not np.isfinite(last[:, 5]).any() and np.isfinite(np.delete(last, 5, axis=1)).all()
    assert sum(qs) == 330


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_prefill_hidden_values_in_a_large_batch(w4, bad):
    """The same with enough items that each is worked on whole: the last key of
    every sequence is seen by its last row only."""
    lens, H = [45] * 8, 16
    cache = Paged(lens, H, 64, 16)
    kv = cache.fill_random()
    for b in range(8):
        k, v = (torch.tensor(x).bfloat16() for x in kv[b])
        v[44, b] = bad
        cache.put(b, k, v)
    q = randn_bf16(8 * 40, H, 64, seed=9).cuda()
    goff = torch.arange(0, 321, 40, dtype=torch.int32, device="cuda")
    out = w4.w4_attn_prefill(q, cache.k, cache.v, goff, cache.kv_len, cache.table, 40, 45)
    assert w4.w4_get_device_error() == 0
    for b in range(8):
        rows = slice(40 * b, 40 * b + 39)
        want = BO.attention(to64(q[rows]), kv[b][0], kv[b][1], np.arange(5, 44), 0.125)
        check(out[rows], None, want, f"sequence {b}")
        last = to64(out[40 * b + 39])
        assert not np.isfinite(last[b]).any() and np.isfinite(np.delete(last, b, axis=0)).all()


def test_page_offsets_past_32_bits(w4):
    """Pools of more than 2^32 elements: pages at both ends of one pool."""
    H, ps, D = 8, 64, 128
    pages = (1 << 32) // (H * ps * D) + 40
    free = torch.cuda.mem_get_info()[0]
    if free < 5 * pages * H * ps * D:
        pytest.skip("not enough device memory")
    pool = torch.empty(2, pages, H, ps, D, dtype=torch.bfloat16, device="cuda")
    c = Paged([150, 70], H, D, ps)
    ids = torch.tensor([[pages - 1, 3, pages - 7], [pages - 20, 0, 1 << 30]], dtype=torch.int32)
    c.table_cpu, c.table, c.k, c.v = ids, ids.cuda(), pool[0], pool[1]
    kv = c.fill_random()
    decode(w4, [150, 70], 16, H, D, ps, cache=c, kv=kv)
    prefill(w4, [130, 70], [150, 70], 16, H, D, ps, cache=c, kv=kv, rows=[0, 40, 69, 129])
    # the cache write: the last position of the first sequence, on its last page
    q, k, v = (randn_bf16(2, h, D, seed=h).cuda() for h in (16, H, H))
    inv = w4.w4_rope_freqs(D)[0].cuda()
    w4.w4_rope_append(q, k, k, c.k, c.v, c.kv_len, c.table, inv)
    assert torch.equal(c.v[pages - 7, :, 149 - 128], k[0]) and torch.equal(c.v[0, :, 69 - 64], k[1])
    assert v.shape == k.shape and w4.w4_get_device_error() == 0


def test_prefill_long(w4):
    rows = [0, 1, 127, 128, 1000, 2047, 2048, 4099]
    prefill(w4, [4100], [4100], 7, 1, 128, 64, rows=rows)
    prefill(w4, [300], [9000], 4, 1, 64, 64, rows=[0, 150, 299])
    prefill(w4, [2, 700], [8000, 6000], 8, 2, 128, 32, window=2000, sinks=9, rows=[0, 1, 699])


def test_prefill_bounds_only_size_the_launch(w4):
    cache = Paged([90, 33], 2, 64, 16)
    kv = cache.fill_random()
    a = prefill(w4, [40, 33], [90, 33], 4, 2, 64, cache=cache, kv=kv)
    b = prefill(w4, [40, 33], [90, 33], 4, 2, 64, cache=cache, kv=kv, max_q=73, max_len=100)
    assert (a.float() - b.float()).abs().max() < 0.05


def test_prefill_matches_decode(w4):
    """One row a sequence: both forms compute the same attention."""
    lens = [1, 50, 700]
    cache = Paged(lens, 2, 128, 16)
    kv = cache.fill_random()
    a = decode(w4, lens, 6, 2, 128, cache=cache, kv=kv, window=300, sinks=2)
    b = prefill(w4, [1] * 3, lens, 6, 2, 128, cache=cache, kv=kv, window=300, sinks=2)
    assert (a.float() - b.float()).abs().max() < 0.05


@pytest.mark.parametrize("Hq,Hkv,D", [(14, 2, 64), (28, 4, 128), (9, 3, 64), (17, 1, 128), (16, 2, 128)])
@pytest.mark.parametrize("qs,lens", [([50, 37], [400, 300]), ([300, 260], [300, 2000]), ([128] * 40, [128] * 40)])
def test_prefill_same_bits(w4, Hq, Hkv, D, qs, lens):
    """A sequence's result depends on its own inputs alone: not on the tokens that
    follow it, nor on what earlier calls left on chip in rows that no query fills."""
    cache = Paged(lens, Hkv, D, 16, fill=0.0)
    cache.fill_random(2.0)
    off = torch.tensor(np.concatenate([[0], np.cumsum(qs)]), dtype=torch.int32, device="cuda")
    T, sc = sum(qs), D ** -0.5

    def run(q, heads):
        return w4.w4_attn_prefill(q, cache.k[:, :heads], cache.v[:, :heads], off, cache.kv_len, cache.table, max(qs),
                                  max(lens), sc).clone()

    q = randn_bf16(T, Hq, D, seed=3, scale=2.0).cuda()
    wide = randn_bf16(T, 16 * Hkv, D, seed=4).cuda()      # 16 heads to one: every row of a tile is a query's
    first = None
    for left in (1.0, 60.0, 1.0, 300.0):
        run((wide * left).bfloat16(), Hkv)
        y = run(q, Hkv)
        other = q.clone()
        other[qs[0]:] *= left
        z = run(other, Hkv)[:qs[0]]
        first = y if first is None else first
        assert torch.equal(first, y), f"after queries of size {left}"
        assert torch.equal(first[:qs[0]], z), f"before tokens of size {left}"
    assert w4.w4_get_device_error() == 0


def test_prefill_bad_device_data(w4):
    q = randn_bf16(60, 4, 64, seed=1).cuda()

    def call(c, goff=(0, 20, 60), max_q=60, max_len=64):
        out = torch.full((60, 4, 64), -3.0, dtype=torch.bfloat16, device="cuda")
        w4.w4_attn_prefill(q, c.k, c.v, torch.tensor(goff, dtype=torch.int32, device="cuda"), c.kv_len, c.table, max_q,
                           max_len, out=out)
        return out, w4.w4_get_device_error()
    c = Paged([40, 50], 2, 64, 16, fill=1.0)
    c.fill_random()
    good, rc = call(c)
    assert rc == 0
    for bad in (-1, c.k.shape[0], -(1 << 31)):
        c.table[1, 1] = bad
        o, rc = call(c)
        assert rc == PAGE_ERR and torch.equal(o[:20], good[:20])
    c = Paged([40, 50], 2, 64, 16, fill=1.0)
    for n, lim in ((-1, 64), (49, 48), (1 << 30, 1 << 30)):
        c.kv_len[1] = n
        _, rc = call(c, max_len=lim)
        assert rc == PAGE_ERR
    c = Paged([40, 50], 2, 64, 16, fill=1.0)
    c.fill_random()
    for goff in ((0, 20, 61), (0, 20, 10), (-3, 20, 60)):
        o, rc = call(c, goff)
        assert rc == ROWS_ERR
    o, rc = call(c, max_q=30)               # the second sequence has 40 rows
    assert rc == ROWS_ERR and (o[20:] == -3.0).all()


def test_streams(w4):
    """Calls follow the stream they are given."""
    s = torch.cuda.Stream()
    lens = [700, 20]
    cache = Paged(lens, 2, 64, 16)
    cache.fill_random()
    q = randn_bf16(2, 4, 64, seed=1).cuda()
    want = w4.w4_attn_decode(q, cache.k, cache.v, cache.kv_len, cache.table, 700)
    torch.cuda.synchronize()
    ws = torch.zeros(w4.w4_attn_decode_workspace_bytes(4, 2, 64), dtype=torch.uint8, device="cuda")
    q2 = torch.zeros_like(q)
    out = torch.empty_like(q)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        q2.copy_(q)
        w4.w4_attn_decode(q2, cache.k, cache.v, cache.kv_len, cache.table, 700, out=out, workspace=ws)
    s.synchronize()
    assert torch.equal(out, want)


def test_graph_replay_follows_the_lengths(w4):
    """A captured step reads lengths and pages on the device: the replay follows
    them as the sequences grow."""
    cache = Paged([100, 230], 2, 64, 16)
    kv = cache.fill_random()
    q = randn_bf16(2, 4, 64, seed=1).cuda()
    ws = torch.zeros(w4.w4_attn_decode_workspace_bytes(4, 2, 64), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        w4.w4_attn_decode(q, cache.k, cache.v, cache.kv_len, cache.table, 230, out=out, workspace=ws)
    for lens in ([1, 230], [100, 17], [64, 0]):
        cache.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        for b, n in enumerate(lens):
            k, v = kv[b]
            check(out[b:b + 1], None, BO.attention(to64(q[b:b + 1]), k[:n], v[:n], [n - 1], 0.125), f"replay {n}")


def test_binding_refusals(w4):
    c = Paged([3, 4], 2, 64, 16, fill=0.0)
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda")
    goff = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    dec = dict(q=q, k_cache=c.k, v_cache=c.v, kv_len=c.kv_len, table=c.table, max_len=4)
    for kw, err in ((dict(q=q.half()), TypeError), (dict(q=q[:1]), ValueError), (dict(q=q[..., :32]), ValueError),
                    (dict(q=q[:, :3]), w4.W4Error), (dict(out=q.float()), TypeError),
                    (dict(lse=torch.zeros(2, 3, device="cuda")), ValueError), (dict(scale=-1.0), w4.W4Error),
                    (dict(window=-1), w4.W4Error), (dict(k_cache=c.k.float()), TypeError),
                    (dict(table=c.table.long()), TypeError)):
        with pytest.raises(err):
            w4.w4_attn_decode(**dict(dec, **kw))
        if "q" not in kw or kw["q"].shape[0] == 2:
            with pytest.raises(err):
                w4.w4_attn_prefill(**dict(dec, **kw), goff=goff, max_q=1)
    with pytest.raises(ValueError):
        w4.w4_attn_prefill(**dec, goff=goff[:2], max_q=1)
    e = q[:0]
    assert w4.w4_attn_prefill(e, c.k, c.v, goff * 0, c.kv_len, c.table, 1, 4).shape == e.shape


def test_integers_past_32_bits_are_refused(w4):
    """They must not be cut to their lower bits (a window of 2^32 to none)."""
    c = Paged([3, 4], 2, 64, 16, fill=0.0)
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda")
    goff = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    args = dict(q=q, k_cache=c.k, v_cache=c.v, kv_len=c.kv_len, table=c.table, max_len=4)
    for big in (1 << 31, 1 << 32, (1 << 32) + 4):
        for name in ("window", "sinks", "max_len"):
            with pytest.raises((ValueError, w4.W4Error)):
                w4.w4_attn_decode(**dict(args, **{name: big}))
            with pytest.raises((ValueError, w4.W4Error)):
                w4.w4_attn_prefill(**dict(args, **{name: big}), goff=goff, max_q=1)
        with pytest.raises((ValueError, w4.W4Error)):
            w4.w4_attn_prefill(**args, goff=goff, max_q=big)


@pytest.mark.parametrize("Hq,Hkv,D", [(17, 1, 128), (40, 1, 64), (24, 1, 64), (128, 1, 128), (66, 2, 64)])
def test_decode_wide_groups_over_long_sequences(w4, Hq, Hkv, D):
    """Several items of 16 heads read the same keys, each cut over CTAs."""
    for lens in ([9000], [1, 700, 3001, 250], [400 + 37 * i for i in range(20)]):
        decode(w4, lens, Hq, Hkv, D, 32, seed=Hq)
    decode(w4, [5000, 90], Hq, Hkv, D, 32, 1000, 33, seed=Hq)


@pytest.mark.parametrize("Hq,Hkv,D", [(28, 4, 128), (16, 8, 64)])
def test_prefill_uneven_batches(w4, Hq, Hkv, D):
    """One long prompt, or one chunk behind a long prefix, among sequences of a few tokens."""
    rows = [0, 1, 15, 700, 1499]
    prefill(w4, [1500] + [16] * 37, [1500] + [16] * 37, Hq, Hkv, D, 64, rows=rows)
    prefill(w4, [1] * 20 + [700] + [1] * 20, [300] * 20 + [900] + [7] * 20, Hq, Hkv, D, 64, rows=rows)
    prefill(w4, [300] + [1] * 7, [12000] + [90] * 7, Hq, Hkv, D, 64, rows=[0, 299])
