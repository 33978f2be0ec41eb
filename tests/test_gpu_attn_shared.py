"""GPU parity of w4_attn_shared against the float64 oracle, with the bounds of w4_attn_prefill (the weights of
the shared keys are rounded to bf16): 2^-8 |o| + (2^-8 + 2^-11) sum w |v|, log-sum-exp 2^-12 + 2^-20 of it."""
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


class Batch:
    """groups: (shared tokens, each sequence's own tokens; None: an unused row).  Whole pages of a prefix are one
    sequence's; the page where it ends is copied to all, as a server does that shares whole pages only."""

    def __init__(self, groups, Hq, Hkv, D, ps=16, layout="hnd", seed=0, before=0, after=0, scale=1.0):
        self.Hq, self.Hkv, self.D, self.ps = Hq, Hkv, D, ps
        self.sizes = [len(own) for _, own in groups]
        self.shared = [n for n, _ in groups]
        of = [i for i, n in enumerate(self.sizes) for _ in range(n)]
        own = [m for _, o in groups for m in o]
        # sequences outside every group have 40 tokens of their own
        lens = [40] * before + [0 if m is None else groups[i][0] + m for i, m in zip(of, own)] + [40] * after
        self.first = np.concatenate([[0], np.cumsum(self.sizes)]) + before
        self.cache = Paged(lens, Hkv, D, ps, layout, seed)
        self.kv = self.cache.fill_random(scale)
        t = self.cache.table_cpu
        for i, n in enumerate(self.shared):
            lead = self.first[i]
            if self.sizes[i] == 0 or lens[lead] == 0:
                continue
            for b in range(lead + 1, self.first[i + 1]):
                if lens[b] == 0:
                    continue
                k, v = self.kv[lead][0][:n], self.kv[lead][1][:n]
                self.kv[b] = (np.concatenate([k, self.kv[b][0][n:]]), np.concatenate([v, self.kv[b][1][n:]]))
                part = n // ps * ps
                self.cache.put(b, *(torch.from_numpy(x) for x in self.kv[b]))
                # the others' entries of whole pages are never looked at
                t[b, :part // ps] = 1 << 30
        self.cache.table = t.cuda()
        self.lens = lens
        B = len(lens)
        q = torch.zeros(B, Hq * D + 24, dtype=torch.bfloat16)
        q[:, 8:8 + Hq * D] = randn_bf16(B, Hq * D, seed=seed + 9)
        self.q = q.cuda()[:, 8:8 + Hq * D].unflatten(1, (Hq, D))
        self.group = torch.tensor(self.first, dtype=torch.int32, device="cuda")
        self.shared_d = torch.tensor(self.shared, dtype=torch.int32, device="cuda")

    def args(self):
        c = self.cache
        return self.q, c.k, c.v, c.kv_len, c.table, self.group, self.shared_d, max(self.lens)

    def run(self, w4, want_err=0, **kw):
        B = len(self.lens)
        out, raw = guarded_empty((B, self.Hq, self.D), torch.bfloat16)
        lse, raw2 = guarded_empty((B, self.Hq), torch.float32)
        out.fill_(-3.0)
        n = w4.w4_attn_shared_scratch_bytes(B, self.Hq, self.Hkv, self.D)
        scratch, raw3 = guarded_empty((n,), torch.uint8)
        scratch.fill_(255)                        # NaN: nothing is taken from it that was not put there
        w4.w4_attn_shared(*self.args(), out=out, lse=lse, scratch=scratch, **kw)
        for r, name in ((raw, "out"), (raw2, "lse"), (raw3, "scratch")):
            check_band(r, name)
        err = w4.w4_get_device_error()
        assert err == want_err if want_err is not None else err in (PAGE_ERR, ROWS_ERR)
        return out, lse

    def check(self, w4, rows=None, **kw):
        out, lse = self.run(w4, **kw)
        for b in range(len(self.lens)) if rows is None else rows:
            n = self.lens[b]
            ref, wl, mag = BO.attention(to64(self.q[b:b + 1]), *self.kv[b], [n - 1], kw.get("scale", self.D ** -0.5))
            what = f"{self.Hq}/{self.Hkv}x{self.D} page {self.ps} sequence {b} length {n}"
            within(out[b:b + 1], ref, U * np.abs(ref) + (U + 2.0 ** -11) * mag, what)
            wl32 = np.abs(np.where(np.isfinite(wl), wl, 0))
            within(lse[b:b + 1].cpu().numpy().astype(np.float64), wl, 2.0 ** -12 + 2.0 ** -20 * wl32, what + " lse")
        return out, lse


HEADS = [(28, 4, 128), (4, 4, 64), (8, 1, 128), (16, 1, 64), (9, 3, 64), (17, 1, 128), (40, 1, 64), (5, 5, 128),
         (128, 1, 64), (65, 1, 128)]


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
def test_heads(w4, Hq, Hkv, D):
    Batch([(200, [1, 17, 40]), (64, [3] * 5)], Hq, Hkv, D, seed=Hq).check(w4)


@pytest.mark.parametrize("n", [0, 1, 15, 16, 17, 127, 128, 129, 255, 300, 1000])
def test_shared_lengths(w4, n):
    Batch([(n, [1, 0, 30] if n else [1, 2, 30])], 6, 2, 64, seed=n).check(w4)
    Batch([(n, [0, 0] if n else [1, 1])], 6, 2, 128, seed=n).check(w4)


@pytest.mark.parametrize("layout", ["hnd", "nhd", "mixed"])
@pytest.mark.parametrize("ps", [16, 32, 128, 4096])
def test_pools(w4, layout, ps):
    Batch([(333, [5, 70]), (100, [1])], 6, 2, 64, ps, layout).check(w4)


@pytest.mark.parametrize("own", [[0], [1], [16], [400], [0, 300, 1, 17, 128, 5, 2, 2, 90]])
def test_own_lengths(w4, own):
    Batch([(150, own)], 28, 4, 128, seed=len(own)).check(w4)


def test_groups_of_every_kind(w4):
    """Empty ones, one without shared keys, unused rows, sequences outside every group, more groups than a warp."""
    Batch([(0, []), (50, [3, 1]), (0, [9, 4]), (130, []), (0, [None, None]), (65, [2, None, 8]), (0, [])], 4, 2, 64,
          before=3, after=2).check(w4)
    Batch([(16 + 7 * (i % 9), [1 + i % 3] * (1 + i % 2)) for i in range(70)], 4, 2, 64, before=1, after=1).check(w4)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [140, 900])
@pytest.mark.parametrize("B", [1, 17, 18, 19, 36, 37, 40, 120])
def test_tiles(w4, B, n, D):
    """18 sequences of 7 heads fill a tile; sequences of every place in a pair of tiles, pairs and lone tiles."""
    Batch([(n, [1 + b % 4 for b in range(B)])], 7, 1, D, seed=B).check(w4)


@pytest.mark.parametrize("blocks", list(range(1, 10)))
def test_lone_tiles_over_few_blocks(w4, blocks):
    """Items of 64-wide heads with one tile take every second block in turn: parts of one block, of odd and
    even numbers of them, one item after the other in a CTA (more items than CTAs)."""
    Batch([(128 * blocks - 7, [2, 1])] * 3, 4, 2, 64, 64, seed=blocks).check(w4)
    b = Batch([(128 * (1 + (i + blocks) % 5), [1]) for i in range(90)], 4, 4, 64, 64, seed=blocks)
    b.check(w4, rows=range(0, 90, 7))


@pytest.mark.parametrize("Hq,Hkv,D,n", [(28, 4, 128, 9000), (8, 1, 64, 30000), (16, 16, 64, 3000)])
def test_long_prefixes_in_many_parts(w4, Hq, Hkv, D, n):
    Batch([(n, [3, 50]), (n // 2 + 5, [1])], Hq, Hkv, D, 64, seed=n).check(w4)


def test_whole_items_and_parts_together(w4):
    """More items than CTAs, of very different lengths."""
    groups = [(20 + 37 * (i % 11), [1 + i % 5] * (1 + i % 4)) for i in range(60)] + [(5000, [2, 3])]
    Batch(groups, 8, 4, 64, 16, seed=3).check(w4)


def test_large_scores_and_a_growing_maximum(w4):
    b = Batch([(700, [40, 3, 90])], 4, 2, 128, scale=20.0)
    b.check(w4)
    b.check(w4, scale=1.0)


def test_keys_without_influence(w4):
    """Every slot that no sequence sees is NaN (Paged fills with it); infinities too."""
    b = Batch([(75, [1, 0]), (16, [5])], 4, 2, 64, 32)
    want, lse = b.check(w4)
    pool = b.cache.k
    seen = torch.zeros(pool.shape[0], b.ps, dtype=torch.bool)
    for s, n in enumerate(b.lens):
        for j in range(n):
            page = int(b.cache.table_cpu[s, j // b.ps])
            if page < pool.shape[0]:
                seen[page, j % b.ps] = True
    hide = ~seen.cuda()[:, None, :, None].expand_as(pool)
    for bad in (float("inf"), float("-inf"), 3e38):
        b.cache.k[hide] = bad
        b.cache.v[hide] = bad
        out, l2 = b.run(w4)
        assert torch.equal(out, want) and torch.equal(l2, lse)


def test_visible_infinities(w4):
    b = Batch([(40, [3, 5])], 4, 2, 64)
    t = b.cache.table_cpu
    b.cache.v[int(t[0, 0]), 0, 2, 7] = float("inf")          # in the prefix: both sequences, heads 0 and 1
    b.cache.v[int(t[1, 2]), 1, 9, 3] = float("-inf")         # key 41 of sequence 1
    out, _ = b.run(w4)
    inf = torch.isinf(out.float())
    assert inf[:, :2, 7].all() and inf[1, 2:, 3].all() and inf.sum() == 6 and not out.isnan().any()


def test_an_unused_first_sequence_still_names_the_pages(w4):
    b = Batch([(40, [3, 9, 1])], 4, 2, 64)
    want, _ = b.check(w4)
    b.cache.kv_len[0] = 0
    out, _ = b.run(w4)
    assert not out[0].any() and torch.equal(out[1:], want[1:])


def test_rows_that_see_nothing(w4):
    b = Batch([(40, [3, None]), (0, [None])], 4, 2, 64)
    b.q[1:] = float("nan")
    out, lse = b.run(w4)
    assert not out[1:].any() and (lse[1:] == float("-inf")).all() and torch.isfinite(out[0].float()).all()


def test_the_same_as_attention_without_sharing(w4):
    """Against w4_attn_decode on whole tables, in a run long enough for several parts and splits of own keys."""
    groups = [(4096, [700, 3, 1, 90] * 3), (2048, [33] * 5)]
    b = Batch(groups, 28, 4, 128, 64)
    t = b.cache.table_cpu.clone()
    for i, n in enumerate(b.shared):
        t[b.first[i]:b.first[i + 1], :n // 64] = t[b.first[i], :n // 64]
    lse = torch.empty(len(b.lens), 28, device="cuda")
    want = w4.w4_attn_decode(b.q, b.cache.k, b.cache.v, b.cache.kv_len, t.cuda(), max(b.lens), lse=lse)
    out, l2 = b.run(w4)
    d = out.float() - want.float()
    assert d.norm() <= 2 * 2.0 ** -8 * want.float().norm() and (l2 - lse).abs().max() < 2.0 ** -11
    first = out.clone()
    for _ in range(3):                                       # the same inputs give the same bits
        out, _ = b.run(w4)
        assert torch.equal(out, first)


def test_flags(w4):
    b = Batch([(40, [3, 1]), (40, [2])], 4, 2, 64)
    table = b.cache.table.clone()
    b.cache.table[b.cache.table >= b.cache.k.shape[0]] = 0   # no other flag than the one looked for
    for name, value, err in (("group", [0, 2, 9], ROWS_ERR), ("group", [0, -1, 3], ROWS_ERR), ("group", [2, 1, 3], ROWS_ERR),
                             ("group", [0, 2, 1 << 30], ROWS_ERR), ("shared_d", [1 << 30, 40], PAGE_ERR),
                             ("shared_d", [-1, 40], PAGE_ERR), ("shared_d", [42, 40], PAGE_ERR)):
        keep = getattr(b, name)
        setattr(b, name, torch.tensor(value, dtype=torch.int32, device="cuda"))
        b.run(w4, want_err=err)
        setattr(b, name, keep)
    b.cache.table = table
    b.check(w4)
    b.cache.table[0, 1] = b.cache.k.shape[0]
    b.run(w4, want_err=PAGE_ERR)


def test_offsets_in_any_order_stay_inside_the_buffers(w4):
    """Decreasing offsets are flagged; what they leave of the lists reads and writes nothing out of range (guard
    bands around the outputs and the scratch), and the next call is sound."""
    b = Batch([(30 + 50 * (i % 4), [1 + 40 * (i % 3)] * (1 + i % 5)) for i in range(40)], 8, 2, 64)
    b.cache.table[b.cache.table >= b.cache.k.shape[0]] = 0
    good, shared = b.group, b.shared_d
    for seed in range(6):
        g = torch.Generator().manual_seed(seed)
        b.group = good[torch.randperm(41, generator=g).cuda()].contiguous()
        b.shared_d = torch.randint(0, max(b.lens), (40,), generator=g, dtype=torch.int32).cuda()
        b.run(w4, want_err=None)
    b.group, b.shared_d = good, shared
    b.run(w4)


def test_max_len_bounds_the_prefix(w4):
    b = Batch([(40, [3, 1])], 4, 2, 64)
    c = b.cache
    w4.w4_attn_shared(b.q, c.k, c.v, c.kv_len, c.table, b.group, b.shared_d, 30)
    assert w4.w4_get_device_error() == PAGE_ERR


def test_captured_and_replayed(w4):
    """A graph whose lengths, offsets and queries change; the scratch is the graph's."""
    b = Batch([(100, [9, 2]), (64, [1, 1, 5])], 28, 4, 128)
    b.check(w4)
    b.cache.table[3:5, :4] = b.cache.table[2, :4]            # pages that stop being shared below
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = w4.w4_attn_shared(*b.args())
    for step in range(3):
        b.q.copy_(randn_bf16(5, 28, 128, seed=step).cuda())
        b.cache.kv_len[0] -= 1
        b.shared_d[1] -= 16
        want = w4.w4_attn_shared(*b.args())
        out.fill_(0)
        graph.replay()
        assert torch.equal(out, want)
    lens = b.cache.kv_len.tolist()
    for s, n in enumerate(lens):
        k, v = b.kv[s]
        ref, _, mag = BO.attention(to64(b.q[s:s + 1]), k[:n], v[:n], [n - 1], 128 ** -0.5)
        within(out[s:s + 1], ref, U * np.abs(ref) + (U + 2.0 ** -11) * mag, f"sequence {s}")
    assert w4.w4_get_device_error() == 0


def test_pages_past_two_to_the_31_values(w4):
    """The batch's pages at the end of a pool of 2.2e9 values (4.4 GB each)."""
    b = Batch([(150, [9, 70]), (64, [3])], 4, 2, 128, 64)
    want, lse = b.check(w4)
    c, far = b.cache, 2 ** 31 // (2 * 64 * 128) + 40
    for name in ("k", "v"):
        pool = torch.empty(far + getattr(c, name).shape[0], 2, 64, 128, dtype=torch.bfloat16, device="cuda")
        pool[far:] = getattr(c, name)
        setattr(c, name, pool)
    c.table = torch.where(c.table < (1 << 30), c.table + far, c.table)
    out, l2 = b.run(w4)
    assert torch.equal(out, want) and torch.equal(l2, lse)


@pytest.mark.parametrize("n,own,Hq,Hkv,D", [(700, [30, 300, 1, 9], 28, 4, 128), (3000, [200] * 24, 8, 2, 64), (64, [1, 2], 4, 4, 64)])
def test_calls_in_a_row_see_what_was_written_just_before(w4, n, own, Hq, Hkv, D):
    """Every call writes new keys at the end of each sequence (and into the prefix's last page) and reads them at
    once, without a pause between calls; each result is that of the same call between synchronizes."""
    import int4_weight_only_gb300 as raw
    b = Batch([(n, own)], Hq, Hkv, D, 64)
    c, B, steps = b.cache, len(own), 60
    g = torch.Generator().manual_seed(n)
    inv = raw.w4_rope_freqs(D)[0].cuda()
    qkv = torch.randn(steps, B, Hq + 2 * Hkv, D, generator=g).bfloat16().cuda()
    table = c.table.clone()
    table[table >= c.k.shape[0]] = 0
    first = torch.tensor([n], dtype=torch.int32, device="cuda")
    k0, v0 = c.k.clone(), c.v.clone()

    def step(i, q):
        x = qkv[i]
        raw.w4_rope_append(x[:1, :Hq], x[:1, Hq:Hq + Hkv], x[:1, Hq + Hkv:], c.k, c.v, first, table[:1], inv)   # key n - 1
        raw.w4_rope_append(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], c.k, c.v, c.kv_len, table, inv, q_out=q)
        return raw.w4_attn_shared(q, c.k, c.v, c.kv_len, table, b.group, b.shared_d, max(b.lens))
    q = torch.empty(B, Hq, D, dtype=torch.bfloat16, device="cuda")
    for _ in range(2):
        c.k.copy_(k0)
        c.v.copy_(v0)
        torch.cuda.synchronize()
        fast = [step(i, q) for i in range(steps)]
        torch.cuda.synchronize()
        c.k.copy_(k0)
        c.v.copy_(v0)
        for i in range(steps):
            torch.cuda.synchronize()
            want = step(i, q)
            torch.cuda.synchronize()
            assert torch.equal(fast[i], want), i
    assert raw.w4_get_device_error() == 0


def test_two_streams_with_their_own_buffers(w4):
    b = Batch([(3000, [9, 200, 1, 40])], 28, 4, 128)
    want, _ = b.check(w4, rows=[0])
    side = [torch.cuda.Stream() for _ in range(2)]
    need = w4.w4_attn_shared_scratch_bytes(4, 28, 4, 128)
    mine = torch.empty(need, dtype=torch.uint8, device="cuda")      # one stream's own, the other's from its calls
    outs = [torch.zeros(4, 28, 128, dtype=torch.bfloat16, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        w4.w4_attn_shared(*b.args(), out=o, scratch=mine if i % 2 else None, stream=side[i % 2])
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs) and w4.w4_get_device_error() == 0


def test_binding_refusals(w4):
    b = Batch([(40, [3, 1])], 4, 2, 64)
    q, k, v, n, t, g, s, m = b.args()
    for bad in ((q[:1], k, v, n, t, g, s, m), (q, k, v, n, t, g[:1], s, m), (q, k, v, n, t, g[:1], s[:0], m),
                (q, k, v[:, :, :8], n, t, g, s, m), (q, k, v, n, t, g, s, 1 << 32), (q, k, v, n, t, g, s, -(1 << 32) + 40)):
        with pytest.raises(ValueError):
            w4.w4_attn_shared(*bad)
    for bad in ((q.float(), k, v, n, t, g, s, m), (q, k, v, n, t, g.long(), s, m), (q, k, v, n, t, g, s.cpu(), m)):
        with pytest.raises(TypeError):
            w4.w4_attn_shared(*bad)
    for kw in (dict(scale=0.0), dict(scratch=torch.empty(64, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(w4.W4Error):
            w4.w4_attn_shared(*b.args(), **kw)
    with pytest.raises(w4.W4Error):
        w4.w4_attn_shared(q[:, :1].expand(-1, 4, -1), k, v, n, t, g, s, m)
