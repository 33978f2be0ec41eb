"""GPU parity of w4_kv_plan against the sequential oracle: whole numbers, equal in every place."""
import random

import numpy as np
import pytest
import torch

from block_helpers import randn_bf16
from helpers import check_band, ensure_built, guarded_empty
from oracle import serve_oracle as SO

pytestmark = pytest.mark.gpu
CODES = dict(PAGE_TABLE=-13, GROUP_TOKENS=-11, NO_PAGES=-14)


@pytest.fixture(scope="module")
def w4():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ensure_built()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def plan(w4, lens, new, free, used, cols, ps, pages, T, seed=0, inplace=False, wide=0):
    B = len(lens)
    g = torch.Generator().manual_seed(seed)
    table = torch.randint(0, max(pages, 1), (B, cols + wide), generator=g, dtype=torch.int32)
    want = SO.plan(lens, new, np.array(free, np.int64), used, table[:, :cols].numpy().astype(np.int64), ps, pages, T)
    full = table.cuda()
    ld, ud = i32(lens), i32([used])
    outs = [guarded_empty(s, d) for s, d in (((B,), torch.int32), ((B + 1,), torch.int32), ((T,), torch.int32),
                                             ((T,), torch.int64), ((B,), torch.int32), ((1,), torch.int32))]
    kv, goff, pos, slots, lo, uo = (o for o, _ in outs)
    for o, _ in outs:
        o.fill_(-77)
    if inplace:
        lo, uo = ld, ud
    fd, nd = i32(free), None if new is None else i32(new)
    rc = w4.load().w4_kv_plan(ld.data_ptr(), None if nd is None else nd.data_ptr(), fd.data_ptr(), len(free), ud.data_ptr(),
                              full.data_ptr(), cols + wide, B, cols, ps, pages, T, kv.data_ptr(), goff.data_ptr(),
                              pos.data_ptr(), slots.data_ptr(), lo.data_ptr(), uo.data_ptr(), None)
    assert rc == 0
    for (_, raw), name in zip(outs, ("kv_len", "goff", "pos", "slots", "lens_out", "used_out")):
        check_band(raw, name)
    for got, name in ((kv, "kv_len"), (goff, "goff"), (pos, "pos"), (slots, "slots"), (lo, "lens_out")):
        bad = np.nonzero(got.cpu().numpy() != want[name])[0]
        assert not len(bad), (name, bad[:5], got.cpu().numpy()[bad[:5]], want[name][bad[:5]])
    assert uo.item() == want["used_out"]
    now = full.cpu().numpy()
    assert np.array_equal(now[:, :cols], want["table"]) and np.array_equal(now[:, cols:], table[:, cols:].numpy())
    err = w4.w4_get_device_error()
    assert err in {CODES[f] for f in want["flags"]} if want["flags"] else err == 0, (err, want["flags"])
    if not inplace:
        assert ld.tolist() == list(lens) and ud.item() == used
    return want


def perm(n, seed=0):
    return torch.randperm(n, generator=torch.Generator().manual_seed(seed)).tolist()


@pytest.mark.parametrize("ps", [16, 64, 4096])
@pytest.mark.parametrize("B", [1, 2, 31, 256, 1024, 1025, 8192])
def test_decode_steps(w4, B, ps):
    r = random.Random(B)
    lens = [r.choice([0, 1, ps - 1, ps, ps + 1, 3 * ps, r.randrange(4 * ps)]) for _ in range(B)]
    plan(w4, lens, None, perm(B + 9), 3, 5, ps, B + 9, B, seed=B)
    plan(w4, lens, [r.randrange(2) for _ in range(B)], perm(B + 9), 0, 5, ps, B + 9, B + 2, seed=B, inplace=True, wide=3)


@pytest.mark.parametrize("B,most,T_more", [(1, 1, 0), (1, 70000, 5), (2, 40000, 3), (3, 5000, 0), (40, 300, 1000), (97, 900, 1),
                                           (1500, 40, 3)])
@pytest.mark.parametrize("ps", [16, 128])
def test_prompts(w4, B, most, T_more, ps):
    r = random.Random(B + ps)
    new = [most if b == 0 else r.choice([0, 1, r.randrange(most + 1)]) for b in range(B)]
    lens = [r.choice([0, r.randrange(3000)]) for _ in range(B)]
    cols = max(-(-(n + m) // ps) for n, m in zip(lens, new)) + 1
    need = sum(-(-(n + m) // ps) - -(-n // ps) for n, m in zip(lens, new))
    plan(w4, lens, new, perm(need + 4, B), 4, cols, ps, need + 4, sum(new) + T_more, seed=ps, inplace=B % 2 == 0)


@pytest.mark.parametrize("short", [1, 3, 30])
def test_free_list_runs_out(w4, short):
    """The first request without pages and those behind it that need some; the others stay."""
    r = random.Random(short)
    lens = [r.randrange(200) for _ in range(60)]
    new = [r.choice([0, 1, 2, 40]) for _ in range(60)]
    need = sum(-(-(n + m) // 16) - -(-n // 16) for n, m in zip(lens, new))
    w = plan(w4, lens, new, perm(need - short, 5), 0, 20, 16, 500, sum(new), inplace=True)
    assert w["flags"] == {"NO_PAGES"}
    plan(w4, lens, new, [], 0, 20, 16, 500, sum(new))
    plan(w4, [5, 16, 16], [1, 1, 0], [3], 1, 4, 16, 9, 2)


def test_bad_lengths_offsets_and_pages(w4):
    big = (1 << 31) - 1
    plan(w4, [5, -1, 7, 100, 3], [1, 1, 1, 1, 1], perm(9), 0, 4, 16, 9, 5)               # -1; past the table
    plan(w4, [5, 6, 7], [1, -4, 2], perm(9), 0, 4, 16, 9, 5)                             # fewer than no tokens
    plan(w4, [big, big, 0, 60], [big, 1, big, 4], perm(9), 0, 4, 16, 9, 8)
    plan(w4, [0, 0, 0, 0], [3, 4, 5, 1], perm(9), 0, 4, 16, 9, 7)                        # rows behind T
    plan(w4, [0, 0, 0, 0], [3, 4, 5, 1], perm(9), 0, 4, 16, 9, 0)
    plan(w4, [0] * 3000, [big] * 3000, perm(9), 0, 4, 16, 9, 100)
    plan(w4, [0, 20, 40], [20, 20, 5], [3, 99, -1, 5, 6], 0, 4, 16, 9, 45)               # pages that are none
    plan(w4, [0, 20], [20, 1], perm(9), -3, 4, 16, 9, 21)                                # used out of range
    plan(w4, [0, 20], [20, 1], perm(9), 10, 4, 16, 9, 21)


def test_slots_past_32_bits(w4):
    pages = (1 << 31) - 1
    w = plan(w4, [4000, 0], [200, 4097], [pages - 1, 600000, 1 << 30], 0, 3, 4096, pages, 4297)
    assert w["slots"].max() > 1 << 42


def test_nothing_to_plan(w4):
    plan(w4, [], [], [], 0, 4, 16, 9, 0)
    plan(w4, [], [], [1, 2], 1, 4, 16, 9, 3)
    plan(w4, [3, 4], [0, 0], [], 0, 4, 16, 9, 0)


def test_binding_refusals(w4):
    lens, used, table, free = i32([1, 2]), i32([0]), torch.zeros(2, 4, dtype=torch.int32, device="cuda"), i32([1, 2])
    with pytest.raises(ValueError):
        w4.w4_kv_plan(lens, None, free, used, table[:1], 16, 9, 2)
    with pytest.raises(ValueError):
        w4.w4_kv_plan(lens, i32([1]), free, used, table, 16, 9, 2)
    with pytest.raises(TypeError):
        w4.w4_kv_plan(lens.long(), None, free, used, table, 16, 9, 2)
    with pytest.raises(ValueError):
        w4.w4_kv_plan(lens, None, free, used, table.t(), 16, 9, 2)
    with pytest.raises(ValueError):
        w4.w4_kv_plan(lens, None, free, used, table, 16, 9, -1)
    for pages, T in ((9, 1 << 32), (-(1 << 32) + 9, 2), (9, -(1 << 32) + 2)):
        with pytest.raises(ValueError):
            w4.w4_kv_plan(lens, None, free, used, table, 16, pages, T)
    with pytest.raises(ValueError):
        w4.w4_kv_plan(lens, None, free, used, table, 16, 9, 2, lens_out=i32([1]))
    with pytest.raises(w4.W4Error):
        w4.w4_kv_plan(lens, None, free, used, table, 48, 9, 2)


def test_a_captured_step_follows_the_lengths(w4):
    """A graph of plan, rotary positions with the cache write, and attention, replayed while the sequences grow
    over page ends: the same as the eager calls on tables made on the host."""
    B, Hq, Hkv, D, ps, steps = 3, 4, 2, 64, 16, 40
    free = i32(perm(64, 7))
    lens, used = i32([0, 13, 30]), i32([0])
    table = torch.full((B, 8), -1, dtype=torch.int32, device="cuda")
    # the pages of what is there already
    w4.w4_kv_plan(i32([0, 0, 0]), lens.clone(), free, used, table, ps, 64, 43, used_out=used)
    kc = torch.randn(64, Hkv, ps, D, device="cuda").bfloat16()
    vc = torch.randn_like(kc)
    kc2, vc2 = kc.clone(), vc.clone()
    inv = w4.w4_rope_freqs(D)[0].cuda()
    qkv = torch.empty(B, Hq + 2 * Hkv, D, dtype=torch.bfloat16, device="cuda")
    active = i32([1, 1, 1])

    def step():
        kv_len, _, pos, slots = w4.w4_kv_plan(lens, active, free, used, table, ps, 64, B, lens_out=lens, used_out=used)
        q = w4.w4_rope_append(qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], kc, vc, kv_len, table, inv)
        return w4.w4_attn_decode(q, kc, vc, kv_len, table, 128), kv_len, slots
    qkv.copy_(randn_bf16(B, Hq + 2 * Hkv, D, seed=0))
    keep = [t.clone() for t in (lens, used, table, kc, vc)]
    step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out, kv_len, slots = step()
    for t, k in zip((lens, used, table, kc, vc), keep):
        t.copy_(k)
    host = table.cpu().clone()
    n, at = [0, 13, 30], used.item()
    fl = free.tolist()
    for i in range(steps):
        qkv.copy_(randn_bf16(B, Hq + 2 * Hkv, D, seed=i + 1))
        on = [1, int(i != 5), int(i % 3 != 0)]
        active.copy_(torch.tensor(on, dtype=torch.int32))
        graph.replay()
        for b in range(B):
            if on[b]:
                if n[b] % ps == 0:
                    host[b, n[b] // ps] = fl[at]
                    at += 1
                n[b] += 1
        assert lens.tolist() == n and used.item() == at and torch.equal(table.cpu(), host)
        kl = i32([m if o else 0 for m, o in zip(n, on)])
        assert torch.equal(kv_len, kl)
        assert slots.tolist() == [host[b, (n[b] - 1) // ps].item() * ps + (n[b] - 1) % ps if on[b] else -1
                                  for b in range(B)] or not all(on)
        q = w4.w4_rope_append(qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], kc2, vc2, kl, host.cuda(), inv)
        assert torch.equal(w4.w4_attn_decode(q, kc2, vc2, kl, host.cuda(), 128), out)
    assert torch.equal(kc, kc2) and torch.equal(vc, vc2) and w4.w4_get_device_error() == 0
