"""GPU parity of w4_rope_append against the float64 oracle: rotated q, the cache
cells it writes, and every other cell of the pool untouched.

Bounds: an output is one bf16 rounding (2^-8) of a cos - c sin in fp32; cos and
sin are within 2^-20 (angle reduction) + 2^-20 (fast sine), so the value is
within 2^-18 of |a| + |c| (times mscale)."""
import numpy as np
import pytest
import torch

from block_helpers import Paged, U, randn_bf16, to64, within
from helpers import check_band, ensure_built, guarded_empty
from oracle import block_oracle as BO

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w4():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ensure_built()


def bound(x, ref, n, inter, m):
    """Of the rotated part: the size of each value's pair."""
    x = np.abs(x)
    mag = np.zeros_like(x)
    ia = np.arange(n) * 2 if inter else np.arange(n)
    ib = ia + 1 if inter else ia + n
    mag[..., ia] = mag[..., ib] = x[..., ia] + x[..., ib]
    return U * np.abs(ref) + 2.0 ** -18 * m * mag


def run(w4, qs, lens, Hq, Hkv, D, rot, inter=False, ps=16, layout="hnd", mscale=1.0, base=1e4, pos=None, seed=0,
        decode=False, lead=0, pad=0, k_offset=0):
    """qs tokens of sequences of length lens; lead rows before and pad rows
    after them belong to no sequence."""
    cache = Paged(lens, Hkv, D, ps, layout, seed, fill=7.0)
    inv = torch.tensor([base ** (-2 * i / max(rot, 1)) for i in range(rot // 2)], dtype=torch.float32)
    T = lead + sum(qs) + pad
    ld = (Hq + 2 * Hkv) * D + k_offset
    qkv = torch.zeros(T, ld, dtype=torch.bfloat16)
    qkv[:, k_offset:] = randn_bf16(T, ld - k_offset, seed=seed)
    heads = qkv.cuda()[:, k_offset:].unflatten(1, (Hq + 2 * Hkv, D))
    off = np.concatenate([[0], np.cumsum(qs)]) + lead
    goff = None if decode else torch.tensor(off, dtype=torch.int32, device="cuda")
    k0, v0 = cache.k.clone(), cache.v.clone()
    qo, raw = guarded_empty((T, Hq, D), torch.bfloat16)
    qo.fill_(-3.0)
    w4.w4_rope_append(heads[:, :Hq], heads[:, Hq:Hq + Hkv], heads[:, Hq + Hkv:], cache.k, cache.v, cache.kv_len,
                      cache.table, inv.cuda(), goff=goff, pos=None if pos is None else pos.cuda(), interleaved=inter,
                      mscale=mscale, q_out=qo)
    check_band(raw, "q_out")
    assert w4.w4_get_device_error() == 0
    x = to64(qkv)[:, k_offset:].reshape(T, Hq + 2 * Hkv, D)
    p = np.full(T, -1)
    seq = np.full(T, -1)
    for b, (n, m) in enumerate(zip(qs, lens)):
        p[off[b]:off[b + 1]] = np.arange(m - n, m)
        seq[off[b]:off[b + 1]] = b
    P = p if pos is None else pos.numpy()
    ref = BO.rope(x[:, :Hq + Hkv], P, inv.double().numpy(), inter, mscale)
    lim = bound(x[:, :Hq + Hkv], ref, rot // 2, inter, mscale)
    got = to64(qo)
    inside = seq >= 0
    assert (got[~inside] == -3.0).all()
    zero = inside & (p < 0)
    assert not got[zero].any()
    live = inside & (p >= 0)
    within(got[live], ref[live, :Hq], lim[live, :Hq], "q")
    kw, vw = to64(k0), to64(v0)
    klim = np.zeros_like(kw)
    for t in np.nonzero(live)[0]:
        pg, sl = int(cache.table_cpu[seq[t], p[t] // ps]), p[t] % ps
        kw[pg, :, sl], klim[pg, :, sl] = ref[t, Hq:], lim[t, Hq:]
        vw[pg, :, sl] = x[t, Hq + Hkv:]
    within(cache.k, kw, klim, "k cache")
    assert np.array_equal(to64(cache.v), vw), "v cache"
    return got


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("Hq,Hkv,D,rot", [(28, 4, 128, 128), (4, 4, 64, 64), (8, 1, 128, 64), (5, 5, 64, 20),
                                          (3, 1, 256, 256), (2, 2, 80, 48), (7, 1, 8, 2), (1, 1, 128, 0)])
def test_layouts(w4, inter, Hq, Hkv, D, rot):
    run(w4, [1, 9, 17, 33], [1, 40, 17, 100], Hq, Hkv, D, rot, inter, seed=D + rot)


@pytest.mark.parametrize("layout", ["hnd", "nhd", "mixed"])
@pytest.mark.parametrize("ps", [16, 64, 4096])
def test_pools(w4, layout, ps):
    run(w4, [5, 70], [21, 130], 6, 2, 64, 64, ps=ps, layout=layout)


def test_decode_form_and_unused_rows(w4):
    run(w4, [1] * 6, [1, 16, 17, 0, 300, 0], 28, 4, 128, 128, decode=True)
    # more rows than cached tokens: the first ones have no position
    run(w4, [4, 3], [2, 3], 4, 2, 64, 32)


def test_rows_outside_sequences(w4):
    run(w4, [3, 0, 5], [3, 9, 50], 4, 2, 64, 64, lead=2, pad=3)


def test_unaligned_projection(w4):
    for off in (1, 2, 4):
        for inter in (False, True):
            run(w4, [3, 5], [30, 5], 4, 2, 64, 64, inter, k_offset=off)


@pytest.mark.parametrize("inter", [False, True])
def test_far_positions(w4, inter):
    """The angle keeps its accuracy where fp32 products do not."""
    pos = torch.tensor([0, 1, 131071, 1048575, 16777213, 7654321, -5, -1000003], dtype=torch.int32)
    run(w4, [8], [64], 4, 2, 128, 128, inter, base=1e6, mscale=1.25, pos=pos)
    run(w4, [8], [64], 4, 2, 128, 64, inter, base=1e4, pos=pos)


def test_in_place_q(w4):
    cache = Paged([9], 2, 64, 16, fill=0.0)
    q, k, v = (randn_bf16(9, h, 64, seed=h).cuda() for h in (6, 2, 2))
    inv = w4.w4_rope_freqs(64)[0].cuda()
    goff = torch.tensor([0, 9], dtype=torch.int32, device="cuda")
    want = w4.w4_rope_append(q, k, v, cache.k, cache.v, cache.kv_len, cache.table, inv, goff)
    w4.w4_rope_append(q, k, v, cache.k, cache.v, cache.kv_len, cache.table, inv, goff, q_out=q)
    assert torch.equal(q, want)


def test_bad_device_data(w4):
    """Pages and lengths out of range write nothing and raise the flag; offsets
    out of range leave their rows alone."""
    codes = {"page": -13, "off": -11}
    inv = w4.w4_rope_freqs(64)[0].cuda()

    def call(c, qs, goff):
        T = sum(qs)
        q, k, v = (randn_bf16(T, h, 64, seed=h).cuda() for h in (4, 2, 2))
        out = torch.full((T, 4, 64), -3.0, dtype=torch.bfloat16, device="cuda")
        before = c.k.clone()
        w4.w4_rope_append(q, k, v, c.k, c.v, c.kv_len, c.table, inv,
                          goff=torch.tensor(goff, dtype=torch.int32, device="cuda"), q_out=out)
        return out, torch.equal(c.k, before)
    for page in (-1, 5, 1 << 30):
        c = Paged([3], 2, 64, 16, fill=1.0)
        c.table[0, 0] = c.k.shape[0] if page == 5 else page
        _, same = call(c, [3], [0, 3])
        assert same and w4.w4_get_device_error() == codes["page"]
    c = Paged([3], 2, 64, 16, fill=1.0)
    c.kv_len.fill_(16 * c.table.shape[1] + 1)
    call(c, [1], [0, 1])
    assert w4.w4_get_device_error() == codes["page"]
    for goff in ([0, 9], [-1, 3], [2, 1]):
        c = Paged([3], 2, 64, 16, fill=1.0)
        out, same = call(c, [3], goff)
        assert same and (out == -3.0).all() and w4.w4_get_device_error() in (0, codes["off"])


def test_binding_refusals(w4):
    c = Paged([3, 4], 2, 64, 16, fill=0.0)
    q, k = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, 2, 64, dtype=torch.bfloat16,
                                                                                 device="cuda")
    inv = torch.ones(32, device="cuda")
    args = dict(q=q, k=k, v=k, k_cache=c.k, v_cache=c.v, kv_len=c.kv_len, table=c.table, inv_freq=inv)
    for kw, err in ((dict(q=q.float()), TypeError), (dict(k=q), ValueError), (dict(v=k[:1]), ValueError),
                    (dict(q=q[..., ::2]), ValueError), (dict(kv_len=c.kv_len.long()), TypeError),
                    (dict(kv_len=c.kv_len[:1]), ValueError), (dict(table=c.table[0]), ValueError),
                    (dict(v_cache=c.v[..., :32]), ValueError), (dict(goff=c.kv_len), ValueError),
                    (dict(pos=c.kv_len[:1]), ValueError), (dict(inv_freq=torch.ones(33, device="cuda")), w4.W4Error),
                    (dict(q=q.cpu()), TypeError)):
        with pytest.raises(err):
            w4.w4_rope_append(**dict(args, **kw))
