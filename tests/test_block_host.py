"""Host side of the decoder-block operators: rotary frequency tables against
the float64 oracle and worked values, the oracle's own closed forms, and every
argument check of the C entry points (no GPU: nothing reaches a kernel)."""
import ctypes
import math
import struct

import numpy as np
import pytest

from helpers import ensure_built
from oracle import block_oracle as BO
from test_abi import _codes

P = ctypes.c_void_p
OK16, ODD = 0x10000, 0x10001


@pytest.fixture(scope="module")
def w4():
    return ensure_built()


@pytest.mark.parametrize("kind,factor,orig", [("plain", 1.0, 0), ("linear", 4.0, 0), ("ntk", 8.0, 0),
                                              ("yarn", 16.0, 4096), ("yarn", 1.0, 8192), ("yarn", 40.0, 32)])
@pytest.mark.parametrize("rot,base", [(128, 1e4), (64, 1e6), (20, 5e5), (4, 1e4)])
def test_rope_freqs(w4, kind, factor, orig, rot, base):
    inv, m = w4.w4_rope_freqs(rot, base, kind, factor, orig)
    want, wm = BO.rope_freqs(rot, base, kind, factor, orig)
    # double arithmetic rounded once to fp32
    np.testing.assert_allclose(inv.numpy(), np.array(want), rtol=2.0 ** -23)
    assert abs(m - wm) <= 2.0 ** -23 * wm


def test_rope_freqs_worked_values(w4):
    inv, m = w4.w4_rope_freqs(4, 100.0)
    assert inv.tolist() == [1.0, np.float32(0.1)] and m == 1.0
    inv, _ = w4.w4_rope_freqs(4, 100.0, "linear", 2.0)
    assert inv.tolist() == [0.5, np.float32(0.05)]
    # NTK stretches the slowest pair by exactly `factor` and keeps the fastest
    inv, _ = w4.w4_rope_freqs(8, 1e4, "ntk", 4.0)
    assert inv[0] == 1.0 and abs(inv[3].item() - 1e4 ** -0.75 / 4) < 1e-9
    _, m = w4.w4_rope_freqs(64, 1e4, "yarn", 8.0, 4096)
    assert abs(m - (0.1 * math.log(8) + 1)) < 1e-6


def test_rope_freqs_refusals(w4):
    for args in ((3, 1e4), (0, 1e4), (64, 1.0), (64, float("inf")), (64, 1e4, "linear", 0.5),
                 (64, 1e4, "yarn", 2.0, 0), (64, 1e4, "yarn", 2.0, 4096, 1.0, 2.0), (2, 1e4, "ntk", 2.0),
                 (64, 1e4, "linear", float("nan"))):
        with pytest.raises(w4.W4Error):
            w4.w4_rope_freqs(*args)
    with pytest.raises(ValueError):
        w4.w4_rope_freqs(64, 1e4, "other")


def test_oracle_closed_forms():
    # one visible key: its value; equal scores: the mean; empty row: zero
    k = np.zeros((5, 1, 4))
    v = np.arange(20.0).reshape(5, 1, 4)
    o, lse, _ = BO.attention(np.ones((3, 1, 4)), k, v, [0, 4, -1], 1.0)
    assert np.array_equal(o[0, 0], v[0, 0]) and np.allclose(o[1, 0], v.mean(0)[0]) and not o[2].any()
    assert lse[0, 0] == 0 and np.isclose(lse[1, 0], math.log(5)) and lse[2, 0] == -np.inf
    see = BO.visible([6], 8, window=2, sinks=3)[0]
    assert see.tolist() == [True, True, True, False, False, True, True, False]
    x = BO.rope(np.array([[[1.0, 0.0, 0.0, 2.0]]]), [1], [math.pi / 2, math.pi])
    assert np.allclose(x, [[[0, 0, 1, -2.0]]])
    x = BO.rope(np.array([[[1.0, 0.0, 0.0, 2.0]]]), [1], [math.pi / 2, math.pi], interleaved=True)
    assert np.allclose(x, [[[0, 1, 0, -2.0]]])


def _kv(**kw):
    d = dict(k=OK16, v=OK16, table=OK16, len=OK16, kp=8192, kh=2048, ks=128, vp=8192, vh=2048, vs=128, ts=4,
             pages=9, ps=16, heads=4, d=128, batch=2, maxp=4)
    d.update(kw)
    return struct.pack("4Q7q6i", *d.values())


def _decode(lib, kv=None, q=OK16, qt=128 * 28, qh=128, out=OK16, lse=None, hq=28, max_len=64, scale=0.1, window=0,
            sinks=0, ws=OK16, wsb=1 << 30):
    return lib.w4_attn_decode(kv if kv is not None else _kv(), q, qt, qh, out, lse, hq, max_len, scale, window,
                              sinks, ws, wsb, None)


def _prefill(lib, kv=None, q=OK16, goff=OK16, out=OK16, T=8, hq=28, max_q=8, max_len=64, scale=0.1):
    return lib.w4_attn_prefill(kv if kv is not None else _kv(), q, 128 * hq, 128, goff, out, None, T, hq, max_q,
                               max_len, scale, 0, 0, None)


def test_cache_refusals(w4):
    lib, c = w4.load(), _codes()
    for kw, code in ((dict(k=0), "NULL_PTR"), (dict(v=0), "NULL_PTR"), (dict(table=0), "NULL_PTR"),
                     (dict(len=0), "NULL_PTR"), (dict(pages=0), "INVALID_ARG"), (dict(maxp=0), "INVALID_ARG"),
                     (dict(heads=0), "INVALID_ARG"), (dict(batch=-1), "INVALID_ARG"),
                     (dict(ps=8), "UNSUPPORTED_SHAPE"), (dict(ps=48), "UNSUPPORTED_SHAPE"),
                     (dict(ps=8192), "UNSUPPORTED_SHAPE"), (dict(k=ODD), "MISALIGNED"),
                     (dict(table=0x10002), "MISALIGNED"), (dict(ks=132), "MISALIGNED"), (dict(vp=0), "INVALID_ARG"),
                     (dict(kh=-8), "INVALID_ARG"), (dict(ts=-1), "INVALID_ARG")):
        want = c["W4_ERR_" + code]
        assert _decode(lib, _kv(**kw)) == want, kw
        assert _prefill(lib, _kv(**kw)) == want, kw
        assert _rope(lib, kv=_kv(**kw)) == want, kw
    assert _decode(lib, _kv(d=96)) == c["W4_ERR_UNSUPPORTED_SHAPE"]
    assert lib.w4_attn_decode(None, OK16, 1, 1, OK16, None, 28, 64, 0.1, 0, 0, OK16, 1 << 30, None) == \
        c["W4_ERR_NULL_PTR"]


def test_attention_refusals(w4):
    lib, c = w4.load(), _codes()
    for kw, code in ((dict(q=None), "NULL_PTR"), (dict(out=None), "NULL_PTR"), (dict(hq=30), "INVALID_ARG"),
                     (dict(hq=0), "INVALID_ARG"), (dict(hq=4 * 129), "UNSUPPORTED_SHAPE"),
                     (dict(scale=0.0), "INVALID_ARG"), (dict(scale=-1.0), "INVALID_ARG"),
                     (dict(scale=float("nan")), "INVALID_ARG"), (dict(scale=float("inf")), "INVALID_ARG"),
                     (dict(max_len=-1), "INVALID_ARG"), (dict(q=ODD), "MISALIGNED"), (dict(out=0x10008), "MISALIGNED")):
        assert _decode(lib, **kw) == c["W4_ERR_" + code], kw
        assert _prefill(lib, **kw) == c["W4_ERR_" + code], kw
    for kw, code in ((dict(window=-1), "INVALID_ARG"), (dict(sinks=-1), "INVALID_ARG"), (dict(qt=4), "MISALIGNED"),
                     (dict(qh=-8), "INVALID_ARG"), (dict(lse=0x10002), "MISALIGNED")):
        assert _decode(lib, **kw) == c["W4_ERR_" + code], kw
    for kw, code in ((dict(goff=None), "NULL_PTR"), (dict(goff=0x10002), "MISALIGNED"), (dict(T=-1), "INVALID_ARG"),
                     (dict(max_q=-1), "INVALID_ARG")):
        assert _prefill(lib, **kw) == c["W4_ERR_" + code], kw
    # nothing to do: no workspace needed, nothing enqueued
    assert _decode(lib, _kv(batch=0), ws=None, wsb=0) == c["W4_OK"]
    assert _prefill(lib, T=0) == c["W4_OK"]
    assert _prefill(lib, max_q=0) == c["W4_OK"]
    assert _decode(lib, ws=None) == c["W4_ERR_WORKSPACE"]
    assert _decode(lib, wsb=16) == c["W4_ERR_WORKSPACE"]
    assert lib.w4_attn_decode_workspace_bytes(30, 4, 128) == 0


def _rope(lib, kv=None, q=OK16, k=OK16, v=OK16, goff=None, pos=None, inv=OK16, m=1.0, rot=128, out=OK16, T=2, hq=28,
          qt=4608):
    return lib.w4_rope_append(kv if kv is not None else _kv(), q, qt, 128, k, 4608, 128, v, 4608, 128, goff, pos, inv,
                              m, rot, 0, out, T, hq, None)


def test_rope_refusals(w4):
    lib, c = w4.load(), _codes()
    for kw, code in ((dict(q=None), "NULL_PTR"), (dict(k=None), "NULL_PTR"), (dict(v=None), "NULL_PTR"),
                     (dict(out=None), "NULL_PTR"), (dict(inv=None), "NULL_PTR"), (dict(rot=130), "INVALID_ARG"),
                     (dict(rot=7), "INVALID_ARG"), (dict(T=3), "INVALID_ARG"), (dict(T=-1), "INVALID_ARG"),
                     (dict(hq=0), "INVALID_ARG"), (dict(qt=-8), "INVALID_ARG"), (dict(m=float("nan")), "INVALID_ARG"),
                     (dict(q=ODD), "MISALIGNED"), (dict(goff=0x10002), "MISALIGNED"), (dict(inv=0x10002), "MISALIGNED")):
        assert _rope(lib, **kw) == c["W4_ERR_" + code], kw
    assert _rope(lib, _kv(d=260), rot=64) == c["W4_ERR_UNSUPPORTED_SHAPE"]
    assert _rope(lib, _kv(batch=0), T=0) == c["W4_OK"]


def test_norm_refusals(w4):
    lib, c = w4.load(), _codes()
    base = dict(y=OK16, r=OK16, wpost=OK16, gate=None, wpre=OK16, rout=OK16, xout=OK16, M=4, K=64, rows=0, a=1.0,
                eps=1e-6, off=0.0)

    def call(**kw):
        return lib.w4_block_norm(*dict(base, **kw).values(), None)
    for kw, code in ((dict(r=None), "NULL_PTR"), (dict(rout=None), "NULL_PTR"), (dict(wpre=None), "NULL_PTR"),
                     (dict(y=None), "INVALID_ARG"), (dict(y=None, wpost=None), "INVALID_ARG"),
                     (dict(M=-1), "INVALID_ARG"), (dict(K=0), "INVALID_ARG"), (dict(K=32769), "UNSUPPORTED_SHAPE"),
                     (dict(eps=-1.0), "INVALID_ARG"), (dict(eps=float("nan")), "INVALID_ARG"),
                     (dict(rows=1), "INVALID_ARG"), (dict(gate=OK16), "INVALID_ARG"),
                     (dict(gate=OK16, rows=3), "INVALID_ARG"), (dict(gate=OK16, rows=-1), "INVALID_ARG"),
                     (dict(a=float("inf")), "INVALID_ARG"), (dict(y=ODD), "MISALIGNED"), (dict(xout=ODD), "MISALIGNED")):
        assert call(**kw) == c["W4_ERR_" + code], kw
    assert call(M=0) == c["W4_OK"]


def test_query_strides_of_extent_one_are_ignored(w4):
    """As those of the cache are: one token, or one head, may have any."""
    lib, c = w4.load(), _codes()
    refused, fine = c["W4_ERR_MISALIGNED"], c["W4_ERR_WORKSPACE"]
    one = _kv(heads=1, batch=1)
    assert _decode(lib, _kv(batch=1), qt=4, ws=None) == fine and _decode(lib, qt=4, ws=None) == refused
    assert _decode(lib, one, hq=1, qh=3, qt=-1, ws=None) == fine and _decode(lib, one, hq=2, qh=3, ws=None) == refused

    def chunk(T, hq, qt, qh):
        return lib.w4_attn_prefill(_kv(heads=1), OK16, qt, qh, OK16, OK16, None, T, hq, 0, 64, 0.1, 0, 0, None)
    assert chunk(1, 1, 3, 0) == c["W4_OK"] and chunk(1, 2, 4, 128) == c["W4_OK"] and chunk(2, 1, 128, 5) == c["W4_OK"]
    assert chunk(2, 1, 4, 128) == refused and chunk(1, 2, 128, 5) == refused
