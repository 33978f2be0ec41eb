"""Host side of the operators of a serving step: the oracle's closed forms and every
argument check of the C entry points (no GPU: nothing reaches a kernel)."""
import struct

import numpy as np
import pytest

from helpers import ensure_built
from oracle import serve_oracle as SO
from test_abi import _codes
from test_block_host import OK16, ODD, _kv


@pytest.fixture(scope="module")
def w4():
    return ensure_built()


def test_oracle_routes():
    z = np.log([[1.0, 2.0, 4.0, 1.0], [1.0, 1.0, 1.0, 1.0]])
    w, ids, row, goff = SO.route(z, 2)
    assert ids.tolist() == [[2, 1], [0, 1]] and np.allclose(w, [[2 / 3, 1 / 3], [0.5, 0.5]])
    assert goff.tolist() == [0, 1, 3, 4, 4] and row.tolist() == [[3, 1], [0, 2]]
    w, ids, _, _ = SO.route(z, 1, renorm=False, scale=3.0)
    assert np.allclose(w, [[1.5], [0.75]])
    # the bias chooses, the weight is the score's
    w, ids, _, _ = SO.route(z[:1], 1, bias=[1.0, 0, 0, 0], renorm=False)
    assert ids.tolist() == [[0]] and np.allclose(w, 1 / 8)
    # runs of two: by their best, or by the sum of both
    w, ids, _, _ = SO.route(np.log([[5.0, 0.1, 4.0, 3.0]]), 1, groups=2, best=1)
    assert ids.tolist() == [[0]]
    w, ids, _, _ = SO.route(np.log([[5.0, 0.1, 4.0, 3.0]]), 1, groups=2, best=2)
    assert ids.tolist() == [[2]]
    # nothing offered
    w, ids, row, goff = SO.route([[-np.inf, np.nan], [0.0, -np.inf]], 2)
    assert ids.tolist() == [[-1, -1], [0, -1]] and row.tolist() == [[-1, -1], [0, -1]] and w.tolist() == [[0, 0], [1, 0]]
    assert goff.tolist() == [0, 1, 1]


def test_oracle_plans():
    table = np.full((3, 4), -1)
    table[0, :2] = [7, 8]
    p = SO.plan([17, 0, 5], [16, 20, 0], [1, 2, 3, 4, 5, 6], 1, table, 16, 9, 38)
    assert p["kv_len"].tolist() == [33, 20, 0] and p["goff"].tolist() == [0, 16, 36, 36] and p["used_out"] == 4
    assert p["table"][0].tolist() == [7, 8, 2, -1] and p["table"][1].tolist() == [3, 4, -1, -1]
    assert p["pos"][:2].tolist() == [17, 18] and p["slots"][0] == 8 * 16 + 1 and p["slots"][15] == 2 * 16
    assert p["slots"][36:].tolist() == [-1, -1] and p["lens_out"].tolist() == [33, 20, 5] and not p["flags"]
    p = SO.plan([0, 15, 16], None, [1], 0, np.full((3, 2), 3), 16, 9, 3)
    assert p["kv_len"].tolist() == [1, 16, 0] and p["flags"] == {"NO_PAGES"} and p["lens_out"].tolist() == [1, 16, 16]


def _route(lib, logits=OK16, half=0, stride=64, bias=None, count=None, T=8, E=64, k=4, score=0, groups=1, top=1, best=1,
           scale=1.0, w=OK16, ids=OK16, row=OK16, goff=OK16, ws=OK16, wsb=1 << 20):
    return lib.w4_moe_route(logits, half, stride, bias, count, T, E, k, score, groups, top, best, 1, scale, w, ids, row,
                            goff, ws, wsb, None)


def test_route_refusals(w4):
    lib, c = w4.load(), _codes()
    for kw, code in ((dict(logits=None), "NULL_PTR"), (dict(w=None), "NULL_PTR"), (dict(ids=None), "NULL_PTR"),
                     (dict(row=None), "NULL_PTR"), (dict(goff=None), "NULL_PTR"), (dict(T=-1), "INVALID_ARG"),
                     (dict(E=0), "INVALID_ARG"), (dict(k=0), "INVALID_ARG"), (dict(k=65), "INVALID_ARG"),
                     (dict(groups=3), "INVALID_ARG"), (dict(groups=0), "INVALID_ARG"), (dict(top=2), "INVALID_ARG"),
                     (dict(top=0), "INVALID_ARG"), (dict(groups=32, top=1), "INVALID_ARG"), (dict(best=0), "INVALID_ARG"),
                     (dict(best=3), "INVALID_ARG"), (dict(score=2), "INVALID_ARG"), (dict(stride=-1), "INVALID_ARG"),
                     (dict(scale=float("nan")), "INVALID_ARG"), (dict(E=1025), "UNSUPPORTED_SHAPE"),
                     (dict(E=128, k=33), "UNSUPPORTED_SHAPE"), (dict(E=64, groups=64, top=64), "UNSUPPORTED_SHAPE"),
                     (dict(T=(1 << 22) + 1), "UNSUPPORTED_SHAPE"), (dict(logits=0x10002), "MISALIGNED"),
                     (dict(logits=ODD, half=1), "MISALIGNED"), (dict(bias=0x10002), "MISALIGNED"),
                     (dict(count=0x10002), "MISALIGNED"), (dict(T=65, ws=None), "WORKSPACE"),
                     (dict(T=65, wsb=8), "WORKSPACE"), (dict(T=65, ws=0x10008), "MISALIGNED")):
        assert _route(lib, **kw) == c["W4_ERR_" + code], kw
    assert w4.w4_moe_route_workspace_bytes(64, 64) == 0 and w4.w4_moe_route_workspace_bytes(65, 0) == 0
    assert w4.w4_moe_route_workspace_bytes(65, 60) >= 64 * 2
    assert w4.w4_moe_route_workspace_bytes(1 << 22, 1024) == 152 * 1024 * 2


def test_move_refusals(w4):
    lib, c = w4.load(), _codes()

    def gather(x=OK16, stride=64, row=OK16, out=OK16, T=4, k=2, K=64, R=8):
        return lib.w4_moe_gather(x, stride, row, out, T, k, K, R, None)

    def combine(x=OK16, row=OK16, w=OK16, shared=None, out=OK16, T=4, k=2, K=64, R=8):
        return lib.w4_moe_combine(x, row, w, shared, out, T, k, K, R, None)
    for kw, code in ((dict(x=None), "NULL_PTR"), (dict(row=None), "NULL_PTR"), (dict(out=None), "NULL_PTR"),
                     (dict(T=-1), "INVALID_ARG"), (dict(k=0), "INVALID_ARG"), (dict(K=0), "INVALID_ARG"),
                     (dict(R=-1), "INVALID_ARG"), (dict(k=33), "UNSUPPORTED_SHAPE"),
                     (dict(K=(1 << 22) + 1), "UNSUPPORTED_SHAPE"), (dict(x=ODD), "MISALIGNED"), (dict(out=ODD), "MISALIGNED"),
                     (dict(row=0x10002), "MISALIGNED")):
        assert gather(**kw) == c["W4_ERR_" + code], kw
        assert combine(**kw) == c["W4_ERR_" + code], kw
    assert gather(stride=-1) == c["W4_ERR_INVALID_ARG"] and gather(T=0, x=None) == c["W4_OK"]
    assert combine(w=None) == c["W4_ERR_NULL_PTR"] and combine(T=0, x=None) == c["W4_OK"]
    assert combine(w=0x10002) == c["W4_ERR_MISALIGNED"] and combine(shared=ODD) == c["W4_ERR_MISALIGNED"]


def test_plan_refusals(w4):
    lib, c = w4.load(), _codes()
    base = dict(lens=OK16, new=None, free=OK16, n=10, used=OK16, table=OK16, ts=8, batch=4, cols=8, ps=16, pages=9, T=4,
                kv=OK16, goff=OK16, pos=OK16, slots=OK16, lens_out=None, used_out=None)

    def call(**kw):
        return lib.w4_kv_plan(*dict(base, **kw).values(), None)
    for kw, code in ((dict(lens=None), "NULL_PTR"), (dict(free=None), "NULL_PTR"), (dict(used=None), "NULL_PTR"),
                     (dict(table=None), "NULL_PTR"), (dict(kv=None), "NULL_PTR"), (dict(goff=None), "NULL_PTR"),
                     (dict(pos=None), "NULL_PTR"), (dict(slots=None), "NULL_PTR"), (dict(batch=-1), "INVALID_ARG"),
                     (dict(n=-1), "INVALID_ARG"), (dict(T=-1), "INVALID_ARG"), (dict(cols=0), "INVALID_ARG"),
                     (dict(pages=0), "INVALID_ARG"), (dict(ts=-8), "INVALID_ARG"), (dict(ts=7), "INVALID_ARG"),
                     (dict(ps=8), "UNSUPPORTED_SHAPE"), (dict(ps=48), "UNSUPPORTED_SHAPE"),
                     (dict(ps=8192), "UNSUPPORTED_SHAPE"), (dict(batch=8193), "UNSUPPORTED_SHAPE"),
                     (dict(T=(1 << 30) + 1), "UNSUPPORTED_SHAPE"), (dict(n=(1 << 30) + 1), "UNSUPPORTED_SHAPE"),
                     (dict(cols=(1 << 26) + 1, ts=1 << 27), "UNSUPPORTED_SHAPE"), (dict(lens=0x10002), "MISALIGNED"),
                     (dict(slots=0x10004), "MISALIGNED"), (dict(lens_out=0x10002), "MISALIGNED")):
        assert call(**kw) == c["W4_ERR_" + code], kw


def _shared(lib, kv=None, q=OK16, qt=128 * 28, qh=128, group=OK16, shared=OK16, G=1, out=OK16, lse=None, hq=28, max_len=64,
            scale=0.1, scratch=OK16, sb=1 << 40):
    return lib.w4_attn_shared(kv if kv is not None else _kv(), q, qt, qh, group, shared, G, out, lse, hq, max_len, scale,
                              scratch, sb, None)


def test_shared_attention_refusals(w4):
    lib, c = w4.load(), _codes()
    for kw, code in ((dict(q=None), "NULL_PTR"), (dict(out=None), "NULL_PTR"), (dict(group=None), "NULL_PTR"),
                     (dict(shared=None), "NULL_PTR"), (dict(G=0), "INVALID_ARG"), (dict(hq=30), "INVALID_ARG"),
                     (dict(hq=4 * 129), "UNSUPPORTED_SHAPE"), (dict(scale=0.0), "INVALID_ARG"),
                     (dict(max_len=-1), "INVALID_ARG"), (dict(qt=0), "INVALID_ARG"), (dict(qh=0), "INVALID_ARG"),
                     (dict(qt=4), "MISALIGNED"), (dict(q=ODD), "MISALIGNED"), (dict(group=0x10002), "MISALIGNED"),
                     (dict(shared=0x10002), "MISALIGNED"), (dict(scratch=None), "WORKSPACE"),
                     (dict(scratch=0x10008), "MISALIGNED")):
        assert _shared(lib, **kw) == c["W4_ERR_" + code], kw
    for kw, code in ((dict(k=0), "NULL_PTR"), (dict(ps=48), "UNSUPPORTED_SHAPE"), (dict(d=96), "UNSUPPORTED_SHAPE"),
                     (dict(ks=132), "MISALIGNED"), (dict(maxp=0), "INVALID_ARG")):
        assert _shared(lib, _kv(**kw)) == c["W4_ERR_" + code], kw
    assert _shared(lib, _kv(batch=0), scratch=None) == c["W4_OK"]
    assert lib.w4_attn_shared_scratch_bytes(4, 30, 4, 128) == 0
    assert struct.calcsize("4Q7q6i") == 112


def test_shared_attention_counts_units_in_32_bits(w4):
    lib, c = w4.load(), _codes()
    kv = _kv(batch=1 << 14, maxp=1 << 20, ts=1 << 20)
    assert _shared(lib, kv, max_len=1 << 24) == c["W4_ERR_UNSUPPORTED_SHAPE"]


def test_shared_attention_takes_what_its_header_says(w4):
    """The largest launch that is taken (it goes on to ask for its scratch) and the first that is refused, by batch and by
    length, for one list item a key-value head and for several."""
    lib, c = w4.load(), _codes()
    taken, refused = c["W4_ERR_WORKSPACE"], c["W4_ERR_UNSUPPORTED_SHAPE"]
    for heads, hq, per in ((4, 28, 1), (4, 32, 1), (4, 36, 1), (2, 64, 2), (1, 128, 8), (1, 17, 2)):
        for n in (16, 4096, 1 << 20):
            most = (1 << 30) // (heads * per * (n // 16 + 8))
            for batch, want in ((most, taken), (most + 1, refused)):
                kv = _kv(heads=heads, batch=batch, maxp=1 << 20, ts=1 << 20)
                assert _shared(lib, kv, hq=hq, max_len=n, scratch=None) == want, (heads, hq, n, batch)
                kv = _kv(heads=heads, batch=batch, maxp=n // 16, ts=n // 16)      # the table is the bound
                assert _shared(lib, kv, hq=hq, max_len=1 << 30, scratch=None) == want, (heads, hq, n, batch)
        batch = 1 << 10
        most = 16 * ((1 << 20) // (heads * per) - 8) + 15
        for n, want in ((most, taken), (most + 1, refused)):
            kv = _kv(heads=heads, batch=batch, maxp=1 << 22, ts=1 << 22)
            assert _shared(lib, kv, hq=hq, max_len=n, scratch=None) == want, (heads, hq, n)
