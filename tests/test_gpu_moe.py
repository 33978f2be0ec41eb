"""GPU parity of w4_moe_route, w4_moe_gather and w4_moe_combine against the float64 oracle.

The ids, rows and offsets have to be the oracle's exactly: scores that fp32 cannot tell apart are
compared in 64 bits.  Weights: the exponential's argument z - m is rounded to 2^-24 |z - m|, the
exponential and the quotient to 2^-22, the sums of at most 32 registers and 5 steps to 37 roundings:
2^-24 |z - m| + 2^-18.7 relative, of which the tests allow (2^-23 |z - m| + 2^-18)."""
import numpy as np
import pytest
import torch

from block_helpers import U, to64, within
from helpers import check_band, ensure_built, guarded_empty
from oracle import serve_oracle as SO

pytestmark = pytest.mark.gpu
NO_GROUPS = dict(groups=1, top=1, best=1)


@pytest.fixture(scope="module")
def w4():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ensure_built()


def guarded_route(w4, z, k, bias=None, score="softmax", groups=1, top=1, best=1, renorm=True, scale=1.0, count=None,
                  stream=None):
    """The C entry point with every output between guard bands."""
    T, E = z.shape
    outs = [guarded_empty(s, d) for s, d in (((T, k), torch.float32), ((T, k), torch.int32), ((T, k), torch.int32),
                                             ((E + 1,), torch.int32))]
    nbytes = w4.w4_moe_route_workspace_bytes(T, E)
    ws, raw = guarded_empty((max(nbytes, 16),), torch.uint8)
    rc = w4.load().w4_moe_route(z.data_ptr(), int(z.dtype is torch.bfloat16), z.stride(0),
                                None if bias is None else bias.data_ptr(), None if count is None else count.data_ptr(), T,
                                E, k, int(score == "sigmoid"), groups, top, best, int(renorm), scale,
                                *(o.data_ptr() for o, _ in outs), ws.data_ptr(), nbytes, None)
    assert rc == 0
    for (_, r), name in zip(outs + [(ws, raw)], ("weights", "ids", "row", "goff", "workspace")):
        check_band(r, name)
    return [o for o, _ in outs]


def same(got, want, z, what):
    """got: (weights, ids, row, goff) on the GPU; z the logits in float64."""
    w, ids, row, goff = (x.cpu().numpy() for x in got)
    ww, wi, wr, wg = want
    bad = np.nonzero((ids != wi).any(1))[0]
    assert not len(bad), (what, bad[:3], ids[bad[:3]], wi[bad[:3]])
    assert np.array_equal(row, wr) and np.array_equal(goff, wg), what
    fin = z[np.isfinite(z)]
    span = fin.max() - fin.min() if fin.size else 0.0
    assert np.isfinite(w).all()
    assert (np.abs(w - ww) <= (2.0 ** -23 * span + 2.0 ** -18) * np.abs(ww) + 1e-37).all(), what


def case(w4, T, E, k, bias=False, half=False, seed=0, count=None, **kw):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(T, E, generator=g) * 1.5 + torch.randn(E, generator=g) * 0.5
    z = (z.bfloat16() if half else z).cuda()
    b = (torch.randn(E, generator=g) * 0.05).cuda() if bias else None
    c = None if count is None else torch.tensor([count], dtype=torch.int32, device="cuda")
    got = guarded_route(w4, z, k, b, count=c, **kw)
    okw = {dict(top="top_groups").get(n, n): v for n, v in kw.items()}
    want = SO.route(to64(z), k, None if b is None else to64(b), count=count, **okw)
    same(got, want, to64(z), f"T {T} E {E} k {k} {kw}")
    api = {dict(top="top_groups", best="group_best").get(n, n): v for n, v in kw.items()}
    again = w4.w4_moe_route(z, k, bias=b, count=c, **api)
    assert all(torch.equal(x, y) for x, y in zip(got, again))


@pytest.mark.parametrize("T", [1, 2, 31, 33, 64, 65, 129, 1003, 5000])
@pytest.mark.parametrize("E,k", [(128, 8), (60, 6)])
def test_route_token_counts(w4, T, E, k):
    case(w4, T, E, k, bias=T % 2 == 1, half=T > 64, score="sigmoid" if T % 2 else "softmax", seed=T)


@pytest.mark.parametrize("E,k", [(1, 1), (2, 2), (8, 2), (31, 31), (32, 32), (33, 4), (64, 8), (65, 3), (129, 8), (256, 8),
                                 (257, 9), (384, 8), (512, 10), (513, 1), (1024, 32)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T", [37, 150])
def test_route_expert_counts(w4, E, k, score, T):
    case(w4, T, E, k, bias=True, score=score, seed=E, renorm=E % 2 == 0, scale=2.5)
    case(w4, T, E, k, half=True, score=score, seed=E + 1, renorm=E % 2 == 1)


@pytest.mark.parametrize("E,groups,top,k", [(64, 8, 3, 6), (256, 8, 4, 8), (160, 8, 3, 6), (60, 4, 2, 5), (96, 32, 5, 8),
                                            (32, 32, 8, 8), (1024, 2, 1, 8), (66, 3, 3, 4), (45, 9, 5, 20), (512, 16, 16, 8)])
@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("bias", [False, True])
def test_route_groups(w4, E, groups, top, k, best, bias):
    case(w4, 130, E, k, bias=bias, groups=groups, top=top, best=best, score="sigmoid", seed=E)
    case(w4, 50, E, k, bias=bias, groups=groups, top=top, best=best, score="softmax", seed=E + 1, half=True)


@pytest.mark.parametrize("count", [-5, 0, 1, 40, 99, 100, 1000])
@pytest.mark.parametrize("T", [50, 100])
def test_route_padding(w4, count, T):
    case(w4, T, 16, 2, count=count)


def test_route_scores_that_fp32_cannot_tell_apart(w4):
    """Biases that undo the scores: all sums lie within the rounding of one fp32 value, and the order is
    in the 64-bit digits; groups of such experts too."""
    g = torch.Generator().manual_seed(1)
    for E, groups, best in ((128, 1, 1), (256, 8, 2), (64, 4, 1)):
        row = torch.randn(E, generator=g)
        z = row.repeat(70, 1)
        bias = (0.75 - torch.sigmoid(row.double())).float()
        z[1::2] += 1e-6 * torch.randn(35, E, generator=g)
        got = guarded_route(w4, z.cuda(), 8, bias.cuda(), "sigmoid", groups, max(groups // 2, 1), best)
        want = SO.route(to64(z), 8, to64(bias), "sigmoid", groups, max(groups // 2, 1), best)
        s = 1 / (1 + np.exp(-to64(z))) + to64(bias)
        assert np.ptp(s) < 2e-6                    # the test is what it says
        same(got, want, to64(z), "near ties")


def test_route_equal_scores_go_to_the_lower_index(w4):
    z = torch.zeros(70, 96)
    z[1::2] = -0.0
    z[::3, 40:] = 1.0
    z[5, ::2] = -0.0                               # of both signs
    for kw in (dict(), dict(bias=torch.zeros(96)), dict(groups=8, top=3), dict(groups=8, top=3, best=2),
               dict(groups=8, top=3, best=2, bias=torch.full((96,), 0.25))):
        for score in ("softmax", "sigmoid"):
            b = kw.get("bias")
            rest = {n: v for n, v in kw.items() if n != "bias"}
            got = guarded_route(w4, z.cuda(), 10, None if b is None else b.cuda(), score, **rest)
            rest = {dict(top="top_groups").get(n, n): v for n, v in rest.items()}
            same(got, SO.route(to64(z), 10, None if b is None else to64(b), score, **rest), to64(z), (kw, score))


@pytest.mark.parametrize("E,groups,top,best", [(256, 8, 4, 2), (256, 8, 4, 1), (96, 1, 1, 1), (1024, 32, 7, 2)])
def test_route_rows_of_one_value(w4, E, groups, top, best):
    """Padded rows: one logit for all experts; alone, with one bias, with experts taken out, with one that differs by
    less than fp32 tells apart after the sigmoid, and with two values a group."""
    g = torch.Generator().manual_seed(E)
    z = torch.zeros(75, E)
    z[1::5] = -3.25
    z[2::5, torch.randperm(E, generator=g)[:E // 3]] = float("-inf")
    z[3::5, 40] = 2.0 ** -20
    z[4::5, ::2] = 1.5
    one = torch.full((E,), 0.375)
    most = one.clone()
    most[7] = float("-inf")
    other = one.clone()
    other[33] += 2.0 ** -22
    for b in (None, torch.zeros(E), one, most, other):
        for score in ("softmax", "sigmoid"):
            got = guarded_route(w4, z.cuda(), 8, None if b is None else b.cuda(), score, groups, top, best)
            want = SO.route(to64(z), 8, None if b is None else to64(b), score, groups, top, best)
            same(got, want, to64(z), f"E {E} groups {groups} best {best} {score}")


def test_route_masked_and_infinite_logits(w4):
    inf, nan = float("inf"), float("nan")
    g = torch.Generator().manual_seed(3)
    z = torch.randn(80, 40, generator=g)
    z[0] = -inf
    z[1] = nan
    z[2, 3:] = -inf                                # fewer than k left
    z[3, ::2] = nan
    z[4, 7] = inf
    z[5, [3, 30]] = inf
    z[6, 8:16] = -inf                              # a whole group
    z[7, 9:16] = -inf                              # one of a group left
    z[70] = -inf
    z[71, 20] = inf
    bias = torch.randn(40, generator=g) * 0.1
    bias[11] = -inf
    bias[12] = nan
    bias[33] = inf
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            for b in (None, bias):
                for kw in (dict(), dict(groups=5, top_groups=2, best=2), dict(groups=5, top_groups=3, best=1)):
                    mine = {dict(top_groups="top").get(n, n): v for n, v in kw.items()}
                    got = guarded_route(w4, z.cuda(), 6, None if b is None else b.cuda(), score, renorm=renorm, **mine)
                    want = SO.route(to64(z), 6, None if b is None else to64(b), score, renorm=renorm, **kw)
                    same(got, want, to64(z), (score, renorm, b is not None, kw))


def test_route_weights_that_underflow_together(w4):
    """Chosen experts far below the largest logit, or all far below zero."""
    z = torch.full((2, 64), -300.0)
    z[:, 0] = 0.0
    z[:, 5], z[:, 9], z[1, 0] = -200.0, -201.0, -400.0
    bias = torch.zeros(64)
    bias[[5, 9]] = 2.0
    bias[0] = -2.0
    for score in ("softmax", "sigmoid"):
        w, ids, _, _ = guarded_route(w4, z.cuda(), 2, bias.cuda(), score)
        assert ids.tolist() == [[5, 9], [5, 9]]
        want = 1 / (1 + np.exp(-1.0))
        assert np.allclose(w.cpu().numpy(), [[want, 1 - want]] * 2, rtol=2.0 ** -16)     # 2^-23 * 100 + 2^-18


def test_route_strides_and_streams(w4):
    g = torch.Generator().manual_seed(4)
    wide = torch.randn(90, 77, generator=g).cuda()
    z = wide[:, 3:63]
    want = SO.route(to64(z), 4)
    same(guarded_route(w4, z, 4), want, to64(z), "slice")
    half = wide.bfloat16()[:, 5:36]
    same(w4.w4_moe_route(half, 4), SO.route(to64(half), 4), to64(half), "bf16 slice")
    same(w4.w4_moe_route(wide[:1].expand(90, -1), 4), SO.route(to64(wide[:1].expand(90, -1)), 4), to64(wide), "one row")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = w4.w4_moe_route(z, 4, stream=side)
    side.synchronize()
    same(got, want, to64(z), "another stream")


def test_route_no_tokens_and_refusals(w4):
    w, ids, row, goff = w4.w4_moe_route(torch.zeros(0, 9, device="cuda"), 2)
    assert w.shape == ids.shape == row.shape == (0, 2) and goff.tolist() == [0] * 10
    z = torch.zeros(4, 8, device="cuda")
    with pytest.raises(ValueError):
        w4.w4_moe_route(z, 2, score="other")
    for bad in (dict(k=1 << 32), dict(k=1 << 30), dict(k=9), dict(k=0), dict(k=2, groups=0), dict(k=2, groups=9),
                dict(k=2, groups=-(1 << 33) + 1), dict(k=2, group_best=3), dict(k=2, top_groups=0)):
        with pytest.raises(ValueError):
            w4.w4_moe_route(z, **bad)
    with pytest.raises(TypeError):
        w4.w4_moe_route(z.half(), 2)
    with pytest.raises(TypeError):
        w4.w4_moe_route(z, 2, bias=torch.zeros(8, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        w4.w4_moe_route(z.t(), 2)
    for bad in (dict(k=2, groups=3), dict(k=2, top_groups=2), dict(k=3, groups=4)):
        with pytest.raises(w4.W4Error):
            w4.w4_moe_route(z, **bad)
    with pytest.raises(w4.W4Error):
        w4.w4_moe_route(z, 2, scale=float("inf"))
    with pytest.raises(w4.W4Error):
        w4.w4_moe_route(torch.zeros(65, 8, device="cuda"), 2, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))


# ------------------------------------------------------------------ to the experts and back
def rows_of(T, k, E=16, seed=0, drop=0.0):
    g = torch.Generator().manual_seed(seed)
    ids = torch.rand(T, max(E, k), generator=g).argsort(1)[:, :k]
    row = torch.empty(T * k, dtype=torch.int64)
    row[ids.flatten().argsort(stable=True)] = torch.arange(T * k)
    if drop:
        row[torch.rand(T * k, generator=g) < drop] = -1
    return row.int().view(T, k)


@pytest.mark.parametrize("K", [1, 7, 8, 12, 100, 256, 2048, 2049, 3580, 9000])
@pytest.mark.parametrize("T,k", [(1, 1), (5, 8), (67, 3), (300, 32)])
def test_gather(w4, K, T, k):
    g = torch.Generator().manual_seed(K)
    wide = torch.randn(T, K + 24, generator=g).bfloat16().cuda()
    row = rows_of(T, k, seed=K, drop=0.2)
    for x in (wide[:, :K].contiguous(), wide[:, 8:8 + K], wide[:, 3:3 + K]):
        out, raw = guarded_empty((T * k + 3, K), torch.bfloat16)
        out.fill_(-3.0)
        assert w4.w4_moe_gather(x, row.cuda(), out=out) is out
        check_band(raw, "out")
        want = torch.full((T * k + 3, K), -3.0, dtype=torch.bfloat16)
        for j in range(k):
            at = row[:, j] >= 0
            want[row[at, j].long()] = x.cpu()[at]
        assert torch.equal(out.cpu(), want)
    assert w4.w4_get_device_error() == 0


@pytest.mark.parametrize("N", [1, 7, 8, 12, 100, 256, 2048, 2049, 3580, 9000])
@pytest.mark.parametrize("T,k", [(1, 1), (5, 8), (67, 3), (40, 32)])
def test_combine(w4, N, T, k):
    """A sum of k + 1 terms in fp32 is off by (k + 1) 2^-24 of their sizes, then one bf16 rounding."""
    g = torch.Generator().manual_seed(N)
    y = torch.randn(T * k, N, generator=g).bfloat16().cuda()
    row = rows_of(T, k, seed=N, drop=0.2)
    w = torch.rand(T, k, generator=g)
    w[row < 0] = float("nan")                      # not read into the sum
    taken = row[row >= 0].long()
    unused = torch.ones(T * k, dtype=torch.bool)
    unused[taken] = False
    y[unused.cuda()] = float("nan")
    for shared in (None, torch.randn(T, N, generator=g).bfloat16().cuda()):
        out, raw = guarded_empty((T, N), torch.bfloat16)
        w4.w4_moe_combine(y, row.cuda(), w.cuda(), shared=shared, out=out)
        check_band(raw, "out")
        terms = np.where((row >= 0).numpy()[..., None], np.nan_to_num(w.numpy().astype(np.float64))[..., None] *
                         np.nan_to_num(to64(y))[row.clamp(min=0).long().numpy()], 0)
        ref, size = terms.sum(1), np.abs(terms).sum(1)
        if shared is not None:
            ref, size = ref + to64(shared), size + np.abs(to64(shared))
        within(out, ref, U * np.abs(ref) + (k + 2) * 2.0 ** -23 * size + 1e-38, f"N {N} T {T} k {k}")
    if T > 1:
        inplace = shared.clone()
        w4.w4_moe_combine(y, row.cuda(), w.cuda(), shared=inplace, out=inplace)
        assert torch.equal(inplace, out)
    assert w4.w4_get_device_error() == 0


def test_visible_infinities_reach_the_sum(w4):
    y = torch.zeros(2, 8, dtype=torch.bfloat16, device="cuda")
    y[0, 1], y[1, 2] = float("inf"), float("nan")
    row = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
    out = w4.w4_moe_combine(y, row, torch.full((1, 2), 0.5, device="cuda"))
    assert out[0, 1] == float("inf") and out[0, 2].isnan() and not out[0, [0, 3, 4, 5, 6, 7]].any()


def test_rows_out_of_range_are_skipped_and_flagged(w4):
    x = torch.ones(2, 16, dtype=torch.bfloat16, device="cuda")
    for bad in (4, -2, 1 << 30, -(1 << 31)):
        row = torch.tensor([[0, bad], [1, -1]], dtype=torch.int32, device="cuda")
        out, raw = guarded_empty((4, 16), torch.bfloat16)
        out.fill_(-3.0)
        w4.w4_moe_gather(x, row, out=out)
        check_band(raw, "out")
        assert (out[:2] == 1).all() and (out[2:] == -3).all() and w4.w4_get_device_error() == -11
        y = w4.w4_moe_combine(out, row, torch.ones(2, 2, device="cuda"))
        assert (y == 1).all() and w4.w4_get_device_error() == -11


def test_rows_past_two_to_the_31_values(w4):
    """A buffer of 2.4e9 values (4.8 GB): rows at its end."""
    R, K = 60000, 40000
    x = torch.randn(3, K, generator=torch.Generator().manual_seed(0)).bfloat16().cuda()
    out = torch.zeros(R, K, dtype=torch.bfloat16, device="cuda")
    row = torch.tensor([[R - 1, 0], [53700, R - 2], [-1, 53686]], dtype=torch.int32, device="cuda")
    w4.w4_moe_gather(x, row, out=out)
    assert torch.equal(out[[R - 1, 0, 53700, R - 2, 53686]], x[[0, 0, 1, 1, 2]])
    assert int(out.any(1).sum()) == 5
    back = w4.w4_moe_combine(out, row, torch.tensor([[0.5, 0.25]] * 3, device="cuda"))
    want = x.float() * torch.tensor([0.75, 0.75, 0.25], device="cuda")[:, None]
    assert (back.float() - want).abs().le(2.0 ** -8 * want.abs()).all() and w4.w4_get_device_error() == 0


def test_move_shapes_without_work(w4):
    row = torch.zeros(0, 3, dtype=torch.int32, device="cuda")
    assert w4.w4_moe_gather(torch.zeros(0, 8, dtype=torch.bfloat16, device="cuda"), row).shape == (0, 8)
    assert w4.w4_moe_combine(torch.zeros(0, 8, dtype=torch.bfloat16, device="cuda"), row,
                             torch.zeros(0, 3, device="cuda")).shape == (0, 8)
    none = torch.full((2, 3), -1, dtype=torch.int32, device="cuda")
    y = w4.w4_moe_combine(torch.zeros(0, 8, dtype=torch.bfloat16, device="cuda"), none, torch.ones(2, 3, device="cuda"))
    assert not y.any() and y.shape == (2, 8)
    with pytest.raises(ValueError):
        w4.w4_moe_gather(torch.zeros(3, 8, dtype=torch.bfloat16, device="cuda"), none)
    with pytest.raises(ValueError):
        w4.w4_moe_combine(torch.zeros(6, 8, dtype=torch.bfloat16, device="cuda"), none, torch.ones(2, 2, device="cuda"))


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("T", [13, 200])
@pytest.mark.usefixtures("w4")
def test_route_to_combine_around_the_grouped_linear(T):
    """The whole expert layer, eager and in a captured graph whose inputs change, against one dequantized
    matrix product a token.  Bounds: the grouped linear's own bar (5e-3 in the norm) and two roundings."""
    import int4_weight_only_gb300 as w4             # without guard bands, whose checks synchronize
    from oracle import w4_oracle as O
    E, k, K, N, G = 16, 4, 256, 192, 32
    g = torch.Generator().manual_seed(T)
    W = torch.randn(E * N, K, generator=g) * 0.05
    p, s, _ = w4.w4_pack_rtn(W.cuda(), G, True)
    What = O.dequantize_f64(p.cpu().numpy(), s.cpu().numpy(), None, G).reshape(E, N, K)
    bias = (torch.randn(E, generator=g) * 0.05).cuda()
    x = torch.empty(T, K, dtype=torch.bfloat16, device="cuda")
    z = torch.empty(T, E, dtype=torch.float32, device="cuda")

    def layer():
        w, ids, row, goff = w4.w4_moe_route(z, k, bias=bias, score="sigmoid", groups=4, top_groups=2, group_best=2)
        y = w4.w4a16_grouped_linear(w4.w4_moe_gather(x, row), goff, p, s, None, None, E, N, K, G, 16)
        return w4.w4_moe_combine(y, row, w, shared=x[:, :N].contiguous())

    def fill(seed):
        g = torch.Generator().manual_seed(seed)
        x.copy_(torch.randn(T, K, generator=g))
        z.copy_(torch.randn(T, E, generator=g))

    def check(out):
        w, ids, _, _ = SO.route(to64(z), k, to64(bias), "sigmoid", 4, 2, 2)
        xs = to64(x)
        ref = xs[:, :N].copy()
        for t in range(T):
            for j in range(k):
                ref[t] += w[t, j] * (What[ids[t, j]] @ xs[t])
        d = to64(out) - ref
        assert np.linalg.norm(d) <= 5e-3 * np.linalg.norm(ref)
    fill(1)
    check(layer())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = layer()
    for seed in (2, 3, 4):
        fill(seed)
        graph.replay()
        check(out)
    first = out.clone()
    graph.replay()
    assert torch.equal(out, first) and w4.w4_get_device_error() == 0


@pytest.mark.parametrize("T,count,tile", [(20, 13, 4), (20, 0, 16), (300, 211, 64), (300, 1, 256), (300, 300, 16)])
def test_padding_through_the_grouped_linear(w4, T, count, tile):
    """Tokens behind `count` have no rows: the grouped linear's offsets end before its rows do, the rows behind stay as
    they were (NaN), and nothing of them comes back."""
    E, k, K, N, G = 8, 3, 128, 96, 32
    g = torch.Generator().manual_seed(T + count)
    p, s, _ = w4.w4_pack_rtn((torch.randn(E * N, K, generator=g) * 0.05).cuda(), G, True)
    x = torch.randn(T, K, generator=g).bfloat16().cuda()
    z = torch.randn(T, E, generator=g).cuda()
    shared = torch.randn(T, N, generator=g).bfloat16().cuda()
    w, ids, row, goff = w4.w4_moe_route(z, k, count=torch.tensor([count], dtype=torch.int32, device="cuda"))
    xs = torch.full((T * k, K), float("nan"), dtype=torch.bfloat16, device="cuda")
    w4.w4_moe_gather(x, row, out=xs)
    y = torch.full((T * k, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    w4.w4a16_grouped_linear(xs, goff, p, s, None, None, E, N, K, G, tile, y=y)
    assert goff[-1] == count * k and y[count * k:].isnan().all() and torch.isfinite(y[:count * k].float()).all()
    out = w4.w4_moe_combine(y, row, w, shared=shared)
    assert torch.equal(out[count:], shared[count:]) and torch.isfinite(out.float()).all()
    full = w4.w4_moe_route(z[:count], k) if count else None
    if full:
        assert torch.equal(full[1], ids[:count]) and torch.equal(full[2], row[:count]) and torch.equal(full[3], goff)
    assert w4.w4_get_device_error() == 0
