"""w4_moe_route where fp32 cannot tell scores or groups apart: rows with a few close candidates and the rest far
off, ranks that are equal, tiny or out of fp32's range.  Ids, rows and offsets have to be the float64 oracle's."""
import numpy as np
import pytest
import torch

from block_helpers import to64
from helpers import ensure_built
from oracle import serve_oracle as SO
from test_gpu_moe import guarded_route, same

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w4():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ensure_built()


def check(w4, z, k, bias=None, score="sigmoid", groups=1, top=1, best=1, what="", **kw):
    got = guarded_route(w4, z.cuda(), k, None if bias is None else bias.cuda(), score, groups, top, best, **kw)
    want = SO.route(to64(z), k, None if bias is None else to64(bias), score, groups, top, best, **kw)
    same(got, want, to64(z), what)
    return want


def probabilities(z, score, dtype):
    z = z.astype(dtype)
    if score == "sigmoid":
        return 1 / (1 + np.exp(-z))
    e = np.exp(z - z.max(1, keepdims=True))
    return e / e.sum(1, keepdims=True)


def logits_of(p, score):
    return np.log(p / (1 - p)) if score == "sigmoid" else np.log(p)


def close_rows(E, k, above, n, rows, score, seed):
    """Logits and a bias that cancels the scores of n experts to within fp32's rounding at a height T; `above` experts
    clearly over them, the others clearly under.  Returns (z, bias, how many scores lie at T)."""
    r = np.random.default_rng(seed)
    perm = r.permutation(E)
    C, A, R = perm[:n], perm[n:n + above], perm[n + above:]
    T, unit = (0.8, 0.5) if score == "sigmoid" else (4.0 / E, 0.5 / E)
    p = np.empty((rows, E))
    p[:, C] = unit * r.uniform(0.6, 1.4, n) * (1 + 8e-8 * r.standard_normal((rows, n)))
    for t in range(rows):
        p[t, A] = unit * (0.8 + 0.02 * r.permutation(above))
        p[t, R] = unit * (0.1 + 0.8 * r.permutation(E - n - above) / E)
    if score == "softmax":
        p /= p.sum(1, keepdims=True)
    z = logits_of(p, score).astype(np.float32)
    exact = probabilities(z, score, np.float64)
    bias = np.zeros(E, np.float32)
    bias[C] = (T - exact[:, C].mean(0)).astype(np.float32)
    bias[A] = np.float32(T)                       # T + unit * 0.8 and more
    s = exact + bias.astype(np.float64)
    near = np.abs(s - T) < 4e-6 * unit / 0.5
    assert (near.sum(1) == n).all() and (np.abs(s - T)[~near] > 0.02 * unit).all()
    return torch.tensor(z), torch.tensor(bias), s, C


def fp32_order_differs(z, bias, score, k):
    """Rows whose choice in plain fp32 is not that of 64 bits."""
    def order(dtype):
        s = probabilities(z.numpy(), score, dtype) + bias.numpy().astype(dtype)
        return np.argsort(-s, axis=1, kind="stable")[:, :k]
    return (order(np.float32) != order(np.float64)).any(1)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,k,above,n", [(64, 8, 0, 2), (64, 8, 6, 3), (128, 8, 4, 5), (128, 6, 5, 12), (256, 8, 7, 20),
                                         (60, 4, 3, 2), (384, 8, 2, 9), (1024, 32, 20, 12), (33, 32, 0, 20)])
def test_a_few_close_candidates(w4, E, k, above, n, score):
    """They are chosen, or the last place is among them; the fp32 order is wrong in many rows."""
    z, bias, s, C = close_rows(E, k, above, n, 150, score, E + n)
    assert fp32_order_differs(z, bias, score, k).any()
    for rows in (150, 40):
        check(w4, z[:rows], k, bias, score, what=f"E {E} k {k} {above} above {n} close {score}")


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("above,n", [(0, 31), (0, 32), (0, 33), (4, 27), (4, 28), (4, 29), (7, 25), (7, 26)])
def test_as_many_candidates_as_lanes(w4, above, n, score):
    """k + n - (k - above) of them: 31, 32 and 33 for the last place and all behind it."""
    z, bias, s, C = close_rows(256, 8, above, n, 90, score, above * 40 + n)
    assert fp32_order_differs(z, bias, score, 8).any()
    check(w4, z, 8, bias, score, what=f"{above} above {n} close {score}")


def close_groups(E, G, above, near, rows, score, with_bias, seed, spread):
    """Logits and a bias whose sums of two scores differ by about `spread` between the border groups (near[i] experts at
    the second score or within its rounding); `above` groups lie over them, the others under."""
    r = np.random.default_rng(seed)
    gs, border = E // G, len(near)
    unit = 0.5 if score == "sigmoid" else 1.0 / E
    s = np.tile(unit * (0.05 + 0.05 * r.random(E)), (rows, 1))
    for i, g in enumerate(r.permutation(G)):
        at = g * gs + r.permutation(gs)
        if i < border:
            one, two, m = 1.4, 1.0, near[i] - 1
        elif i < border + above:
            one, two, m = 1.6 + 0.01 * i, 1.2 + 0.01 * i, 1
        else:
            one, two, m = 0.8 - 0.01 * i, 0.5 - 0.005 * i, 1
        s[:, at[0]] = unit * one * (1 + spread * r.standard_normal(rows))
        s[:, at[1:1 + m]] = unit * two * (1 + spread * r.standard_normal((rows, m)))
    bias = (unit * r.uniform(-0.04, 0.04, E) * with_bias).astype(np.float32)
    p = s - bias
    if score == "softmax":                        # of a sum of one
        bias, p = (bias / p.sum(1).mean()).astype(np.float32), p / p.sum(1).mean()
    z = logits_of(p, score).astype(np.float32)
    return torch.tensor(z), torch.tensor(bias) if with_bias else None


def group_sums(z, bias, score, G, dtype):
    s = probabilities(z.numpy(), score, dtype)
    if bias is not None:
        s = s + bias.numpy().astype(dtype)
    top = -np.sort(-s.reshape(len(s), G, -1), axis=2)[..., :2]
    return top[..., 0] + top[..., 1], top[..., 1], s


def border_differs(z, bias, score, G, top):
    """Rows in which plain fp32 keeps other groups than 64 bits; and each row's experts that can be among the best two of
    a group within 2e-6 of the border."""
    kept = []
    for dtype in (np.float32, np.float64):
        rank, second, s = group_sums(z, bias, score, G, dtype)
        order = np.argsort(-rank, axis=1, kind="stable")[:, :top]
        kept.append(np.sort(order, axis=1))
    last = -np.sort(-rank, axis=1)[:, top - 1:top]
    scale = s.max(1, keepdims=True)
    open_ = np.abs(rank - last) < 6e-6 * scale
    cand = (s.reshape(len(s), G, -1) > (second - 4e-6 * scale)[..., None]) & open_[..., None]
    return (kept[0] != kept[1]).any(1), cand.sum((1, 2))


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("E,G,top,above,near,k", [(64, 8, 4, 3, [2, 2], 6), (256, 8, 4, 2, [2, 3, 2, 4], 8),
                                                  (128, 4, 2, 1, [2, 2, 5], 4), (96, 32, 9, 7, [2, 2, 2, 3], 8),
                                                  (512, 8, 2, 0, [3, 4, 2], 4)])
def test_a_few_close_groups(w4, E, G, top, above, near, k, bias, score):
    z, b = close_groups(E, G, above, near, 150, score, bias, E + top, 1.5e-7)
    wrong, cand = border_differs(z, b, score, G, top)
    assert wrong.any() and np.mean(cand <= 32) > 0.9 and np.mean(cand >= 4) > 0.9
    for rows in (150, 40):
        check(w4, z[:rows], k, b, score, G, top, 2, what=f"E {E} {G} groups {near} {score} bias {bias}")


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,G,top,above,near,k", [(64, 8, 4, 3, [2, 2], 6), (256, 8, 4, 2, [2, 3, 2, 4], 8),
                                                  (96, 32, 9, 7, [2, 2, 2, 3], 8)])
def test_a_few_close_groups_by_their_best(w4, E, G, top, above, near, k, score):
    """Ranked by one biased score, of which the border groups' lie within an fp32 rounding."""
    z, b = close_groups(E, G, above, near, 150, score, True, E + top, 1e-7)
    kept = []
    for dtype in (np.float32, np.float64):
        s = probabilities(z.numpy(), score, dtype) + b.numpy().astype(dtype)
        kept.append(np.sort(np.argsort(-s.reshape(150, G, -1).max(2), axis=1, kind="stable")[:, :top], axis=1))
    # (of two border groups, the host's fp32 exponential happens to order all rows on some machines)
    assert len(near) == 2 or (kept[0] != kept[1]).any()
    for rows in (150, 40):
        check(w4, z[:rows], k, b, score, G, top, 1, what=f"E {E} {G} groups {near} {score}")


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("near", [[8, 8, 8, 7], [8, 8, 8, 8], [8, 8, 8, 9]])
def test_as_many_candidates_of_close_groups_as_lanes(w4, near, score):
    z, b = close_groups(256, 8, 2, near, 120, score, False, sum(near), 1.5e-7)
    wrong, cand = border_differs(z, b, score, 8, 4)
    assert wrong.any() and np.mean(cand == sum(near)) > 0.9
    check(w4, z, 8, b, score, 8, 4, 2, what=f"{near} {score}")


@pytest.mark.parametrize("E,G,top", [(32, 4, 2), (256, 8, 3), (96, 32, 20)])
def test_groups_that_offer_one_expert_and_two(w4, E, G, top):
    """Alike logits and biases are no tie where one group ranks by one score and another by the sum of two, however
    near to zero the scores are."""
    gs = E // G
    rows = []
    for x in (-100.0, -60.0, -17.5, 0.0, 0.3, 1.0, -0.7):
        for alone in ((0,), (1,), (0, 2), (G - 1,), tuple(range(1, G))):
            row = torch.full((E,), x)
            for g in alone:
                row[g * gs:(g + 1) * gs] = float("-inf")
                row[g * gs + (g + 1) % gs] = x
            rows.append(row)
    z = torch.stack(rows + rows)
    biases = [None, torch.zeros(E)]
    for x in (0.0, 0.3, 1.0, -0.7):               # p + bias is what the rounding of the bias leaves
        biases.append(torch.full((E,), -float(np.float32(1 / (1 + np.exp(-np.float64(np.float32(x))))))))
    for b in biases:
        for score in ("sigmoid", "softmax"):
            check(w4, z, 6, b, score, G, top, 2, what=f"E {E} {score}")


def test_ranks_out_of_range_of_fp32(w4):
    """Sums of two scores beyond the largest fp32 value of either sign: biases of the type's lowest value take experts
    out as far as anything else is left, and large ones are compared as what they are."""
    low, big = torch.finfo(torch.float32).min, 3.0e38
    g = torch.Generator().manual_seed(0)
    z = torch.randn(80, 32, generator=g)
    z[::2, :8] = float("-inf")                    # nothing offered in group 0
    masked = torch.zeros(32)
    masked[8:24] = low                            # groups 1 and 2
    check(w4, z, 12, masked, "sigmoid", 4, 2, 2, what="lowest")
    check(w4, z, 12, masked, "softmax", 4, 3, 2, what="lowest")
    up = torch.zeros(32)
    up[[9, 10]], up[[17, 18]], up[[25, 26]] = big, 3.2e38, 3.1e38
    for top in (1, 2, 3):
        check(w4, z, 4, up, "sigmoid", 4, top, 2, what=f"large, {top}")
    up[[10, 20]] = float("inf")
    for top in (1, 2):
        check(w4, z, 4, up, "sigmoid", 4, top, 2, what=f"infinite, {top}")
        check(w4, z, 4, up, "sigmoid", 4, top, 1, what=f"infinite, by one, {top}")


@pytest.mark.parametrize("off", [-1e4, -1e9, torch.finfo(torch.float32).min])
@pytest.mark.parametrize("best", [1, 2])
def test_experts_switched_off_by_a_finite_bias(w4, off, best):
    g = torch.Generator().manual_seed(5)
    z = torch.randn(140, 256, generator=g)
    b = torch.randn(256, generator=g) * 0.05
    b[[3, 77, 78, 200]] = off
    b[32:64] = off                                # a whole group
    for score in ("sigmoid", "softmax"):
        check(w4, z, 8, b, score, 8, 4, best, what=f"{off} {score}")
    check(w4, z, 8, b, "sigmoid", what=f"{off}")
    check(w4, z, 20, b, "sigmoid", 8, 8, best, what=f"{off}")


def test_small_scores_in_groups(w4):
    g = torch.Generator().manual_seed(6)
    for shift in (-15.0, -40.0, -86.0):
        z = torch.randn(140, 256, generator=g) + shift
        check(w4, z, 8, None, "sigmoid", 8, 4, 2, what=f"{shift}")
        check(w4, z, 8, torch.randn(256, generator=g) * 1e-7, "sigmoid", 8, 4, 2, what=f"{shift} biased")


def test_masks_and_small_scores_cost_no_second_choice(w4):
    """A token that has to be chosen in 64 bits altogether takes 20 times as long as one that has not.  A mask in the bias, or
    scores that are all small, must not send every token there: the time stays within four times that of plain ones."""
    g = torch.Generator().manual_seed(7)
    z = torch.randn(8192, 256, generator=g).cuda()
    b = (torch.randn(256, generator=g) * 0.05).cuda()

    def us(z, b):
        def call():
            w4.w4_moe_route(z, 8, bias=b, score="sigmoid", groups=8, top_groups=4, group_best=2)
        times = []
        for _ in range(6):
            start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            start.record()
            for _ in range(10):
                call()
            end.record()
            end.synchronize()
            times.append(start.elapsed_time(end))
        return min(times[1:])
    plain = us(z, b)
    for off in (-1e4, -1e9, torch.finfo(torch.float32).min):
        masked = b.clone()
        masked[[3, 77]] = off
        assert us(z, masked) < 4 * plain, off
    assert us(z - 40.0, None) < 4 * us(z, None)


def test_scores_below_the_normal_range(w4):
    """Scores that the approximate exponential flushes to zero against biases of their size."""
    z = torch.full((70, 16), -1000.0)
    bias = torch.zeros(16)
    bias[3] = 3e-39
    z[:, 5] = -88.0                               # p = 6.1e-39
    z[1::2, 9] = -88.5                            # 3.7e-39
    want = check(w4, z, 3, bias, what="flushed")
    assert want[1][0, :2].tolist() == [5, 3] and want[1][1].tolist() == [5, 9, 3]
    check(w4, z, 3, bias, "sigmoid", 4, 2, 2, what="flushed, in groups")
