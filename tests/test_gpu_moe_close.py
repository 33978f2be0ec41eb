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
