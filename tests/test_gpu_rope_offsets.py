"""Token offsets out of range or decreasing raise the device flag, also where
no row belongs to the sequence that has them."""
import pytest
import torch

from block_helpers import Paged, randn_bf16
from helpers import ensure_built

pytestmark = pytest.mark.gpu
ROWS_ERR = -11


@pytest.fixture(scope="module")
def w4():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ensure_built()


def run(w4, T, goff):
    cache = Paged([20] * (len(goff) - 1), 2, 64, 16, fill=0.0)
    q, k, v = (randn_bf16(T, h, 64, seed=h).cuda() for h in (4, 2, 2))
    w4.w4_rope_append(q, k, v, cache.k, cache.v, cache.kv_len, cache.table, w4.w4_rope_freqs(64)[0].cuda(),
                      goff=torch.tensor(goff, dtype=torch.int32, device="cuda"))
    return w4.w4_get_device_error()


@pytest.mark.parametrize("T,goff", [
    (8, [0, 5, 3, 8]), (3, [0, 9]), (3, [-1, 3]), (3, [2, 1]), (3, [0, 3, 4]), (3, [0, 1, 3, 2]), (1, [0, 1, -7, 1]),
    (5, [0] * 20 + [4, 2] + [5] * 60), (2, [0, 1, 2] + [2] * 90 + [1, 2]), (40, list(range(41)) + [39]),
    (5, [0, 5] + [5] * 300 + [6])])
def test_bad_offsets_raise_the_flag(w4, T, goff):
    assert run(w4, T, goff) == ROWS_ERR


@pytest.mark.parametrize("T,goff", [(8, [0, 5, 5, 8]), (3, [1, 2]), (3, [0, 0, 0]), (2, [0, 1] + [2] * 200),
                                    (40, list(range(41)))])
def test_good_offsets_do_not(w4, T, goff):
    assert run(w4, T, goff) == 0
