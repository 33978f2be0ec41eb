"""w4_moe_route over more tokens than one run of the order's kernel a CTA holds (128 on each of 152), and the rows of
buffers without rows."""
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


@pytest.mark.parametrize("T,E,k,count", [(19456, 16, 2, None), (19457, 60, 6, None), (25000, 60, 6, 24000),
                                         (39000, 33, 5, None), (60001, 9, 9, 59000), (25000, 60, 6, 100)])
def test_later_runs_of_the_order(w4, T, E, k, count):
    g = torch.Generator().manual_seed(T)
    z = (torch.randn(T, E, generator=g) + torch.randn(E, generator=g)).bfloat16()
    z[7::11] = float("-inf")                      # tokens without an expert, and with few
    z[5::13, 1:] = float("-inf")
    c = None if count is None else torch.tensor([count], dtype=torch.int32, device="cuda")
    got = guarded_route(w4, z.cuda(), k, count=c)
    same(got, SO.route(to64(z), k, count=count), to64(z), f"T {T} E {E} k {k}")


@pytest.mark.parametrize("K", [8, 2, 7])
def test_rows_to_and_from_a_buffer_without_rows(w4, K):
    """Every place is -1: nothing is copied, the sum is the shared row; any other place is flagged."""
    x = torch.ones(3, K, dtype=torch.bfloat16, device="cuda")
    none = torch.full((3, 2), -1, dtype=torch.int32, device="cuda")
    empty = torch.empty(0, K, dtype=torch.bfloat16, device="cuda")
    assert w4.w4_moe_gather(x, none, out=empty) is empty
    assert torch.equal(w4.w4_moe_combine(empty, none, torch.ones(3, 2, device="cuda"), shared=x), x)
    assert w4.w4_get_device_error() == 0
    none[1, 1] = 0
    w4.w4_moe_gather(x, none, out=empty)
    assert w4.w4_get_device_error() == -11
