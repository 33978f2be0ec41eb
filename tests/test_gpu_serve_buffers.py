"""Arguments of the calls of a serving step that are refused before anything is launched: a caller's own scratch in
memory of another kind, and sizes that do not fit in 32 bits, whose lower halves would be calls of other sizes."""
import pytest
import torch

from helpers import ensure_built
from test_gpu_attn_shared import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w4():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ensure_built()


def wrong(n):
    """(error, buffer of n bytes or more): on the host, of no tensor's kind, not in one piece, of one byte repeated."""
    gpu = torch.zeros(2 * n, dtype=torch.uint8, device="cuda")
    return ((TypeError, torch.zeros(n, dtype=torch.uint8)), (TypeError, bytearray(n)), (ValueError, gpu[::2]),
            (ValueError, gpu[:1].expand(n)), (ValueError, gpu.view(-1, 2)[:, 0]))


def test_shared_attention(w4):
    b = Batch([(40, [3, 1])], 4, 2, 64)
    want, _ = b.check(w4)
    n = w4.w4_attn_shared_scratch_bytes(2, 4, 2, 64)
    for error, scratch in wrong(n):
        with pytest.raises(error):
            w4.w4_attn_shared(*b.args(), scratch=scratch)
    for good in (torch.zeros(n, dtype=torch.uint8, device="cuda"), torch.zeros(-(-n // 4), device="cuda")):
        assert torch.equal(w4.w4_attn_shared(*b.args(), scratch=good), want)
    assert w4.w4_get_device_error() == 0


def test_routing(w4):
    z = torch.randn(100, 24, device="cuda")
    want = w4.w4_moe_route(z, 3)
    n = w4.w4_moe_route_workspace_bytes(100, 24)
    for error, workspace in wrong(n):
        with pytest.raises(error):
            w4.w4_moe_route(z, 3, workspace=workspace)
    got = w4.w4_moe_route(z, 3, workspace=torch.zeros(n, dtype=torch.uint8, device="cuda"))
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_sizes_past_32_bits(w4):
    """(Views of one row where the call takes them, else up to 9 GB that nothing writes.)"""
    far, bf = 1 << 32, torch.bfloat16
    one = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    row = torch.zeros(1, 8, dtype=bf, device="cuda")
    weight = torch.ones(1, 1, device="cuda")
    with pytest.raises(ValueError, match="32-bit"):
        w4.w4_moe_route(row.expand(far + 1, 8), 2)
    with pytest.raises(ValueError, match="32-bit"):
        w4.w4_moe_combine(torch.empty(far + 1, 1, dtype=bf, device="cuda"), one, weight)
    with pytest.raises(ValueError, match="32-bit"):
        w4.w4_moe_gather(torch.empty(1, 1, dtype=bf, device="cuda"), one, out=torch.empty(far + 1, 1, dtype=bf, device="cuda"))
    with pytest.raises(ValueError, match="32-bit"):
        w4.w4_moe_gather(torch.empty(1, far + 8, dtype=bf, device="cuda"), one)
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="32-bit"):
        w4.w4_kv_plan(lens, None, lens, lens, torch.empty(1, far // 2, dtype=torch.int32, device="cuda"), 16, 9, 1)
    torch.cuda.empty_cache()
