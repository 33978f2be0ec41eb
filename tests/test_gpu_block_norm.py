"""GPU parity of w4_block_norm against the float64 oracle.

Bounds: a bf16 output is one rounding (2^-8 of its value) of an fp32 result.
The fp32 result itself is off by a few 2^-24 per product, plus the row sum:
K <= 32768 terms added as at most 32 + 5 + 32 partial sums in sequence, under
2^-17 of the norm.  r' can cancel, so its fp32 error is taken against the size
of its terms (2^-21, from the norm of y and three products)."""
import numpy as np
import pytest
import torch

from block_helpers import U, randn_bf16, to64, within
from helpers import ensure_built, guarded_empty, check_band
from oracle import block_oracle as BO

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w4():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ensure_built()


def run(w4, M, K, post, gate, a=1.0, off=0.0, eps=1e-6, seed=0, y_scale=0.7, offset=0):
    y, r = randn_bf16(M, K, seed=seed, scale=y_scale), randn_bf16(M, K, seed=seed + 1, scale=2.0)
    wpre = (1 - off + randn_bf16(K, seed=seed + 2, scale=0.2)).bfloat16()
    wpost = (1 - off + randn_bf16(K, seed=seed + 3, scale=0.2)).bfloat16() if post else None
    g = randn_bf16(gate, K, seed=seed + 4) if gate else None

    def dev(t):             # on the GPU, `offset` elements past an allocation's start
        if t is None:
            return None
        buf = torch.empty(t.numel() + offset, dtype=t.dtype, device="cuda")
        out = buf[offset:].view(t.shape)
        out.copy_(t)
        return out
    ro, raw_r = guarded_empty((M, K), torch.bfloat16)
    xo, raw_x = guarded_empty((M, K), torch.bfloat16)
    got_r, got_x = w4.w4_block_norm(dev(y), dev(r), dev(wpre), dev(wpost), dev(g), a, eps, off, r_out=ro, x_out=xo)
    check_band(raw_r, "r_out")
    check_band(raw_x, "x_out")
    wr, wx, size = BO.block_norm(to64(y), to64(r), to64(wpre), None if wpost is None else to64(wpost),
                                 None if g is None else to64(g), a, eps, off)
    within(got_r, wr, U * np.abs(wr) + 2.0 ** -17 * size, f"r' {M}x{K}")
    wmag = np.abs(off + to64(wpre)) / np.sqrt((wr * wr).mean(1, keepdims=True) + eps)
    within(got_x, wx, (U + 2.0 ** -16) * np.abs(wx) + 2.0 ** -17 * size * wmag, f"x {M}x{K}")
    return got_r, got_x


@pytest.mark.parametrize("M,K", [(1, 1), (2, 7), (1, 8), (3, 100), (5, 257), (7, 3580), (1, 3584), (16, 3584),
                                 (33, 3840), (4, 4096), (3, 4104), (2, 8191), (2, 8192), (5, 16384), (2, 20001),
                                 (2, 32768), (1, 32767), (1500, 520)])
@pytest.mark.parametrize("post,gate,a,off", [(False, 0, 1.0, 0.0), (True, 1, 0.25, 1.0)])
def test_sizes(w4, M, K, post, gate, a, off):
    run(w4, M, K, post, gate, a, off, seed=M + K)


@pytest.mark.parametrize("gate", [0, 1, 3, 12])
@pytest.mark.parametrize("post", [False, True])
def test_gate_rows(w4, post, gate):
    run(w4, 12, 264, post, gate, -1.5)


@pytest.mark.parametrize("offset", [1, 2, 4])
@pytest.mark.parametrize("K", [64, 1000])
def test_unaligned_buffers(w4, K, offset):
    run(w4, 5, K, True, 5, 0.5, offset=offset)


def test_no_pre_norm_and_no_block(w4):
    r = randn_bf16(9, 640, seed=1).cuda()
    y, wpost = randn_bf16(9, 640, seed=2).cuda(), randn_bf16(640, seed=3).cuda()
    got, x = w4.w4_block_norm(y, r, None, wpost)
    assert x is None
    want, _, size = BO.block_norm(to64(y), to64(r), None, to64(wpost))
    within(got, want, U * np.abs(want) + 2.0 ** -17 * size)
    got, x = w4.w4_block_norm(None, r, wpost)
    assert got is r
    _, want, _ = BO.block_norm(None, to64(r), to64(wpost))
    within(x, want, (U + 2.0 ** -16) * np.abs(want))


def test_in_place(w4):
    """r_out may be r (and x_out y): the same bits as out of place."""
    for K in (3584, 101):
        y, r = randn_bf16(6, K, seed=1).cuda(), randn_bf16(6, K, seed=2).cuda()
        w, p = randn_bf16(K, seed=3).cuda(), randn_bf16(K, seed=4).cuda()
        want = w4.w4_block_norm(y, r, w, p)
        y2, r2 = y.clone(), r.clone()
        w4.w4_block_norm(y2, r2, w, p, r_out=r2, x_out=y2)
        assert torch.equal(r2, want[0]) and torch.equal(y2, want[1])


def test_extreme_values(w4):
    """A zero row normalizes to zero, large and tiny rows keep their norm, and
    NaN or infinity stays in its own row."""
    K = 512
    r = randn_bf16(6, K, seed=5)
    r[0] = 0
    r[1] *= 1e15
    r[2] *= 1e-12
    r[3, 7] = float("nan")
    r[4, 9] = float("inf")
    w = torch.ones(K).bfloat16()
    _, x = w4.w4_block_norm(None, r.cuda(), w.cuda(), eps=1e-30)
    x = to64(x)
    _, want, _ = BO.block_norm(None, to64(r), to64(w), eps=1e-30)
    assert not x[0].any()
    ok = [1, 2, 5]
    within(x[ok], want[ok], (U + 2.0 ** -16) * np.abs(want[ok]))
    assert np.isnan(x[3]).all()
    assert np.isnan(x[4, 9]) and not x[4, :9].any()


def test_rows_do_not_depend_on_the_batch(w4):
    y, r = randn_bf16(700, 3584, seed=1).cuda(), randn_bf16(700, 3584, seed=2).cuda()
    w = randn_bf16(3584, seed=3).cuda()
    a, b = w4.w4_block_norm(y, r, w, w), w4.w4_block_norm(y[5:6].contiguous(), r[5:6].contiguous(), w, w)
    assert torch.equal(a[0][5:6], b[0]) and torch.equal(a[1][5:6], b[1])


def test_binding_refusals(w4):
    r = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(TypeError):
        w4.w4_block_norm(r.float(), r, w)
    with pytest.raises(ValueError):
        w4.w4_block_norm(r[:3], r, w)
    with pytest.raises(ValueError):
        w4.w4_block_norm(r, r, w[:32])
    with pytest.raises(ValueError):
        w4.w4_block_norm(r.t().contiguous().t(), r, w)
    with pytest.raises(w4.W4Error):
        w4.w4_block_norm(r, r, w, gate=r[:3].contiguous())
    e = r[:0]
    assert w4.w4_block_norm(e, e, w)[1].shape == (0, 64)


def test_a_gate_without_rows_is_refused(w4):
    """Its pointer is null, which means no gate: it must not be taken for one."""
    r = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        w4.w4_block_norm(r, r, w, gate=r[:0])
    e = r[:0]
    assert w4.w4_block_norm(e, e, w, gate=e)[1].shape == (0, 64)
