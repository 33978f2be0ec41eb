"""The serving step of examples/moe_block.py row by row: attention with and without sharing on the same inputs at every
step, and every hidden row whose experts are the same in both runs (none is left out for being far off)."""
import pytest
import torch

from block_helpers import U
from test_gpu_moe_block import CONFIGS, RMS, ex, serve  # noqa: F401

pytestmark = pytest.mark.gpu
OWN = [0, 5, 33, 1, 0, 17]


@pytest.mark.parametrize("cfg", CONFIGS)
@pytest.mark.parametrize("n", [64, 150, 700])
def test_attention_of_every_step(ex, cfg, n, monkeypatch):  # noqa: F811
    """Each form is within U |o| + e sum w |v| of the exact output, e = 2^-8 + 2^-11 with sharing (weights rounded to
    bf16) and 2^-11 without; sum w |v| is the same attention over |v|, off by the roundings of its own, 2^-7 of it."""
    w4, steps = ex.w4, []
    real = w4.w4_attn_shared

    def both(q, k, v, kv_len, table, group, shared, max_len):
        out = real(q, k, v, kv_len, table, group, shared, max_len)
        want = w4.w4_attn_decode(q, k, v, kv_len, table, max_len).float()
        size = w4.w4_attn_decode(q, k, v.abs(), kv_len, table, max_len).float() * (1 + 2.0 ** -7)
        off = (out.float() - want).abs()
        # |o| of each form by the other's: off by `off`, which is small beside it
        steps.append((off <= 2 * U * (want.abs() + off) + (2.0 ** -8 + 2.0 ** -10) * size).all().item())
        return out
    monkeypatch.setattr(w4, "w4_attn_shared", both)
    serve(ex, cfg, n, OWN, 40, True)
    assert len(steps) == 40 and all(steps), [i for i, s in enumerate(steps) if not s]


@pytest.mark.parametrize("cfg", CONFIGS)
@pytest.mark.parametrize("n", [64, 150, 700])
def test_rows_with_the_same_experts(ex, cfg, n, monkeypatch):  # noqa: F811
    w4, ids, steps = ex.w4, [], 40
    real = w4.w4_moe_route

    def record(*args, **kw):
        got = real(*args, **kw)
        ids.append(got[1].sort(1)[0])
        return got
    monkeypatch.setattr(w4, "w4_moe_route", record)
    outs, chosen = [], []
    for shared in (True, False):
        ids.clear()
        outs.append(serve(ex, cfg, n, OWN, steps, shared).float())
        chosen.append(torch.stack(ids[-steps:]))
    same = (chosen[0] == chosen[1]).all(-1)
    assert same.float().mean() > 0.9
    d, size = (outs[0] - outs[1]).square().mean(-1).sqrt(), outs[1].square().mean(-1).sqrt()
    assert (d[same] <= 4 * RMS * size[same]).all()
    assert d[same].square().mean().sqrt() <= RMS * size[same].square().mean().sqrt()
