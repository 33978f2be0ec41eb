"""float64 oracle of the decoder-block operators: the norms around a block,
rotary positions, and masked softmax attention.  Plain numpy, from the
formulas in include/w4.h; shares nothing with the CUDA library."""
from __future__ import annotations

import math

import numpy as np


def block_norm(y, r, w_pre, w_post=None, gate=None, res_scale=1.0, eps=1e-6, w_offset=0.0):
    """(r', x, size): size is the magnitude of the terms of r', for tolerances."""
    r = np.asarray(r, np.float64)
    out, size = r, np.abs(r)
    if y is not None:
        u = np.asarray(y, np.float64)
        if w_post is not None:
            u = u / np.sqrt((u * u).mean(1, keepdims=True) + eps) * (w_offset + np.asarray(w_post, np.float64))
        if gate is not None:
            g = np.asarray(gate, np.float64)
            u = u * np.repeat(g, r.shape[0] // g.shape[0], axis=0)
        out, size = r + res_scale * u, np.abs(r) + np.abs(res_scale * u)
    if w_pre is None:
        return out, None, size
    norm = np.sqrt((out * out).mean(1, keepdims=True) + eps)
    return out, out / norm * (w_offset + np.asarray(w_pre, np.float64)), size


def rope_freqs(rot_dim, base, kind="plain", factor=1.0, orig_len=0, beta_fast=32.0, beta_slow=1.0):
    """Frequencies in float64 and the factor on cos and sin."""
    if kind == "ntk":
        base = base * factor ** (rot_dim / (rot_dim - 2))
    f = [base ** (-2.0 * i / rot_dim) for i in range(rot_dim // 2)]
    if kind == "linear":
        return [x / factor for x in f], 1.0
    if kind != "yarn":
        return f, 1.0

    def pair(turns):           # the (real) pair index that turns so often over orig_len
        return rot_dim / 2 * math.log(orig_len / (2 * math.pi * turns)) / math.log(base)
    lo, hi = max(math.floor(pair(beta_fast)), 0), min(math.ceil(pair(beta_slow)), rot_dim - 1)
    out = []
    for i, x in enumerate(f):
        t = min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
        out.append(x * (1 - t) + x / factor * t)
    return out, (0.1 * math.log(factor) + 1 if factor > 1 else 1.0)


def rope(x, pos, inv_freq, interleaved=False, mscale=1.0):
    """x [T, H, D] rotated at positions pos [T] in its first 2 len(inv_freq) values."""
    x = np.asarray(x, np.float64).copy()
    n = len(inv_freq)
    ang = np.asarray(pos, np.float64)[:, None] * np.asarray(inv_freq, np.float64)
    c, s = np.cos(ang)[:, None] * mscale, np.sin(ang)[:, None] * mscale
    ia = np.arange(n) * 2 if interleaved else np.arange(n)
    ib = ia + 1 if interleaved else ia + n
    a, b = x[..., ia].copy(), x[..., ib].copy()
    x[..., ia] = a * c - b * s
    x[..., ib] = a * s + b * c
    return x


def visible(p, n, window=0, sinks=0):
    """[len(p), n] bool: key j is seen from position p."""
    p = np.asarray(p)[:, None]
    j = np.arange(n)[None]
    ok = j <= p
    if window:
        ok &= (p - j < window) | (j < sinks)
    return ok


def attention(q, k, v, p, scale, window=0, sinks=0):
    """q [T, Hq, D] at positions p [T], k, v [n, Hkv, D] -> (o [T, Hq, D],
    lse [T, Hq], sum of w |v|).  Keys that no row of p sees are not touched;
    a masked key has no influence whatever it holds."""
    q = np.asarray(q, np.float64)
    T, Hq, D = q.shape
    n, Hkv, _ = k.shape
    g = Hq // Hkv
    see = visible(p, n, window, sinks)
    o = np.zeros((T, Hq, D))
    mag = np.zeros((T, Hq, D))
    lse = np.full((T, Hq), -np.inf)
    with np.errstate(invalid="ignore"):
        for t in range(T):
            at = np.nonzero(see[t])[0]
            if not len(at):
                continue
            for h in range(Hq):
                kk, vv = np.asarray(k[at, h // g], np.float64), np.asarray(v[at, h // g], np.float64)
                s = kk @ q[t, h] * scale
                m = s.max()
                w = np.exp(s - m)
                lse[t, h] = m + np.log(w.sum())
                w /= w.sum()
                o[t, h] = w @ vv
                mag[t, h] = w @ np.abs(vv)
    return o, lse, mag
