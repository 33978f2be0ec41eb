"""Timing cases of the decoder-block operators that sit between the INT4 linear layers.

Four operators: the norms around a block (w4_block_norm), rotary positions with the write into a paged
key-value cache (w4_rope_append), attention of one new token over that cache (w4_attn_decode) and attention of
a prompt or a chunk of one (w4_attn_prefill).  `run` computes a case either in plain torch operations in 32
bits or, where `own` is true, with the library's calls; `exact` computes it in 64 bits from the definitions.

Sizes: the 7B shapes of workloads.py (hidden 3584, 28 query and 4 key-value heads of 128), the 12B hidden size
3840, and generic head layouts (no grouping, groups of 4, 7 and 8, one shared head; heads of 64 and 128).
"""
import math
import random

import torch

own = False

EPS = 1e-6


# ------------------------------------------------------------------ cases
def listed():
    return [
        # norms: one token between o and gate|up of the 7B block
        dict(name="norm_7b_1tok", op="norm", M=1, K=3584, post=False, gate=0, scale=1.0),
        # a ragged batch of prompt tokens, norms on both sides and a gate per sequence
        dict(name="norm_gated_odd", op="norm", M=1001, K=3580, post=True, gate=7, scale=0.5),
        # a full prefill step at the 12B hidden size, norms on both sides of the block
        dict(name="norm_12b_8192tok", op="norm", M=8192, K=3840, post=True, gate=0, scale=1.0),
        # rotary + cache write: a small decode batch of the 7B block
        dict(name="rope_7b_8seq", op="rope", B=8, q_min=1, q_max=1, len_min=100, len_max=4000, hq=28, hkv=4, d=128,
             rot=128, inter=False, yarn=1.0, page=16, mix=11),
        # long contexts: stretched frequencies, half of the head rotated, adjacent pairs, chunks of odd length
        dict(name="rope_long_interleaved", op="rope", B=24, q_min=1, q_max=257, len_min=2000, len_max=131072, hq=32,
             hkv=8, d=128, rot=64, inter=True, yarn=16.0, page=32, mix=12),
        # a prefill step of the 7B block, several prompts
        dict(name="rope_7b_prefill", op="rope", B=4, q_min=1500, q_max=2500, len_min=3000, len_max=8192, hq=28, hkv=4,
             d=128, rot=128, inter=False, yarn=1.0, page=64, mix=13),
        # decode attention: one user, a short chat
        dict(name="decode_1seq_517", op="decode", B=1, len_min=517, len_max=517, hq=28, hkv=4, d=128, window=0, sinks=0,
             page=16, mix=21),
        # a serving batch with ragged lengths
        dict(name="decode_64seq_ragged", op="decode", B=64, len_min=1, len_max=8192, hq=28, hkv=4, d=128, window=0,
             sinks=0, page=16, mix=22),
        # a few very long contexts
        dict(name="decode_8seq_128k", op="decode", B=8, len_min=120001, len_max=131071, hq=28, hkv=4, d=128, window=0,
             sinks=0, page=64, mix=23),
        # prompt attention: a short chunk on top of a cached prefix, sliding window with first tokens kept
        dict(name="prefill_chunk_window", op="prefill", B=5, q_min=33, q_max=300, len_min=1500, len_max=6000, hq=16,
             hkv=16, d=64, window=1024, sinks=4, page=16, mix=31),
        # the 7B prefill of 2048 tokens
        dict(name="prefill_7b_2048", op="prefill", B=1, q_min=2048, q_max=2048, len_min=2048, len_max=2048, hq=28, hkv=4,
             d=128, window=0, sinks=0, page=64, mix=32),
        # a long prompt
        dict(name="prefill_7b_8192", op="prefill", B=1, q_min=8192, q_max=8192, len_min=8192, len_max=8192, hq=28, hkv=4,
             d=128, window=0, sinks=0, page=128, mix=33),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))))))


HEADS = [(28, 4, 128), (32, 8, 128), (16, 16, 64), (24, 3, 64), (14, 2, 64), (8, 1, 128), (5, 5, 128)]
MOST_PAIRS = 28 * 128 * 8192 * 4096        # hq * d * visible pairs of the longest prompt


def draw(rng):
    op = rng.choice(["norm", "rope", "decode", "decode", "prefill", "prefill"])
    hq, hkv, d = rng.choice(HEADS)
    page = rng.choice([16, 32, 64, 128])
    mix = rng.randrange(1 << 20)
    if op == "norm":
        K = _log(rng, 256, 8192)
        if rng.random() < 0.7:
            K = (K + 7) // 8 * 8
        M = _log(rng, 1, 8192)
        return dict(op=op, M=M, K=K, post=rng.random() < 0.5, gate=rng.choice([0, 1, M]), scale=rng.choice([1.0, 0.25]))
    if op == "rope":
        B = _log(rng, 1, 64)
        hi = _log(rng, 1, 4096 // B + 1) if rng.random() < 0.6 else 1
        lo = _log(rng, 1, hi)
        top = _log(rng, max(hi, 16), 131072)
        return dict(op=op, B=B, q_min=lo, q_max=hi, len_min=hi, len_max=top, hq=hq, hkv=hkv, d=d,
                    rot=rng.choice([d, d, d // 2]), inter=rng.random() < 0.5, yarn=rng.choice([1.0, 1.0, 8.0]), page=page,
                    mix=mix)
    window, sinks = rng.choice([(0, 0), (0, 0), (4096, 4), (_log(rng, 100, 2000), rng.randrange(0, 40))])
    if op == "decode":
        B = _log(rng, 1, 128)
        top = _log(rng, 16, min(131072, (1 << 29) // (B * hkv * d)))
        return dict(op=op, B=B, len_min=_log(rng, 1, top), len_max=top, hq=hq, hkv=hkv, d=d, window=window, sinks=sinks,
                    page=page, mix=mix)
    B = rng.randrange(1, 6)
    hi = _log(rng, 1, 4096)
    top = _log(rng, hi, min(32768, max(hi, MOST_PAIRS // (hq * d * hi * B))))
    lo = _log(rng, max(1, hi // 3), hi)
    return dict(op=op, B=B, q_min=lo, q_max=hi, len_min=max(hi, top // 2), len_max=top, hq=hq, hkv=hkv, d=d, window=window,
                sinks=sinks, page=page, mix=mix)


def _lens(c):
    """(tokens of this step, length after it) of each sequence: spread over the case's ranges, a longest one among them."""
    r = random.Random(c["mix"])
    kv = [c["len_max"] if b == 0 else _log(r, c["len_min"], c["len_max"]) for b in range(c["B"])]
    if c["op"] == "decode":
        return [1] * c["B"], kv
    q = [c["q_max"] if b == 0 else _log(r, c["q_min"], c["q_max"]) for b in range(c["B"])]
    return q, [max(n, m) for n, m in zip(kv, q)]


def _visible(q, n, window, sinks):
    """Visible (query, key) pairs of q tokens ending at length n."""
    if not window:
        return q * n - q * (q - 1) // 2
    return sum(min(p + 1, window) + min(sinks, max(0, p + 1 - window)) for p in range(n - q, n))


def work(c):
    if c["op"] == "norm":
        n = c["M"] * c["K"]
        vec = (1 + c["post"]) * c["K"] + c["gate"] * c["K"]
        return dict(bytes=8 * n + 2 * vec, flops=(10 + 4 * c["post"]) * n)
    qs, kv = _lens(c)
    T, hq, hkv, d = sum(qs), c["hq"], c["hkv"], c["d"]
    if c["op"] == "rope":
        return dict(bytes=4 * T * (hq + 2 * hkv) * d, flops=3 * T * (hq + hkv) * c["rot"])
    pairs = sum(_visible(q, n, c["window"], c["sinks"]) for q, n in zip(qs, kv))
    w = c["window"]
    keys = sum(n if not w else min(n, min(n, q + w - 1) + min(c["sinks"], max(0, n - q - w + 1))) for q, n in zip(qs, kv))
    return dict(bytes=4 * keys * hkv * d + 4 * T * hq * d, flops=4 * pairs * hq * d)


# ------------------------------------------------------------------ inputs
def _inv_freq(rot, yarn):
    """Rotary frequencies (base 1e6), stretched by yarn's bands for contexts `yarn` times 8192: the fast ones kept, the slow
    ones divided, a ramp between; and the factor on cos and sin."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    f = 1e6 ** (-2 * i / rot)
    turns = 8192 * f / (2 * math.pi)
    keep = ((turns - 1) / (32 - 1)).clamp(0, 1)
    return (f * keep + f / yarn * (1 - keep)).float(), 0.1 * math.log(yarn) + 1.0


def prepare(case, seed):
    c = dict(case)
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)

    def randn(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.bfloat16).mul_(scale)

    if c["op"] == "norm":
        M, K = c["M"], c["K"]
        c["y"] = randn(M, K, scale=0.7)
        c["r"] = randn(M, K, scale=2.0)
        c["r"][:, ::97] *= 12.0                    # the few large channels of a residual stream
        c["w_pre"] = 1 + randn(K, scale=0.1)
        c["w_post"] = 1 + randn(K, scale=0.1) if c["post"] else None
        c["g"] = randn(c["gate"], K, scale=0.5) if c["gate"] else None
        return c
    qs, kv = _lens(c)
    B, hq, hkv, d, page = c["B"], c["hq"], c["hkv"], c["d"], c["page"]
    T = sum(qs)
    goff = [0]
    for n in qs:
        goff.append(goff[-1] + n)
    c["goff"] = torch.tensor(goff, dtype=torch.int32, device=dev)
    c["kv_len"] = torch.tensor(kv, dtype=torch.int32, device=dev)
    c["max_q"], c["max_len"], c["T"] = max(qs), max(kv), T
    cols = -(-max(kv) // page)
    table = torch.zeros(B, cols, dtype=torch.int32)
    if c["op"] == "rope":
        # the pool holds the pages that this step writes; the rest of each table names page 0
        need = [(b, j) for b in range(B) for j in range((kv[b] - qs[b]) // page, -(-kv[b] // page))]
    else:
        need = [(b, j) for b in range(B) for j in range(-(-kv[b] // page))]
    pages = len(need) + 1
    at = torch.randperm(pages - 1, generator=torch.Generator().manual_seed(seed)) + 1
    rows = torch.tensor(need)
    table[rows[:, 0], rows[:, 1]] = at.int()
    c["table"] = table.to(dev)
    if c["op"] == "rope":
        c["qkv"] = randn(T, (hq + 2 * hkv) * d, scale=1.3)
        inv, c["m"] = _inv_freq(c["rot"], c["yarn"])
        c["inv_freq"] = inv.to(dev)
        c["k_cache"] = torch.zeros(pages, hkv, page, d, dtype=torch.bfloat16, device=dev)
        c["v_cache"] = torch.zeros_like(c["k_cache"])
        return c
    c["q"] = randn(T, hq, d, scale=1.4)
    c["k_cache"] = randn(pages, hkv, page, d)
    c["k_cache"][..., :: d // 4] *= 2.0            # the large channels of keys
    c["v_cache"] = randn(pages, hkv, page, d)
    return c


# ------------------------------------------------------------------ one pass
def run(s):
    return _run_own(s) if own else _PLAIN[s["op"]](s)


def _run_own(s):
    import int4_weight_only_gb300 as w4
    op = s["op"]
    if op == "norm":
        return w4.w4_block_norm(s["y"], s["r"], s["w_pre"], s["w_post"], s["g"], s["scale"], EPS)
    if op == "rope":
        hq, hkv, d = s["hq"], s["hkv"], s["d"]
        qkv = s["qkv"].view(s["T"], hq + 2 * hkv, d)
        q = w4.w4_rope_append(qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], s["k_cache"], s["v_cache"],
                              s["kv_len"], s["table"], s["inv_freq"], goff=None if s["q_max"] == 1 else s["goff"],
                              interleaved=s["inter"], mscale=s["m"])
        return q, s["k_cache"], s["v_cache"]
    if op == "decode":
        return w4.w4_attn_decode(s["q"], s["k_cache"], s["v_cache"], s["kv_len"], s["table"], s["max_len"],
                                 window=s["window"], sinks=s["sinks"])
    return w4.w4_attn_prefill(s["q"], s["k_cache"], s["v_cache"], s["goff"], s["kv_len"], s["table"], s["max_q"],
                              s["max_len"], window=s["window"], sinks=s["sinks"])


def _plain_norm(s):
    y, r = s["y"].float(), s["r"].float()
    if s["w_post"] is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * s["w_post"].float()
    if s["g"] is not None:
        rows = torch.arange(s["M"], device=y.device) // (s["M"] // s["gate"])
        y = y * s["g"].float()[rows]
    r = r + s["scale"] * y
    x = r * torch.rsqrt(r.square().mean(-1, keepdim=True) + EPS) * s["w_pre"].float()
    return r.bfloat16(), x.bfloat16()


def _tokens(s):
    """Sequence and position of every token."""
    t = torch.arange(s["T"], device=s["goff"].device)
    b = torch.searchsorted(s["goff"], t, right=True) - 1
    return b, s["kv_len"][b] - s["goff"][b + 1] + t


def _angles(pos, inv):
    """pos * inv modulo 2 pi in 32 bits: both factors split into 12-bit parts, whose products are exact, and each reduced
    with 2 pi = 6.28125 + a rest (a plain 32-bit product is 0.004 off at position 131071)."""
    hi = (pos // 4096).float()[:, None] * 4096
    lo = (pos % 4096).float()[:, None]
    fh = (inv.view(torch.int32) & -4096).view(torch.float32)
    parts = torch.stack([hi * fh, lo * fh, hi * (inv - fh), lo * (inv - fh)])
    k = torch.round(parts * (1 / (2 * math.pi)))
    return (parts - k * 6.28125 - k * (2 * math.pi - 6.28125)).sum(0)


def _plain_rope(s):
    hq, hkv, d, rot = s["hq"], s["hkv"], s["d"], s["rot"]
    b, pos = _tokens(s)
    x = s["qkv"].view(s["T"], hq + 2 * hkv, d).float()
    qk, v = x[:, :hq + hkv], x[:, hq + hkv:]
    a = _angles(pos, s["inv_freq"])
    cos, sin = (a.cos() * s["m"])[:, None], (a.sin() * s["m"])[:, None]
    if s["inter"]:
        u, w = qk[..., 0:rot:2], qk[..., 1:rot:2]
        turned = torch.stack([u * cos - w * sin, u * sin + w * cos], dim=-1).flatten(-2)
    else:
        u, w = qk[..., :rot // 2], qk[..., rot // 2:rot]
        turned = torch.cat([u * cos - w * sin, u * sin + w * cos], dim=-1)
    qk = torch.cat([turned, qk[..., rot:]], dim=-1).bfloat16()
    at, slot = s["table"][b, pos // s["page"]].long(), pos % s["page"]
    s["k_cache"][at, :, slot] = qk[:, hq:]
    s["v_cache"][at, :, slot] = v.bfloat16()
    return qk[:, :hq].contiguous(), s["k_cache"], s["v_cache"]


def _rows_of_cache(s, pool):
    """[B, keys, Hkv, D] in 32 bits."""
    x = pool[s["table"].long()].float()
    return x.permute(0, 1, 3, 2, 4).flatten(1, 2)


def _softmax_av(score, see, v):
    score = score.masked_fill_(~see, -math.inf)
    m = score.amax(-1, keepdim=True).clamp_min_(-3e38)
    p = score.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    return torch.einsum("bhgql,blhd->bqhgd", p, v), total


def _plain_decode(s):
    return _plain_attention(s, s["q"].view(s["B"], 1, s["hkv"], -1, s["d"]), s["kv_len"].long()[:, None] - 1).view_as(s["q"])


def _plain_attention(s, q, pos):
    """q [B, Q, Hkv, g, D], pos [B, Q] (negative: no token) -> [B, Q, Hkv, g, D] bf16."""
    k, v = _rows_of_cache(s, s["k_cache"]), _rows_of_cache(s, s["v_cache"])
    j = torch.arange(k.shape[1], device=k.device)
    p = pos[:, :, None]
    see = j <= p
    if s["window"]:
        see = see & ((p - j < s["window"]) | (j < s["sinks"]))
    score = torch.einsum("bqhgd,blhd->bhgql", q.float() / math.sqrt(s["d"]), k)
    o, total = _softmax_av(score, see[:, None, None], v)
    total = total.permute(0, 3, 1, 2, 4)
    return torch.where(total > 0, o / total, 0.0).bfloat16()


def _plain_prefill(s):
    b, pos = _tokens(s)
    i = torch.arange(s["T"], device=b.device) - s["goff"][b]
    q = s["q"].new_zeros(s["B"], s["max_q"], s["hkv"], s["hq"] // s["hkv"], s["d"])
    q[b, i] = s["q"].view(s["T"], s["hkv"], -1, s["d"])
    at = torch.full((s["B"], s["max_q"]), -1, device=b.device)
    at[b, i] = pos.long()
    return _plain_attention(s, q, at)[b, i].reshape(s["T"], s["hq"], s["d"])


_PLAIN = {"norm": _plain_norm, "rope": _plain_rope, "decode": _plain_decode, "prefill": _plain_prefill}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "norm":
        y, r = s["y"].double(), s["r"].double()
        if s["post"]:
            y = y / (y.pow(2).sum(1, keepdim=True) / s["K"] + EPS).sqrt() * s["w_post"].double()
        if s["gate"]:
            y = y * s["g"].double().repeat_interleave(s["M"] // s["gate"], 0)
        r = r + y * s["scale"]
        return r, r / (r.pow(2).sum(1, keepdim=True) / s["K"] + EPS).sqrt() * s["w_pre"].double()
    qs, kv = _lens(case)
    hq, hkv, d, page = s["hq"], s["hkv"], s["d"], s["page"]
    dev = s["kv_len"].device
    t0 = 0
    if s["op"] == "rope":
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        qkv = s["qkv"].double().reshape(s["T"], hq + 2 * hkv, d)
        out = []
        for b, (n, m) in enumerate(zip(qs, kv)):
            p = torch.arange(m - n, m, device=dev)
            x = qkv[t0:t0 + n]
            t0 += n
            turn = torch.polar(torch.full((), s["m"], dtype=torch.float64, device=dev),
                               p.double()[:, None] * s["inv_freq"].double())[:, None]
            head, half = x[:, :hq + hkv, :s["rot"]], s["rot"] // 2
            z = head.unflatten(-1, (half, 2)) if s["inter"] else head.unflatten(-1, (2, half)).transpose(-1, -2)
            z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * turn)
            z = z if s["inter"] else z.transpose(-1, -2)
            z = torch.cat([z.flatten(-2), x[:, :hq + hkv, s["rot"]:]], -1)
            out.append(z[:, :hq])
            cell = s["table"][b].long()[p // page] * page + p % page
            kc.transpose(1, 2)[cell // page, cell % page] = z[:, hq:]
            vc.transpose(1, 2)[cell // page, cell % page] = x[:, hq + hkv:]
        return torch.cat(out), kc, vc
    out = torch.empty(s["T"], hq, d, dtype=torch.float64, device=dev)
    for b, (n, m) in enumerate(zip(qs, kv)):
        ids = s["table"][b, :-(-m // page)].long()
        p = torch.arange(m - n, m, device=dev)[:, None]
        j = torch.arange(m, device=dev)[None]
        hide = j > p
        if s["window"]:
            hide = hide | ((j <= p - s["window"]) & (j >= s["sinks"]))
        for h in range(hkv):
            k = s["k_cache"][ids, h].double().reshape(-1, d)[:m]
            v = s["v_cache"][ids, h].double().reshape(-1, d)[:m]
            for g in range(h * (hq // hkv), (h + 1) * (hq // hkv)):
                a = (s["q"][t0:t0 + n, g].double() @ k.T / d ** 0.5).masked_fill(hide, -math.inf)
                out[t0:t0 + n, g] = torch.softmax(a, 1) @ v
        t0 += n
    return out
