"""Timing cases of the operators of a serving step around routed experts and a shared cache.

Five operators: the choice of experts for every token with the order in which the grouped linears take them
(w4_moe_route), tokens copied into that order (w4_moe_gather), the experts' outputs weighted and summed back
(w4_moe_combine), page tables and slot maps from request lengths (w4_kv_plan) and attention of one new token per
sequence where groups of sequences share a long prefix (w4_attn_shared).  `run` computes a case either in plain
torch operations or, where `own` is true, with the library's calls; `exact` computes it in 64 bits from the
definitions.

Sizes: the expert layers of workloads.py (128 experts, 8 of them per token, hidden 2048), the 7B shapes (hidden
3584, 28 query and 4 key-value heads of 128), and generic expert counts and head layouts.
"""
import math
import random

import torch

own = False


# ------------------------------------------------------------------ cases
def listed():
    return [
        # routing of a small decode batch of the expert layers
        dict(name="route_16tok", op="route", T=16, E=128, k=8, score="softmax", bias=False, groups=1, top_groups=1,
             best=1, renorm=True, scale=1.0, half=True),
        # an odd number of tokens and of experts, a bias for balance, bf16 logits (equal ones are common)
        dict(name="route_odd", op="route", T=1003, E=60, k=6, score="sigmoid", bias=True, groups=1, top_groups=1, best=1,
             renorm=True, scale=1.0, half=True),
        # a prefill step of a large expert layer: groups of experts, ranked by their two best
        dict(name="route_16k_groups", op="route", T=16384, E=256, k=8, score="sigmoid", bias=True, groups=8, top_groups=4,
             best=2, renorm=True, scale=2.5, half=False),
        # tokens into expert order: a decode batch, a prefill step
        dict(name="gather_16tok", op="gather", T=16, E=128, k=8, K=2048),
        dict(name="gather_8192tok", op="gather", T=8192, E=128, k=8, K=2048),
        # experts' outputs back to tokens: a ragged chunk with a shared expert, a prefill step
        dict(name="combine_odd_shared", op="combine", T=333, E=64, k=6, N=3580, shared=True),
        dict(name="combine_8192tok", op="combine", T=8192, E=128, k=8, N=2048, shared=False),
        # a decode step of a serving batch: one token each, a few rows unused
        dict(name="plan_decode_256seq", op="plan", B=256, new_min=0, new_max=1, len_max=16384, page=16, mix=41),
        # prompts admitted next to running sequences
        dict(name="plan_mixed_prompts", op="plan", B=97, new_min=1, new_max=8192, len_max=65536, page=32, mix=42),
        # several answers to one prompt
        dict(name="shared_4seq_1k", op="shared", B=4, G=1, shared_min=1024, shared_max=1024, own_min=1, own_max=200, hq=28,
             hkv=4, d=128, page=16, mix=51),
        # a few documents, questions to each
        dict(name="shared_48seq_3docs", op="shared", B=48, G=3, shared_min=3000, shared_max=30000, own_min=1, own_max=900,
             hq=32, hkv=8, d=64, page=32, mix=52),
        # a large batch behind one long prompt
        dict(name="shared_256seq_32k", op="shared", B=256, G=1, shared_min=32768, shared_max=32768, own_min=1, own_max=2000,
             hq=28, hkv=4, d=128, page=64, mix=53),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))))))


HEADS = [(28, 4, 128), (32, 8, 128), (16, 16, 64), (24, 3, 64), (14, 2, 64), (8, 1, 128), (32, 8, 64)]
MOST_PAIRS = 256 * 28 * 128 * 34768            # sequences * hq * d * keys of the largest listed case


def draw(rng):
    op = rng.choice(["route", "route", "gather", "combine", "plan", "shared", "shared", "shared"])
    E = rng.choice([8, 16, 32, 60, 64, 128, 160, 256, 384])
    k = rng.choice([i for i in (1, 2, 4, 6, 8) if i <= E // 4])
    if op == "route":
        T = _log(rng, 1, 16384)
        groups = rng.choice([1, 1, 4, 8]) if E % 8 == 0 and E >= 64 else 1
        top = groups if groups == 1 else rng.randrange(groups // 2, groups + 1)
        return dict(op=op, T=min(T, 16384 * 256 // E), E=E, k=k, score=rng.choice(["softmax", "sigmoid"]),
                    bias=rng.random() < 0.5, groups=groups, top_groups=top, best=1 if groups == 1 else rng.choice([1, 2]),
                    renorm=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]), half=rng.random() < 0.5)
    if op in ("gather", "combine"):
        n = _log(rng, 256, 8192)
        if rng.random() < 0.7:
            n = (n + 7) // 8 * 8
        T = _log(rng, 1, max(1, min(8192, 8192 * 8 * 2048 // (n * k))))
        if op == "gather":
            return dict(op=op, T=T, E=E, k=k, K=n)
        return dict(op=op, T=T, E=E, k=k, N=n, shared=rng.random() < 0.5)
    page = rng.choice([16, 32, 64, 128])
    mix = rng.randrange(1 << 20)
    if op == "plan":
        B = _log(rng, 1, 512)
        hi = _log(rng, 1, 65536 // B) if rng.random() < 0.6 else 1
        return dict(op=op, B=B, new_min=rng.choice([0, 1]) if hi == 1 else _log(rng, 1, hi), new_max=hi,
                    len_max=_log(rng, 64, 65536), page=page, mix=mix)
    hq, hkv, d = rng.choice(HEADS)
    B = _log(rng, 2, 256)
    G = min(B, rng.choice([1, 1, 1, 2, 5]))
    top = _log(rng, 2 * page, min(65536, MOST_PAIRS // (hq * d * B)))
    most = _log(rng, 1, min(4000, max(1, MOST_PAIRS // (hq * d * B) - top + 1)))
    return dict(op=op, B=B, G=G, shared_min=max(page, top // 8), shared_max=top, own_min=1, own_max=most, hq=hq, hkv=hkv,
                d=d, page=page, mix=mix)


def _plan_lens(c):
    """(length before, new tokens) of each request; a row in eight of a decode batch may be unused."""
    r = random.Random(c["mix"])
    lens, new = [], []
    for b in range(c["B"]):
        if c["new_max"] == 1:
            n = c["new_min"] if b and r.random() < 0.125 else 1
        else:
            n = c["new_max"] if b == 0 else _log(r, max(1, c["new_min"]), c["new_max"])
        # a request of many new tokens is a prompt, most often its first chunk
        old = 0 if n > 64 and r.random() < 0.7 else _log(r, 1, c["len_max"])
        lens.append(old)
        new.append(n)
    return lens, new


def _shared_lens(c):
    """Sizes of the groups, their shared lengths (whole pages) and every sequence's own tokens."""
    r = random.Random(c["mix"])
    cuts = sorted(r.sample(range(1, c["B"]), c["G"] - 1))
    sizes = [b - a for a, b in zip([0] + cuts, cuts + [c["B"]])]
    page = c["page"]
    shared = [c["shared_max"] if i == 0 else _log(r, c["shared_min"], c["shared_max"]) for i in range(c["G"])]
    shared = [max(1, n // page) * page for n in shared]
    mine = [c["own_max"] if b == 0 else _log(r, c["own_min"], c["own_max"]) for b in range(c["B"])]
    return sizes, shared, mine


def work(c):
    op = c["op"]
    if op == "route":
        T, E, k = c["T"], c["E"], c["k"]
        return dict(bytes=T * E * (2 if c["half"] else 4) + 12 * T * k + 4 * (E + 1) + (4 * E if c["bias"] else 0),
                    flops=8 * T * E)
    if op == "gather":
        n = c["T"] * c["K"]
        return dict(bytes=2 * n * (1 + c["k"]) + 4 * c["T"] * c["k"], flops=0)
    if op == "combine":
        n = c["T"] * c["N"]
        return dict(bytes=2 * n * (1 + c["k"] + c["shared"]) + 8 * c["T"] * c["k"], flops=2 * n * (c["k"] + c["shared"]))
    if op == "plan":
        lens, new = _plan_lens(c)
        page = c["page"]
        pages = sum(-(-(n + m) // page) - -(-n // page) for n, m in zip(lens, new))
        return dict(bytes=20 * c["B"] + 12 * sum(new) + 8 * pages, flops=0)
    sizes, shared, mine = _shared_lens(c)
    hq, hkv, d, B = c["hq"], c["hkv"], c["d"], c["B"]
    keys = sum(shared) + sum(mine)
    pairs = sum(n * m for n, m in zip(sizes, shared)) + sum(mine)
    return dict(bytes=4 * keys * hkv * d + 4 * B * hq * d, flops=4 * pairs * hq * d)


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    c = dict(case)
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)

    def randn(*shape, scale=1.0, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device=dev, dtype=dtype).mul_(scale)

    op = c["op"]
    if op == "route":
        T, E = c["T"], c["E"]
        # some experts are liked more than others
        x = randn(T, E, scale=1.3, dtype=torch.float32) + randn(E, scale=0.5, dtype=torch.float32)
        c["logits"] = x.bfloat16() if c["half"] else x
        c["b"] = randn(E, scale=0.03, dtype=torch.float32) if c["bias"] else None
        return c
    if op in ("gather", "combine"):
        T, E, k = c["T"], c["E"], c["k"]
        ids = torch.rand(T, E, generator=g, device=dev).argsort(1)[:, :k]
        order = ids.flatten().argsort(stable=True)
        row = torch.empty_like(order)
        row[order] = torch.arange(T * k, device=dev)
        c["row"] = row.int().view(T, k)
        if op == "gather":
            c["x"] = randn(T, c["K"])
            return c
        w = torch.rand(T, k, generator=g, device=dev) + 0.1
        c["w"] = w / w.sum(1, keepdim=True)
        c["y"] = randn(T * k, c["N"])
        c["s"] = randn(T, c["N"], scale=0.5) if c["shared"] else None
        return c
    page = c["page"]
    if op == "plan":
        lens, new = _plan_lens(c)
        B = c["B"]
        held = [-(-n // page) for n in lens]
        need = [-(-(n + m) // page) - h for n, m, h in zip(lens, new, held)]
        cols = max(h + m for h, m in zip(held, need)) + 4
        pages = sum(held) + sum(need) + 64
        order = torch.randperm(pages, generator=g, device=dev).int()
        # the pages that the requests hold, then the free ones, of which a few are given out already
        held_d = torch.tensor(held, device=dev)
        at = held_d.cumsum(0)[:, None] - held_d[:, None] + torch.arange(cols, device=dev)
        c["table"] = torch.where(torch.arange(cols, device=dev) < held_d[:, None], order[at.clamp(max=pages - 1)], -1)
        c["free"] = order[max(0, sum(held) - 5):].contiguous()
        c["used"] = torch.tensor([min(5, sum(held))], dtype=torch.int32, device=dev)
        c["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        c["new"] = torch.tensor(new, dtype=torch.int32, device=dev)
        c["lens_out"], c["used_out"] = torch.empty_like(c["lens"]), torch.empty_like(c["used"])
        c["T"], c["pages"] = sum(new) + 3, pages          # the launch has a few rows more than tokens
        return c
    sizes, shared, mine = _shared_lens(c)
    B, hq, hkv, d = c["B"], c["hq"], c["hkv"], c["d"]
    of = [i for i, n in enumerate(sizes) for _ in range(n)]
    kv = [shared[i] + m for i, m in zip(of, mine)]
    heads = [n // page for n in shared]                   # pages of each prefix
    tails = [-(-m // page) for m in mine]
    pages = sum(heads) + sum(tails) + 1
    order = (torch.randperm(pages - 1, generator=torch.Generator().manual_seed(seed)) + 1).int()
    table = torch.zeros(B, max(heads[i] + t for i, t in zip(of, tails)), dtype=torch.int32)
    first, at = [], 0
    for n in heads:
        first.append(at)
        at += n
    for b, (i, t) in enumerate(zip(of, tails)):
        table[b, :heads[i]] = order[first[i]:first[i] + heads[i]]
        table[b, heads[i]:heads[i] + t] = order[at:at + t]
        at += t
    c["table"] = table.to(dev)
    c["kv_len"] = torch.tensor(kv, dtype=torch.int32, device=dev)
    c["group"] = torch.tensor([0] + sizes, dtype=torch.int32).cumsum(0).int().to(dev)
    c["shared"] = torch.tensor(shared, dtype=torch.int32, device=dev)
    c["max_len"] = max(kv)
    c["q"] = randn(B, hq, d, scale=1.4)
    c["k_cache"] = randn(pages, hkv, page, d)
    c["k_cache"][..., :: d // 4] *= 2.0                   # the large channels of keys
    c["v_cache"] = randn(pages, hkv, page, d)
    return c


# ------------------------------------------------------------------ one pass
def run(s):
    return _run_own(s) if own else _PLAIN[s["op"]](s)


def _run_own(s):
    import int4_weight_only_gb300 as w4
    op = s["op"]
    if op == "route":
        return w4.w4_moe_route(s["logits"], s["k"], bias=s["b"], score=s["score"], groups=s["groups"],
                               top_groups=s["top_groups"], group_best=s["best"], renorm=s["renorm"], scale=s["scale"])
    if op == "gather":
        return w4.w4_moe_gather(s["x"], s["row"])
    if op == "combine":
        return w4.w4_moe_combine(s["y"], s["row"], s["w"], shared=s["s"])
    if op == "plan":
        out = w4.w4_kv_plan(s["lens"], s["new"], s["free"], s["used"], s["table"], s["page"], s["pages"], s["T"],
                            lens_out=s["lens_out"], used_out=s["used_out"])
        return (*out, s["lens_out"], s["used_out"], s["table"])
    return w4.w4_attn_shared(s["q"], s["k_cache"], s["v_cache"], s["kv_len"], s["table"], s["group"], s["shared"],
                             s["max_len"])


def _plain_route(s):
    x, E, k = s["logits"].float(), s["E"], s["k"]
    T = x.shape[0]
    # scores next to the border are told apart in 64 bits; without a bias the logits have their order
    wide = x.double()
    score = torch.sigmoid(wide) if s["score"] == "sigmoid" else torch.exp(wide - wide.amax(1, keepdim=True))
    if s["score"] != "sigmoid":
        score = score / score.sum(1, keepdim=True)
    key = wide if s["b"] is None else score + s["b"].double()
    if s["groups"] > 1:
        by_group = (key if s["best"] == 1 or s["b"] is not None else score).view(T, s["groups"], -1)
        rank = by_group.sort(dim=2, descending=True)[0][..., :s["best"]].sum(2)
        kept = rank.sort(dim=1, descending=True, stable=True)[1][:, :s["top_groups"]]
        keep = torch.zeros_like(rank, dtype=torch.bool).scatter_(1, kept, True)
        key = key.masked_fill(~keep.repeat_interleave(E // s["groups"], 1), -math.inf)
    ids = key.sort(dim=1, descending=True, stable=True)[1][:, :k]
    p = torch.sigmoid(x) if s["score"] == "sigmoid" else torch.exp(x - x.amax(1, keepdim=True))
    if s["score"] != "sigmoid":
        p = p / p.sum(1, keepdim=True)
    w = p.gather(1, ids)
    if s["renorm"]:
        w = w / w.sum(1, keepdim=True)
    by_expert, order = ids.flatten().sort(stable=True)
    row = torch.empty_like(order)
    row[order] = torch.arange(T * k, device=x.device)
    goff = torch.searchsorted(by_expert, torch.arange(E + 1, device=x.device))
    return w * s["scale"], ids.int(), row.int().view(T, k), goff.int()


def _plain_gather(s):
    out = s["x"].new_empty(s["row"].numel(), s["K"])
    out[s["row"].flatten().long()] = s["x"].repeat_interleave(s["k"], 0)
    return out


def _plain_combine(s):
    y = (s["y"][s["row"].long()].float() * s["w"][..., None]).sum(1)
    return (y if s["s"] is None else y + s["s"].float()).bfloat16()


def _plain_plan(s):
    page, T, table, B = s["page"], s["T"], s["table"], s["B"]
    dev = table.device
    old, new = s["lens"].long(), s["new"].long()
    end = new.cumsum(0)
    goff = torch.cat([end.new_zeros(1), end])
    have, want = (old + page - 1) // page, (old + new + page - 1) // page
    start = s["used"].long() + (want - have).cumsum(0) - (want - have)
    cols = torch.arange(table.shape[1], device=dev)
    fresh = (cols >= have[:, None]) & (cols < want[:, None])
    at = (start[:, None] + cols - have[:, None]).clamp(0, s["free"].numel() - 1)
    table.copy_(torch.where(fresh, s["free"][at], table))
    t = torch.arange(T, device=dev)
    b = torch.searchsorted(end, t, right=True)
    real = b < B
    b = b.clamp(max=B - 1)
    pos = torch.where(real, old[b] + t - goff[b], -1)
    p = pos.clamp(min=0)
    slots = torch.where(real, table[b, p // page].long() * page + p % page, -1)
    s["lens_out"].copy_(old + new)
    s["used_out"].copy_(s["used"] + (want - have).sum())
    kv_len = torch.where(new > 0, old + new, 0)
    return kv_len.int(), goff.int(), pos.int(), slots, s["lens_out"], s["used_out"], table


def _plain_shared(s):
    """Every sequence's whole cache, as if nothing were shared."""
    B, hkv, d = s["B"], s["hkv"], s["d"]
    ids = s["table"].long()
    k = s["k_cache"][ids].float().permute(0, 1, 3, 2, 4).flatten(1, 2)
    v = s["v_cache"][ids].float().permute(0, 1, 3, 2, 4).flatten(1, 2)
    q = s["q"].view(B, hkv, -1, d).float() / math.sqrt(d)
    score = torch.einsum("bhgd,blhd->bhgl", q, k)
    hide = torch.arange(k.shape[1], device=k.device) >= s["kv_len"][:, None]
    score = score.masked_fill_(hide[:, None, None], -math.inf)
    p = score.sub_(score.amax(-1, keepdim=True)).exp_()
    o = torch.einsum("bhgl,blhd->bhgd", p, v) / p.sum(-1, keepdim=True)
    return o.reshape(B, -1, d).bfloat16()


_PLAIN = {"route": _plain_route, "gather": _plain_gather, "combine": _plain_combine, "plan": _plain_plan,
          "shared": _plain_shared}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "route":
        z = s["logits"].double()
        T, E = z.shape
        p = 1 / (1 + torch.exp(-z)) if s["score"] == "sigmoid" else torch.softmax(z, 1)
        rank = z if s["b"] is None else p + s["b"].double()
        if s["groups"] > 1:
            rows = (rank if s["b"] is not None or s["best"] == 1 else p).unflatten(1, (s["groups"], E // s["groups"]))
            total = torch.topk(rows, s["best"], dim=2)[0].sum(2)
            low = torch.topk(total, s["top_groups"], dim=1)[0][:, -1:]
            out = (total < low)[:, :, None].expand(-1, -1, E // s["groups"]).flatten(1)
            rank = torch.where(out, -math.inf, rank)
        rank, w = rank.clone(), []
        for _ in range(s["k"]):
            best = (rank == rank.amax(1, keepdim=True)).int().argmax(1, keepdim=True)     # the first of equal ones
            w.append(p.gather(1, best))
            rank.scatter_(1, best, -math.inf)
        w = torch.cat(w, 1)
        if s["renorm"]:
            w = w / w.sum(1, keepdim=True)
        return s["scale"] * w, None, None, None
    if op == "gather":
        out = torch.empty(s["T"] * s["k"], s["K"], dtype=torch.float64, device=s["x"].device)
        for j in range(s["k"]):
            out[s["row"][:, j].long()] = s["x"].double()
        return out
    if op == "combine":
        out = 0 if s["s"] is None else s["s"].double()
        for j in range(s["k"]):
            out = out + s["w"][:, j:j + 1].double() * s["y"][s["row"][:, j].long()].double()
        return out
    if op == "plan":
        return None
    d, per = s["d"], s["hq"] // s["hkv"]
    out = torch.empty(s["B"], s["hq"], d, dtype=torch.float64, device=s["q"].device)
    for b, n in enumerate(s["kv_len"].tolist()):
        ids = s["table"][b, :-(-n // s["page"])].long()
        k, v = (x[ids].transpose(0, 1).flatten(1, 2)[:, :n].double() for x in (s["k_cache"], s["v_cache"]))
        a = torch.bmm(s["q"][b].double().view(s["hkv"], per, d), k.transpose(1, 2)) * d ** -0.5
        out[b] = torch.bmm(torch.softmax(a, -1), v).flatten(0, 1)
    return out
