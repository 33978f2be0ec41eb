"""float64 oracle of the operators of a serving step: expert routing with the
order of the choices, and page plans.  Plain numpy and Python loops, from the
definitions in include/w4.h; shares nothing with the CUDA library."""
from __future__ import annotations

import numpy as np


def _scores(z, score):
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-z))
    m = z.max()
    if m == -np.inf:
        return np.zeros_like(z)
    e = (z == np.inf).astype(np.float64) if m == np.inf else np.exp(z - m)
    return e / e.sum()


def route(logits, k, bias=None, score="softmax", groups=1, top_groups=1, best=1, renorm=True, scale=1.0, count=None):
    """(weights [T, k], ids, row [T, k], goff [E + 1])."""
    z = np.array(logits, np.float64)
    z[np.isnan(z)] = -np.inf
    T, E = z.shape
    w, ids = np.zeros((T, k)), np.full((T, k), -1, np.int64)
    for t in range(T if count is None else min(max(count, 0), T)):
        x = z[t]
        p = _scores(x, score)
        s = p if bias is None else p + np.asarray(bias, np.float64)
        order = x if bias is None else s
        offered = (x > -np.inf) & (s > -np.inf)
        if groups > 1:
            by = x if bias is None and best == 1 else s
            rank = []
            for g in range(groups):
                at = range(g * (E // groups), (g + 1) * (E // groups))
                top = sorted((by[e] for e in at if offered[e]), reverse=True)[:best]
                rank.append(sum(top) if top else -np.inf)
            kept = sorted(range(groups), key=lambda g: (-rank[g], g))[:top_groups]
            offered &= np.isin(np.arange(E) // (E // groups), kept)
        chosen = sorted(np.nonzero(offered)[0], key=lambda e: (-order[e], e))[:k]
        for j, e in enumerate(chosen):
            ids[t, j], w[t, j] = e, p[e]
        if renorm and chosen:
            c = x[chosen]
            if score == "softmax":
                q = _scores(c, "softmax")
            else:
                # sigmoid over the largest of the chosen: ratios that survive underflow
                lift = min(c.max(), 0.0)
                q = np.array([_scores(v, "sigmoid") if lift == 0 else np.exp(v - lift) / (1 + np.exp(v)) for v in c])
                q = q / q.sum()
            w[t, :len(chosen)] = q
    row, n = np.full((T, k), -1, np.int64), 0
    goff = np.zeros(E + 1, np.int64)
    at = [[] for _ in range(E)]
    for t in range(T):
        for j in range(k):
            if ids[t, j] >= 0:
                at[ids[t, j]].append((t, j))
    for e in range(E):
        for t, j in at[e]:
            row[t, j] = n
            n += 1
        goff[e + 1] = n
    return w * scale, ids, row, goff


def plan(lens, new, free, used, table, page_size, pages, T):
    """dict of kv_len, goff, pos, slots, lens_out, used_out, table and the flags raised."""
    B, cols = table.shape
    table = table.copy()
    flags = set()
    if not 0 <= used <= len(free):
        flags.add("PAGE_TABLE")
        used = min(max(used, 0), len(free))
    kv_len, lens_out = np.zeros(B, np.int64), np.array(lens, np.int64)
    goff, pos, slots = np.zeros(B + 1, np.int64), np.full(T, -1, np.int64), np.full(T, -1, np.int64)
    row, at, end = 0, used, used                # rows and pages asked for so far, pages given
    for b in range(B):
        old, n = int(lens[b]), 1 if new is None else int(new[b])
        sized = old >= 0 and n >= 0 and old + n <= cols * page_size
        row0 = row
        row += max(n, 0)
        goff[b + 1] = min(row, T)
        if not sized:
            flags.add("PAGE_TABLE")
            continue
        if row > T:
            flags.add("GROUP_TOKENS")
            continue
        held, need = -(-old // page_size), -(-(old + n) // page_size) - -(-old // page_size)
        at += need
        if need and at > len(free):
            flags.add("NO_PAGES")
            continue
        if need:
            table[b, held:held + need] = free[at - need:at]
            end = at
        lens_out[b] = old + n
        kv_len[b] = old + n if n else 0
        for i in range(n):
            p = old + i
            pos[row0 + i] = p
            page = table[b, p // page_size]
            if 0 <= page < pages:
                slots[row0 + i] = page * page_size + p % page_size
            else:
                flags.add("PAGE_TABLE")
    return dict(kv_len=kv_len, goff=goff, pos=pos, slots=slots, lens_out=lens_out, used_out=end, table=table,
                flags=flags)
