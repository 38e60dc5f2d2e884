"""Plain forms of the planning of a step, the attention over shared prefixes and the rotation of cached
keys: loops over sequences, float64. Imported only by tests."""
from __future__ import annotations

import math

import torch

from cache_reference import gather, pages_of


def plan(change, kv, base, table, free, n_free, page, cols, max_rows):
    """(lengths, free entries, cu_q, table, free list, [(position, slot map, sequence)] per row), as lists. table None: dense."""
    up = lambda n: -(-n // page)
    paged = table is not None
    table = [list(r) for r in table] if paged else None
    stack = list(free[:n_free]) if paged else []
    if paged:
        for b, (x, n) in enumerate(zip(change, kv)):
            if x < 0:
                stack += table[b][up(max(0, n + x)):up(n)]
    back, given = len(stack), list(stack)
    lengths, cu, rows, waiting = [], [0], [], False
    for b, (x, n) in enumerate(zip(change, kv)):
        m = 0
        if x > 0 and n + x <= cols * page:
            need = up(n + x) - up(n) if paged else 0
            waiting = waiting or need > len(stack) or cu[-1] + x > max_rows
            m = 0 if waiting else x
            for j in range(up(n), up(n + m) if paged else up(n)):
                table[b][j] = stack.pop()
        for s in range(n, n + m):
            rows.append((base[b] + s, (table[b][s // page] if paged else b) * page + s % page, b))
        lengths.append(n + m if x > 0 else max(0, n + x))
        cu.append(cu[-1] + m)
    if paged:
        free = list(free)
        for i in range(n_free, len(stack)):
            free[i] = given[i]
        assert len(stack) <= back
    return lengths, len(stack), cu, table, free, rows


def prefix_attention(q, cu, kv, keys, values, table, groups, prefixes, pkeys, pvalues, ptable, kv_heads):
    """(out, lse, spread, slack) as cache_reference.attention gives them; groups: sequences of each."""
    total, hq, d = q.shape
    out = torch.full((total, hq, d), math.nan, dtype=torch.float64, device=q.device)
    lse = torch.full((total, hq), math.nan, dtype=torch.float64, device=q.device)
    spread, slack = torch.zeros_like(out), torch.zeros_like(lse)
    group = [g for g, n in enumerate(groups) for _ in range(n)]
    for b, n in enumerate(kv):
        m, r0 = cu[b + 1] - cu[b], cu[b]
        p = prefixes[group[b]] if b < len(group) else 0
        if m == 0:
            continue
        for h in range(kv_heads):
            k, v = gather(keys, table, b, h, n), gather(values, table, b, h, n)
            if p:
                k = torch.cat((gather(pkeys, ptable, group[b], h, p), k))
                v = torch.cat((gather(pvalues, ptable, group[b], h, p), v))
            seen = torch.arange(p + n, device=q.device)[None] <= (p + n - m + torch.arange(m, device=q.device))[:, None]
            seen = seen | (torch.arange(p + n, device=q.device) < p)[None]
            for j in range(h * (hq // kv_heads), (h + 1) * (hq // kv_heads)):
                y = q[r0:r0 + m, j].double()
                x = (y @ k.T / math.sqrt(d)).masked_fill(~seen, -math.inf)
                ab = y.abs() @ k.abs().T / math.sqrt(d)
                if p + n == 0:
                    out[r0:r0 + m, j], lse[r0:r0 + m, j] = 0, -math.inf
                    continue
                top = x.amax(-1, keepdim=True)
                top = torch.where(top.isinf(), torch.zeros_like(top), top)
                e = torch.exp(x - top)
                l = e.sum(-1, keepdim=True)
                e = torch.where(l > 0, e / l, torch.zeros_like(e))
                out[r0:r0 + m, j] = e @ v
                spread[r0:r0 + m, j] = e @ v.abs()
                lse[r0:r0 + m, j] = (l.log() + top)[:, 0]
                slack[r0:r0 + m, j] = ab.masked_fill(~seen, 0).amax(-1)
    return out, lse, spread, slack


def turned(x, at, start, to_freq, from_freq, rot, interleaved, scale):
    """Keys x [n, d] turned from positions `start` to `at` in float64, and the size of each element's pair."""
    y, size = x.double().clone(), x.double().abs()
    i = torch.arange(rot // 2, device=x.device)
    a, c = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    t = at.double()[:, None] * to_freq.double() - start.double()[:, None] * from_freq.double()
    p, q = x[:, a].double(), x[:, c].double()
    y[:, a] = scale * (p * torch.cos(t) - q * torch.sin(t))
    y[:, c] = scale * (q * torch.cos(t) + p * torch.sin(t))
    size[:, a] = size[:, c] = abs(scale) * torch.hypot(p, q)
    return y, size
