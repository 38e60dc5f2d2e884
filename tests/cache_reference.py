"""Plain float64 forms of the cache operators, one sequence, head and slot range at a time.
Imported only by tests. Every function works on the pool as the library sees it."""
from __future__ import annotations

import math

import torch


def pages_of(table, b, n, page_size):
    cols = -(-n // page_size)
    return [b] * cols if table is None else table[b, :cols].tolist()


def gather(pool, table, b, h, n):
    """Slots [0, n) of KV head h of sequence b, float64 [n, d]."""
    ps = pool.shape[2]
    parts = [pool[p, h, :min(ps, n - i * ps)] for i, p in enumerate(pages_of(table, b, n, ps))]
    return torch.cat(parts).double() if parts else pool.new_zeros(0, pool.shape[3]).double()


def attention(q, cu, kv, keys, values, table, kv_heads):
    """(out, lse, spread, slack) in float64; spread = sum p |v|, slack = the largest sum of
    |q k| / sqrt(d) over a row's keys (what the logits' rounding goes by)."""
    total, hq, d = q.shape
    out = torch.full((total, hq, d), math.nan, dtype=torch.float64, device=q.device)
    lse = torch.full((total, hq), math.nan, dtype=torch.float64, device=q.device)
    spread, slack = torch.zeros_like(out), torch.zeros_like(lse)
    for b, n in enumerate(kv):
        m, r0 = cu[b + 1] - cu[b], cu[b]
        for j in range(hq):
            h = j // (hq // kv_heads)
            k, v = gather(keys, table, b, h, n), gather(values, table, b, h, n)
            x = q[r0:r0 + m, j].double() @ k.T / math.sqrt(d)
            ab = q[r0:r0 + m, j].double().abs() @ k.abs().T / math.sqrt(d)
            seen = torch.arange(n, device=q.device)[None] <= (n - m + torch.arange(m, device=q.device))[:, None]
            x = x.masked_fill(~seen, -math.inf)
            top = x.amax(-1, keepdim=True) if n else x.new_full((m, 1), -math.inf)
            p = torch.exp(x - torch.where(top.isinf(), torch.zeros_like(top), top))
            l = p.sum(-1, keepdim=True)
            p = torch.where(l > 0, p / l, torch.zeros_like(p))
            out[r0:r0 + m, j] = p @ v
            spread[r0:r0 + m, j] = p @ v.abs()
            lse[r0:r0 + m, j] = (l.log() + torch.where(top.isinf(), torch.zeros_like(top), top))[:, 0]
            slack[r0:r0 + m, j] = ab.masked_fill(~seen, 0).amax(-1) if n else 0
    return out, lse, spread, slack


def weights(q, lse, cu, kv, keys, table, scores):
    """Scores after the call in float64, and the largest sum of |q k| / sqrt(d) of each slot."""
    total, hq, d = q.shape
    kv_heads = scores.shape[1]
    out, slack = scores.double(), torch.zeros_like(scores.double())
    for b, n in enumerate(kv):
        m, r0 = cu[b + 1] - cu[b], cu[b]
        if n == 0 or m == 0:
            continue
        for j in range(hq):
            h = j // (hq // kv_heads)
            k = gather(keys, table, b, h, n)
            x = q[r0:r0 + m, j].double() @ k.T / math.sqrt(d)
            ab = q[r0:r0 + m, j].double().abs() @ k.abs().T / math.sqrt(d)
            seen = torch.arange(n, device=q.device)[None] <= (n - m + torch.arange(m, device=q.device))[:, None]
            p = torch.where(seen, torch.exp(x - lse[r0:r0 + m, j].double()[:, None]), torch.zeros_like(x))
            out[b, h, :n] += p.sum(0)
            slack[b, h, :n] = torch.maximum(slack[b, h, :n], ab.amax(0))
    return out, slack


def rotate(x, w, eps, inv_freq, pos, rot, interleaved):
    """Norm and rotation of [rows, heads, d] in float64, and the norm of each element's pair."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()
    y, size = x.clone(), x.abs()
    i = torch.arange(rot // 2, device=x.device)
    a, c = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    t = pos.double()[:, None] * inv_freq.double()[None]
    cos, sin = torch.cos(t)[:, None], torch.sin(t)[:, None]
    y[..., a] = x[..., a] * cos - x[..., c] * sin
    y[..., c] = x[..., c] * cos + x[..., a] * sin
    size[..., a] = size[..., c] = torch.hypot(x[..., a], x[..., c])
    return y, size


def keep(score, n, n_sink, window, budget):
    """Slots kept of one head, ascending: by the definition, with Python's own sort."""
    if n <= budget:
        return list(range(n))
    s = score[:n].tolist()
    value = [(-math.inf, 0) if math.isnan(x) else (x, 1) for x in s]
    middle = sorted(range(n_sink, n - window), key=lambda i: (-value[i][0], -value[i][1], i))
    sure = list(range(n_sink)) + list(range(n - window, n))
    return sorted(sure + middle[:budget - n_sink - window])
