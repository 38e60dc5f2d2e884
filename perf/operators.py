"""Cases and plain forms of the operators around a key/value cache.

A serving loop fills the cache that the sampled decode attention reads: it normalises
and rotates the new tokens' queries and keys and writes keys and values into the cache
(`append`), attends from the new tokens to everything before them (`attend`), adds up
how much attention every cached key received (`weights`), and keeps only the keys that
received most of it once the cache is over its budget (`evict`).

The cache of one layer is a pool of pages [n_pages][kv_heads][page_size][head_dim] and a
table of page numbers per sequence; without a table, page b is the whole cache of
sequence b, which is one layer of the dense layout [batch][kv_heads][capacity][head_dim].
New tokens lie packed: those of sequence b are rows cu_q[b] to cu_q[b + 1]; token i of a
chunk of m tokens sits in cache slot kv_len[b] - m + i and sees the slots up to its own.

`run` computes a case in its plain form, or, with `own` set, by the library's calls.
"""
import math

import torch

own = False

THETA = 500000.0  # base of the rotation's frequencies
EPS = 1e-6


# ----------------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------------

def _case(name, op, dtype, heads, d, page, q_lens, kv_lens, **more):
    c = {"op": op, "dtype": dtype, "q_heads": heads[0], "kv_heads": heads[1], "d": d, "page": page,
         "q_lens": ",".join(map(str, q_lens)), "kv_lens": ",".join(map(str, kv_lens))}
    c.update(more)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one generated token for each of 16 sequences deep in their contexts: latency
        _case("append_step_b16", "append", "bf16", (32, 8), 128, 64, [1] * 16, [16000 + 331 * i for i in range(16)],
              rot=128, interleaved=False),
        # a long prompt's chunk into a dense cache: bandwidth
        _case("append_prompt_8k", "append", "bf16", (32, 8), 128, 0, [8192], [8192], rot=128, interleaved=False),
        # ragged prompts in fp32, half of each head rotated, pairs next to each other
        _case("append_ragged_f32", "append", "f32", (8, 4), 64, 16, [1, 517, 33, 1200, 250], [9, 517, 700, 1331, 4000],
              rot=32, interleaved=True),
        # one token over a short cache: latency
        _case("attend_step_2k", "attend", "bf16", (32, 8), 128, 0, [1], [2048]),
        # one token each over four long dense caches of the 64-head shape: bandwidth
        _case("attend_step_b4_96k", "attend", "bf16", (64, 8), 128, 0, [1] * 4, [98304, 90001, 98304, 81920]),
        # a chunk of a long prompt over the pages written so far: matrix rate
        _case("attend_chunk_2k_32k", "attend", "bf16", (32, 8), 128, 64, [2048], [32768]),
        # a batch of odd chunks and single tokens together, heads of 64, short pages
        _case("attend_ragged_d64", "attend", "bf16", (16, 4), 64, 16, [1, 700, 33, 1, 257, 5, 128],
              [3001, 700, 1999, 9000, 4100, 77, 128]),
        # full-precision chunk over a short cache
        _case("attend_chunk_f32", "attend", "f32", (8, 8), 64, 0, [500], [2048]),
        # attention received by the keys of one long cache from one token
        _case("weights_step_64k", "weights", "bf16", (32, 8), 128, 64, [1], [65536]),
        # attention received from the last chunk of a prompt
        _case("weights_chunk_1k_16k", "weights", "bf16", (32, 8), 128, 0, [1000], [16384]),
        # a long dense cache cut to an eighth
        _case("evict_96k_to_12k", "evict", "bf16", (32, 8), 128, 0, [1], [98304], budget=12288, n_sink=4, window=64),
        # a paged batch of short caches, some already within the budget
        _case("evict_paged_b6", "evict", "f32", (8, 4), 64, 32, [1] * 6, [2000, 777, 1024, 1025, 1500, 4097],
              budget=1000, n_sink=4, window=64),
    ]


_HEADS = ((1, 1), (8, 8), (6, 2), (16, 4), (28, 4), (32, 8), (64, 8), (40, 40), (12, 1))
_PAGES = (0, 0, 16, 32, 48, 64, 128, 256)


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("append", "attend", "attend", "weights", "evict"))
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    heads, d, page = rng.choice(_HEADS), rng.choice((64, 128, 128)), rng.choice(_PAGES)
    small = 1 if dtype == "bf16" else 4
    if op == "append":
        total = _log(rng, 1, 8192 * 32 * 128 // (heads[0] * d) // small // 2 + 1)
        total = min(total, 16384)
        batch = min(total, _log(rng, 1, 32))
        q = [total // batch + (i < total % batch) for i in range(batch)]
        kv = [m + rng.randint(0, 4000) for m in q]
        return _case(None, op, dtype, heads, d, page, q, kv, rot=rng.choice((d, d, d // 2, 16)),
                     interleaved=rng.random() < 0.5)
    if op == "evict":
        batch = _log(rng, 1, 8)
        top = max(64, min(131072, 98304 * 8 // (batch * heads[1]) // small))
        n = _log(rng, 16, top)
        kv = [max(1, n - rng.randint(0, n // 3)) for _ in range(batch)]
        return _case(None, op, dtype, heads, d, page, [1] * batch, kv, budget=max(8 if n < 512 else 72, int(n * rng.uniform(0.05, 0.6))),
                     n_sink=rng.choice((0, 4)), window=rng.choice((0, 1, 3)) if n < 512 else rng.choice((0, 24, 64)))
    kind = rng.choice(("step", "step", "draft", "chunk", "ragged"))
    if kind == "step":
        batch = _log(rng, 1, 16)
        top = max(32, min(131072, 4 * 8 * 90000 // (batch * heads[1]) // small))
        kv = [max(1, n - rng.randint(0, n // 4)) for n in [_log(rng, 1, top)] * batch]
        q = [1] * batch
    elif kind == "draft":
        batch = _log(rng, 1, 8)
        q = [rng.randint(2, 12) for _ in range(batch)]
        top = max(32, min(65536, 2 * 8 * 90000 // (batch * heads[1]) // small))
        kv = [m + _log(rng, 1, top) for m in q]
    else:
        batch = 1 if kind == "chunk" else rng.randint(2, 7)
        q = [_log(rng, 1, 2048 // small // batch + 1) for _ in range(batch)]
        # rows x heads x keys, padded to the longest chunk and the longest cache
        room = 2048 * 32 * 32768 // ((2 if kind == "chunk" else 8) * small * small)
        top = max(64, min(32768, room // (batch * heads[0] * max(q))))
        kv = [m + rng.randint(0, top) for m in q]
    return _case(None, op, dtype, heads, d, page, q, kv)


# ----------------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------------

def _lens(text):
    return [int(x) for x in text.split(",")]


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _pool(case, lens, cap=0):
    """(page size, pages per sequence, pages in the pool) of a cache that holds `lens`."""
    if case["page"] == 0:
        return max(max(lens), cap), 1, len(lens)
    ps = case["page"]
    return ps, -(-max(lens) // ps), sum(-(-n // ps) for n in lens) + 3


def _table(case, lens, gen, dev):
    """A page table whose pages are in no order; numbers behind a sequence's end are never looked at."""
    if case["page"] == 0:
        return None
    ps, cols, pages = _pool(case, lens)
    order = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
    need = torch.tensor([-(-n // ps) for n in lens], device=dev)
    first = torch.cumsum(need, 0) - need
    col = torch.arange(cols, device=dev)
    at = (first[:, None] + col).clamp(max=pages - 1)
    return torch.where(col < need[:, None], order[at], torch.zeros_like(order[at])).contiguous()


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    dt = _dtype(case)
    q_lens, kv_lens = _lens(case["q_lens"]), _lens(case["kv_lens"])
    hq, hk, d, op = case["q_heads"], case["kv_heads"], case["d"], case["op"]
    ps, cols, pages = _pool(case, kv_lens)
    total = sum(q_lens)
    cu = [0]
    for m in q_lens:
        cu.append(cu[-1] + m)

    def normal(*shape, by=1.0):
        return (torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32) * by).to(dt)

    s = {"case": dict(case), "op": op, "ps": ps, "cols": cols, "pages": pages, "max_q": max(q_lens), "max_kv": max(kv_lens),
         "cu_q": torch.tensor(cu, dtype=torch.int32, device=dev),
         "kv_len": torch.tensor(kv_lens, dtype=torch.int32, device=dev),
         "table": _table(case, kv_lens, gen, dev),
         "keys": normal(pages, hk, ps, d), "status": torch.zeros(1, dtype=torch.int32, device=dev)}
    if op != "weights":
        s["values"] = normal(pages, hk, ps, d)
    if op == "append":
        # queries, keys and values as a fused projection leaves them, in one row per token
        qkv = normal(total, (hq + 2 * hk) * d, by=1.7)
        s["q"] = qkv[:, :hq * d].unflatten(1, (hq, d))
        s["k"] = qkv[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d))
        s["v"] = qkv[:, (hq + hk) * d:].unflatten(1, (hk, d))
        s["q_norm"], s["k_norm"] = (1 + 0.2 * normal(d).float()).to(dt), (1 + 0.2 * normal(d).float()).to(dt)
        half = torch.arange(case["rot"] // 2, device=dev, dtype=torch.float64)
        s["inv_freq"] = THETA ** (-2.0 * half / case["rot"])
        # where a token stands in its text: later than its slot once keys were evicted
        later = torch.randint(0, 100000, (len(q_lens),), generator=gen, device=dev)
        row = torch.arange(total, device=dev)
        b = torch.searchsorted(s["cu_q"][1:].long(), row, right=True)
        s["positions"] = (later[b] + (s["kv_len"] - s["cu_q"][1:])[b] + row).to(torch.int32)
        s["q_out"] = torch.empty(total, hq, d, dtype=dt, device=dev)
    if op in ("attend", "weights"):
        s["q"] = normal(total, hq, d, by=1.5)
        s["lse"] = torch.empty(total, hq, dtype=torch.float32, device=dev)
    if op == "attend":
        s["out"] = torch.empty(total, hq, d, dtype=dt, device=dev)
    if op == "weights":
        s["lse"] = _lse(s)
        # what the tokens before have added, of the size that this chunk adds
        s["scores"] = torch.rand(len(kv_lens), hk, cols * ps, generator=gen, device=dev) * (hq // hk * max(q_lens) / max(kv_lens))
    if op == "evict":
        # a few keys hold most of the attention, and the newest have none yet
        sc = torch.randn(len(kv_lens), hk, cols * ps, generator=gen, device=dev).mul_(2.0).exp_()
        sc[torch.rand(sc.shape, generator=gen, device=dev) < 0.05] = 0.0
        s["scores"] = sc
        new = [min(n, case["budget"]) for n in kv_lens]
        s["dps"], s["dcols"], s["dpages"] = _pool(case, new, cap=case["budget"])
        s["dtable"] = _table(case, new, gen, dev)
        s["dkeys"] = torch.zeros(s["dpages"], hk, s["dps"], d, dtype=dt, device=dev)
        s["dvalues"] = torch.zeros_like(s["dkeys"])
        s["dscores"] = torch.zeros(len(kv_lens), hk, s["dcols"] * s["dps"], device=dev)
        s["dlen"] = torch.zeros(len(kv_lens), dtype=torch.int32, device=dev)
        s["kept"] = torch.full((len(kv_lens), hk, case["budget"]), -1, dtype=torch.int32, device=dev)
    return s


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    q_lens, kv_lens = _lens(case["q_lens"]), _lens(case["kv_lens"])
    hq, hk, d, op = case["q_heads"], case["kv_heads"], case["d"], case["op"]
    total = sum(q_lens)
    # (query, key) pairs that the mask leaves
    pairs = sum(m * n - m * (m - 1) // 2 for m, n in zip(q_lens, kv_lens))
    if op == "append":
        # square, sum and scale of each normed value, and the rotation's four products and two sums a pair
        return {"bytes": 2 * total * (hq + 2 * hk) * d * es + 4 * total,
                "flops": total * (hq + hk) * (4 * d + 3 * case["rot"])}
    if op == "attend":
        return {"bytes": 2 * total * hq * d * es + 4 * total * hq + 2 * sum(kv_lens) * hk * d * es, "flops": 4 * d * hq * pairs}
    if op == "weights":
        return {"bytes": total * hq * (d * es + 4) + sum(kv_lens) * hk * (d * es + 8), "flops": 2 * d * hq * pairs}
    new = [min(n, case["budget"]) for n in kv_lens]
    return {"bytes": hk * (4 * sum(kv_lens) + sum(new) * (4 * d * es + 8)), "flops": hk * sum(kv_lens)}


# ----------------------------------------------------------------------------------
# plain forms
# ----------------------------------------------------------------------------------

def _dense(s, pool, n):
    """[batch, kv_heads, n, d] of a pool's pages in the order of the sequences."""
    if s["table"] is None:
        return pool[:, :, :n]
    b, (_, hk, ps, d) = s["table"].shape[0], pool.shape
    return pool[s["table"].long()].transpose(1, 2).reshape(b, hk, s["cols"] * ps, d)[:, :, :n]


def _padded(s):
    """Rows of the packed tokens laid out [batch, max_q], clipped where a sequence has fewer, and each token's (batch, index)."""
    cu, m = s["cu_q"].long(), s["max_q"]
    at = (cu[:-1, None] + torch.arange(m, device=cu.device)).clamp(max=s["q"].shape[0] - 1)
    row = torch.arange(s["q"].shape[0], device=cu.device)
    b = torch.searchsorted(cu[1:], row, right=True)
    return at, b, row - cu[b]


def _logits(s):
    """fp32 logits [batch, kv_heads, group, max_q, n] with -inf where a key is not seen, and the seen (query, key) pairs."""
    c = s["case"]
    hq, hk, d, n, m = c["q_heads"], c["kv_heads"], c["d"], s["max_kv"], s["max_q"]
    at, _, _ = _padded(s)
    q = s["q"][at].float().unflatten(2, (hk, hq // hk)).permute(0, 2, 3, 1, 4)
    k = _dense(s, s["keys"], n).float()
    x = torch.matmul(q.reshape(q.shape[0], hk, hq // hk * m, d), k.transpose(2, 3)).mul_(1.0 / math.sqrt(d))
    x = x.unflatten(2, (hq // hk, m))
    cu, slot = s["cu_q"], torch.arange(n, device=k.device)
    i = torch.arange(m, device=k.device)
    own_slot = (s["kv_len"] - (cu[1:] - cu[:-1]))[:, None] + i
    seen = (slot <= own_slot[:, :, None]) & (i < (cu[1:] - cu[:-1])[:, None])[:, :, None]
    seen = seen[:, None, None]
    return x.masked_fill_(~seen, -math.inf), seen


def _lse(s):
    x, _ = _logits(s)
    top = x.amax(-1, keepdim=True).clamp(min=-3e38)
    lse = x.sub_(top).exp_().sum(-1).log() + top[..., 0]
    _, b, i = _padded(s)
    return lse.permute(0, 3, 1, 2).flatten(2)[b, i].contiguous()


def _plain_attend(s):
    c = s["case"]
    x, _ = _logits(s)
    top = x.amax(-1, keepdim=True).clamp(min=-3e38)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    slot = torch.arange(s["max_kv"], device=x.device)
    v = _dense(s, s["values"], s["max_kv"]).float()
    v = torch.where((slot < s["kv_len"][:, None])[:, None, :, None], v, torch.zeros((), device=v.device))
    o = torch.matmul(p.flatten(2, 3), v).unflatten(2, (c["q_heads"] // c["kv_heads"], s["max_q"]))
    o = o / total.clamp(min=1e-38)
    lse = total[..., 0].log() + top[..., 0]
    _, b, i = _padded(s)
    o = o.permute(0, 3, 1, 2, 4).flatten(2, 3)[b, i]
    return {"out": o.to(s["q"].dtype), "lse": lse.permute(0, 3, 1, 2).flatten(2)[b, i]}


def _plain_weights(s):
    c = s["case"]
    x, seen = _logits(s)
    at, _, _ = _padded(s)
    lse = s["lse"][at].unflatten(2, (c["kv_heads"], -1)).permute(0, 2, 3, 1)
    p = torch.where(seen, x.sub_(lse[..., None]).exp_(), torch.zeros((), device=x.device))
    s["scores"][:, :, :s["max_kv"]] += p.sum((2, 3))
    return {"scores": s["scores"]}


def _rotate(x, cos, sin, rot, interleaved):
    x1, x2 = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    y1, y2 = x1 * cos - x2 * sin, x2 * cos + x1 * sin
    y = torch.stack((y1, y2), -1).flatten(-2) if interleaved else torch.cat((y1, y2), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _plain_append(s):
    c = s["case"]
    angle = s["positions"].double()[:, None] * s["inv_freq"]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def normed(x, w):
        x = x.float()
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
        return _rotate(x, cos, sin, c["rot"], c["interleaved"]).to(s["keys"].dtype)

    cu = s["cu_q"].long()
    row = torch.arange(s["q"].shape[0], device=cu.device)
    b = torch.searchsorted(cu[1:], row, right=True)
    slot = s["kv_len"].long()[b] - cu[b + 1] + row
    page = b if s["table"] is None else s["table"].long()[b, slot // s["ps"]]
    s["keys"][page, :, slot % s["ps"]] = normed(s["k"], s["k_norm"])
    s["values"][page, :, slot % s["ps"]] = s["v"]
    s["q_out"] = normed(s["q"], s["q_norm"])
    return {"q": s["q_out"], "keys": s["keys"], "values": s["values"]}


def _plain_evict(s):
    c = s["case"]
    n, budget = s["max_kv"], c["budget"]
    slot = torch.arange(n, device=s["keys"].device)
    length = s["kv_len"].long()[:, None, None]
    score = s["scores"][:, :, :n]
    sure = (slot < c["n_sink"]) | (slot >= length - c["window"])
    # the first `budget` of the slots ordered by (within the length, always kept, score), ties by slot
    rank = torch.where(slot < length, torch.where(sure, torch.full_like(score, math.inf), score), torch.full_like(score, -math.inf))
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :budget]
    new = torch.clamp(s["kv_len"].long(), max=budget)
    i = torch.arange(order.shape[-1], device=order.device)
    live = (i < new[:, None, None]).expand_as(order)
    kept = torch.sort(torch.where(live, order, torch.full_like(order, n)), dim=-1).values
    b, h, j = torch.nonzero(live, as_tuple=True)
    src = kept[b, h, j]
    page = b if s["table"] is None else s["table"].long()[b, src // s["ps"]]
    to = b if s["dtable"] is None else s["dtable"].long()[b, j // s["dps"]]
    s["dkeys"][to, h, j % s["dps"]] = s["keys"][page, h, src % s["ps"]]
    s["dvalues"][to, h, j % s["dps"]] = s["values"][page, h, src % s["ps"]]
    s["dscores"][b, h, j] = score[b, h, src]
    s["kept"][b, h, j] = src.to(torch.int32)
    s["dlen"] = new.to(torch.int32)
    return {"keys": s["dkeys"], "values": s["dvalues"], "scores": s["dscores"], "kept": s["kept"], "len": s["dlen"]}


# ----------------------------------------------------------------------------------
# the library's calls
# ----------------------------------------------------------------------------------

def _own_run(s):
    import lsh_sampled_sparse_centered_gb300 as mp
    c, op = s["case"], s["op"]
    cfg = s.get("cfg")
    if cfg is None:  # the configuration and the workspace that a program makes once
        shape = dict(batch=len(_lens(c["kv_lens"])), kv_heads=c["kv_heads"], q_heads=c["q_heads"], head_dim=c["d"], dtype=c["dtype"])
        cfg = s["cfg"] = mp.make_cache_config(page_size=s["ps"], n_pages=s["pages"], max_pages=s["cols"], **shape)
        if op == "append":
            s["rotary"] = mp.make_rotary(rot_dim=c["rot"], interleaved=c["interleaved"], eps=EPS)
        if op == "attend":
            size = mp.mp_chunk_workspace_bytes(cfg, s["q"].shape[0], s["max_q"], s["max_kv"])
            s["workspace"] = torch.empty(size, dtype=torch.uint8, device=s["q"].device)
        if op == "evict":
            s["dcfg"] = mp.make_cache_config(page_size=s["dps"], n_pages=s["dpages"], max_pages=s["dcols"], **shape)
            size = mp.mp_evict_workspace_bytes(cfg, s["max_kv"], c["budget"])
            s["workspace"] = torch.empty(size, dtype=torch.uint8, device=s["keys"].device)
    if op == "append":
        mp.mp_cache_append(cfg, s["rotary"], s["q"], s["k"], s["v"], s["q_norm"], s["k_norm"], s["inv_freq"], s["positions"],
                           s["cu_q"], s["kv_len"], s["keys"], s["values"], s["table"], s["q_out"], s["status"])
        return {"q": s["q_out"], "keys": s["keys"], "values": s["values"]}
    if op == "attend":
        mp.mp_chunk_attention(cfg, s["q"], s["cu_q"], s["kv_len"], s["max_q"], s["max_kv"], s["keys"], s["values"], s["table"],
                              s["out"], s["lse"], s["workspace"], s["status"])
        return {"out": s["out"], "lse": s["lse"]}
    if op == "weights":
        mp.mp_cache_weights(cfg, s["q"], s["lse"], s["cu_q"], s["kv_len"], s["max_q"], s["max_kv"], s["keys"], s["table"], s["scores"],
                            s["status"])
        return {"scores": s["scores"]}
    mp.mp_cache_evict(cfg, s["dcfg"], s["keys"], s["values"], s["table"], s["kv_len"], s["max_kv"], s["scores"], c["n_sink"], c["window"],
                      c["budget"], s["dkeys"], s["dvalues"], s["dtable"], s["dscores"], s["dlen"], s["kept"], s["workspace"], s["status"])
    return {"keys": s["dkeys"], "values": s["dvalues"], "scores": s["dscores"], "kept": s["kept"], "len": s["dlen"]}


def run(state):
    if own:
        return _own_run(state)
    return {"append": _plain_append, "attend": _plain_attend, "weights": _plain_weights, "evict": _plain_evict}[state["op"]](state)


# ----------------------------------------------------------------------------------
# the definitions in 64 bits
# ----------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    q_lens, kv_lens = _lens(case["q_lens"]), _lens(case["kv_lens"])
    hq, hk, d, ps, op = case["q_heads"], case["kv_heads"], case["d"], s["ps"], case["op"]
    table = s["table"].cpu().tolist() if s["table"] is not None else [[b] for b in range(len(kv_lens))]
    total = sum(q_lens)

    def rows(pool, b, h, n, per, pages):
        return torch.cat([pool[pages[b][j], h, :min(per, n - j * per)] for j in range(-(-n // per))])

    if op in ("attend", "weights"):
        out = torch.zeros(total, hq, d, dtype=torch.float64, device="cuda")
        lse = torch.zeros(total, hq, dtype=torch.float64, device="cuda")
        scores = s["scores"].double() if op == "weights" else None
        t0 = 0
        for b, (m, n) in enumerate(zip(q_lens, kv_lens)):
            for j in range(hq):
                h = j // (hq // hk)
                k = rows(s["keys"], b, h, n, ps, table).double()
                for u in range(0, m, 512):
                    e = min(m, u + 512)
                    x = (s["q"][t0 + u:t0 + e, j].double() @ k.T) / d ** 0.5
                    limit = torch.arange(n - m + u, n - m + e, device="cuda")
                    x = x + torch.where(torch.arange(n, device="cuda") > limit[:, None], -math.inf, 0.0).double()
                    if op == "weights":
                        scores[b, h, :n] += torch.exp(x - s["lse"][t0 + u:t0 + e, j].double()[:, None]).sum(0)
                        continue
                    z = torch.logsumexp(x, -1)
                    lse[t0 + u:t0 + e, j] = z
                    out[t0 + u:t0 + e, j] = torch.exp(x - z[:, None]) @ rows(s["values"], b, h, n, ps, table).double()
            t0 += m
        return {"scores": scores} if op == "weights" else {"out": out, "lse": lse}

    if op == "append":
        rot, keys, values = case["rot"], s["keys"].double(), s["values"].double()
        first = torch.arange(0, rot, 2, device="cuda") if case["interleaved"] else torch.arange(rot // 2, device="cuda")
        second = first + (1 if case["interleaved"] else rot // 2)
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                           s["positions"].double()[:, None] * s["inv_freq"][None])[:, None]

        def turned(x, w):
            x = x.double()
            x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / d + EPS) * w.double()
            z = torch.complex(x[..., first], x[..., second]) * turn
            x[..., first], x[..., second] = z.real, z.imag
            return x

        kk, t0 = turned(s["k"], s["k_norm"]), 0
        for b, (m, n) in enumerate(zip(q_lens, kv_lens)):
            at = n - m
            while at < n:
                end = min(n, (at // ps + 1) * ps)
                t, page, o = t0 + at - (n - m), table[b][at // ps], at % ps
                keys[page, :, o:o + end - at] = kk[t:t + end - at].transpose(0, 1)
                values[page, :, o:o + end - at] = s["v"][t:t + end - at].transpose(0, 1).double()
                at = end
            t0 += m
        return {"q": turned(s["q"], s["q_norm"]), "keys": keys, "values": values}

    budget, dps = case["budget"], s["dps"]
    to = s["dtable"].cpu().tolist() if s["dtable"] is not None else [[b] for b in range(len(kv_lens))]
    scores, kept = s["dscores"].double(), s["kept"].clone()
    keys, values = s["dkeys"].double(), s["dvalues"].double()
    for b, n in enumerate(kv_lens):
        for h in range(hk):
            live = s["scores"][b, h, :n]
            keep = torch.ones(n, dtype=torch.bool, device="cuda")
            if n > budget:
                low, high = case["n_sink"], n - case["window"]
                want = budget - case["n_sink"] - case["window"]
                middle = live[low:high]
                edge = torch.sort(middle).values[len(middle) - want] if want else math.inf
                keep[low:high] = middle > edge
                tied = torch.nonzero(middle == edge)[:, 0]
                keep[low + tied[:want - int((middle > edge).sum())]] = True
            at = torch.nonzero(keep)[:, 0]
            m = len(at)
            kept[b, h, :m] = at.to(torch.int32)
            scores[b, h, :m] = live[at].double()
            k, v = rows(s["keys"], b, h, n, ps, table)[at], rows(s["values"], b, h, n, ps, table)[at]
            for j in range(-(-m // dps)):
                e = min(m, (j + 1) * dps)
                keys[to[b][j], h, :e - j * dps] = k[j * dps:e].double()
                values[to[b][j], h, :e - j * dps] = v[j * dps:e].double()
    return {"keys": keys, "values": values, "scores": scores, "kept": kept,
            "len": torch.tensor([min(n, budget) for n in kv_lens], dtype=torch.int32, device="cuda")}
