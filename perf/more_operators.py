"""Cases and plain forms of the operators that plan, share and move a key/value cache.

A serving loop decides per step by how many tokens each sequence grows or is rolled back,
and from that come the page tables, the packed rows and where each of them goes (`plan`).
Sequences that begin with the same long text keep its keys and values once and attend to
them together (`prefix`). Keys that have moved to other positions, or whose frequencies
were scaled for a longer context, are turned to where they now stand (`rotate`).

The cache of one layer is a pool of pages [n_pages][kv_heads][page_size][head_dim] and a
table of page numbers per sequence; without a table, page b is the whole cache of
sequence b. New tokens lie packed: those of sequence b are rows cu_q[b] to cu_q[b + 1]; token i
of a chunk of m tokens sits in cache slot kv_len[b] - m + i and sees its sequence's own slots
up to that one, and the whole prefix of its group: group g are the sequences cu_group[g] to
cu_group[g + 1], those behind the last group have no prefix.

`run` computes a case in its plain form, or, with `own` set, by the library's calls.
"""
import math

import torch

own = False

THETA = 500000.0  # base of the rotation's frequencies


# ----------------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------------

def _text(numbers):
    return ",".join(map(str, numbers))


def _lens(text):
    return [int(x) for x in text.split(",")] if text else []


def _plan(name, batch, page, low, high, kinds, prompt=0, scarce=False):
    """`batch` sequences of low..high slots. kinds: shares, in percent, of those that grow by one token, grow
    by a prompt's chunk of up to `prompt` tokens, are rolled back by a few, have ended, and wait.
    scarce: too few pages are free, so that the last of them have to wait."""
    c = {"op": "plan", "batch": batch, "page": page, "low": low, "high": high, "kinds": _text(kinds), "prompt": prompt, "scarce": scarce}
    if name:
        c["name"] = name
    return c


def _prefix(name, dtype, heads, d, page, groups, q_lens, kv_lens):
    """groups: (sequences, prefix length) of each group."""
    c = {"op": "prefix", "dtype": dtype, "q_heads": heads[0], "kv_heads": heads[1], "d": d, "page": page,
         "sequences": _text(n for n, _ in groups), "prefixes": _text(p for _, p in groups),
         "q_lens": _text(q_lens), "kv_lens": _text(kv_lens)}
    if name:
        c["name"] = name
    return c


def _rotate(name, dtype, kv_heads, d, page, kv_lens, kind, rot, interleaved):
    """kind: `evicted` (each head kept other slots and they move up), `scaled` (the frequencies change, the positions
    stay) or `moved` (a whole sequence starts elsewhere)."""
    c = {"op": "rotate", "dtype": dtype, "kv_heads": kv_heads, "d": d, "page": page, "kv_lens": _text(kv_lens), "kind": kind,
         "rot": rot, "interleaved": interleaved}
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one more token for each of 64 running sequences: latency
        _plan("plan_step_b64", 64, 64, 200, 16000, (100, 0, 0, 0, 0)),
        # a busy step of a large batch: most decode, some take prompt chunks, drafts are rolled back, some end
        _plan("plan_mixed_b1000", 1000, 16, 1, 4000, (70, 8, 10, 6, 6), prompt=700),
        # four short answers to one system prompt: latency
        _prefix("prefix_step_b4_2k", "bf16", (32, 8), 128, 64, [(4, 2048)], [1] * 4, [17, 64, 120, 200]),
        # 32 samples of one long prompt: bandwidth
        _prefix("prefix_step_b32_32k", "bf16", (32, 8), 128, 64, [(32, 32768)], [1] * 32, [100 + 29 * i for i in range(32)]),
        # 128 questions about one very long document: matrix rate over the prefix, bandwidth over their own slots
        _prefix("prefix_step_b128_96k", "bf16", (32, 8), 128, 0, [(128, 98304)], [1] * 128, [64 + 13 * i for i in range(128)]),
        # three system prompts in one batch and sequences without one; drafts of a few tokens, odd lengths, short pages
        _prefix("prefix_groups_d64", "bf16", (16, 4), 64, 16, [(5, 3001), (9, 777), (1, 5000)],
                [1, 5, 3, 1, 4, 1, 1, 6, 2, 1, 1, 3, 1, 1, 5, 1, 4], [33, 205, 3, 1000, 64, 77, 1, 300, 450, 16, 15, 400, 90, 700, 5, 2100, 99]),
        # the first chunks of six questions about one document: matrix rate
        _prefix("prefix_chunks_16k", "bf16", (32, 8), 128, 64, [(6, 16384)], [100, 517, 64, 300, 33, 250], [100, 517, 64, 300, 900, 250]),
        # full precision, some tokens each over a short prefix
        _prefix("prefix_chunk_f32", "f32", (8, 8), 64, 0, [(5, 2000)], [20, 1, 33, 7, 40], [20, 300, 33, 150, 40]),
        # a cut cache whose kept keys move up, other slots in every head: bandwidth
        _rotate("rotate_evicted_12k", "bf16", 8, 128, 0, [12288] * 4, "evicted", 128, False),
        # a long cache whose frequencies are scaled for a longer context: bandwidth
        _rotate("rotate_scaled_96k", "bf16", 8, 128, 64, [98304], "scaled", 128, False),
        # a paged batch of short caches, half of each head rotated, pairs next to each other
        _rotate("rotate_moved_f32", "f32", 4, 64, 16, [9, 517, 700, 1331, 4000], "moved", 32, True),
    ]


_HEADS = ((1, 1), (8, 8), (6, 2), (16, 4), (28, 4), (32, 8), (64, 8), (40, 40), (12, 1))
_PAGES = (0, 0, 16, 32, 48, 64, 128, 256)


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("plan", "prefix", "prefix", "prefix", "rotate"))
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    heads, d, page = rng.choice(_HEADS), rng.choice((64, 128, 128)), rng.choice(_PAGES)
    small = 1 if dtype == "bf16" else 4
    if op == "plan":
        batch = _log(rng, 1, 1000)
        cuts = sorted(rng.randint(0, 100) for _ in range(4))
        kinds = [b - a for a, b in zip([0] + cuts, cuts + [100])]
        low = _log(rng, 1, 2000)
        return _plan(None, batch, rng.choice((16, 32, 48, 64, 128, 256)), low, low + _log(rng, 1, 2000), kinds, prompt=_log(rng, 1, 700),
                     scarce=rng.random() < 0.2)
    if op == "rotate":
        batch = _log(rng, 1, 8)
        n = _log(rng, 1, max(16, min(131072, 98304 * 8 * 128 // (batch * heads[1] * d) // small)))
        kv = [max(1, n - rng.randint(0, n // 3)) for _ in range(batch)]
        return _rotate(None, dtype, heads[1], d, page, kv, rng.choice(("evicted", "scaled", "moved")), rng.choice((d, d, d // 2, 16)),
                       rng.random() < 0.5)
    kind = rng.choice(("step", "step", "draft", "chunk"))
    n_groups = rng.choice((1, 1, 1, 2, 3, 5))
    if kind == "chunk":
        sizes = [rng.randint(1, 4) for _ in range(n_groups)]
    else:
        sizes = [max(1, _log(rng, 1, 128) // n_groups) for _ in range(n_groups)]
    loose = rng.choice((0, 0, 1, 3))  # sequences behind the last group
    batch = sum(sizes) + loose
    most = {"step": 1, "draft": 9, "chunk": max(1, 1200 // small // batch)}[kind]
    q = [rng.randint(1, most) if kind != "chunk" else _log(rng, 1, most) for _ in range(batch)]
    # rows x heads x slots of the prefixes, and bytes of the own slots
    room = 128 * 32 * 98304 * 128 // (heads[0] * d) // (small * small)
    top = max(16, min(98304, room // max(1, sum(q)), 2 * 98304 * 8 // heads[1]))
    prefixes = [rng.choice((0, 1, top)) if rng.random() < 0.1 else _log(rng, 1, top) for _ in range(n_groups)]
    top = max(8, min(2000, 128 * 8 * 900 // (batch * heads[1]) // small, room // (heads[0] * max(q) * batch)))
    kv = [m + rng.randint(0, top) for m in q]
    return _prefix(None, dtype, heads, d, page, list(zip(sizes, prefixes)), q, kv)


# ----------------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------------

def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _pool(page, lens):
    """(page size, pages per sequence, pages in the pool) of a cache that holds `lens`."""
    if page == 0:
        return max(1, max(lens)), 1, len(lens)
    return page, max(1, -(-max(lens) // page)), sum(-(-n // page) for n in lens) + 3


def _table(order, lens, page, cols, skip=0):
    """Page tables of sequences of `lens` from the pages order[skip:]; numbers behind a sequence's end are zero."""
    need = torch.tensor([-(-n // page) for n in lens], device=order.device)
    first = torch.cumsum(need, 0) - need + skip
    col = torch.arange(cols, device=order.device)
    at = (first[:, None] + col).clamp(max=order.numel() - 1)
    return torch.where(col < need[:, None], order[at], torch.zeros_like(order[at])).contiguous()


def _ints(numbers, dev):
    return torch.tensor(list(numbers), dtype=torch.int32, device=dev)


def _offsets(numbers, dev):
    at = [0]
    for n in numbers:
        at.append(at[-1] + n)
    return _ints(at, dev)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    return {"plan": _prepare_plan, "prefix": _prepare_prefix, "rotate": _prepare_rotate}[case["op"]](case, gen, dev)


def _prepare_plan(case, gen, dev):
    batch, ps = case["batch"], case["page"]

    def number(low, high, n=batch):  # low..high of each
        return low + (torch.rand(n, generator=gen, device=dev) * (high - low + 1)).long().clamp(max=high - low)

    kv = number(case["low"], case["high"])
    kind = torch.multinomial(torch.tensor([k + 1e-3 for k in _lens(case["kinds"])], device=dev), batch, replacement=True, generator=gen)
    change = torch.where(kind == 0, torch.ones_like(kv), torch.zeros_like(kv))
    if case["prompt"]:
        change = torch.where(kind == 1, number(1, case["prompt"]), change)
    change = torch.where(kind == 2, -number(1, 8), change)
    change = torch.where(kind == 3, -kv, change)
    cap = case["high"] + max(1, case["prompt"])
    cols = -(-cap // ps)
    pages = batch * cols + 3
    # the pages in use lie in no order, and neither do the free ones
    order = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
    need = -(-kv // ps)
    first = torch.cumsum(need, 0) - need
    col = torch.arange(cols, device=dev)
    at = (first[:, None] + col).clamp(max=pages - 1)
    table = torch.where(col < need[:, None], order[at], torch.full_like(order[at], -1)).contiguous()
    used = need.sum()
    free = order[(torch.arange(pages, device=dev) + used) % pages].contiguous()
    rows = batch * max(1, case["prompt"])
    n_free = (pages - used).clamp(max=batch // 3) if case["scarce"] else pages - used
    s = {"case": dict(case), "op": "plan", "ps": ps, "cols": cols, "pages": pages, "max_rows": rows,
         "change": change.to(torch.int32), "base": number(0, 100000).to(torch.int32), "kv_len": kv.to(torch.int32), "table": table, "free": free,
         "n_free": n_free.to(torch.int32).reshape(1), "new_len": torch.zeros(batch, dtype=torch.int32, device=dev),
         "new_free": torch.zeros(1, dtype=torch.int32, device=dev), "cu_q": torch.zeros(batch + 1, dtype=torch.int32, device=dev),
         "status": torch.zeros(1, dtype=torch.int32, device=dev)}
    for name in ("positions", "slots", "row_seq"):
        s[name] = torch.full((rows,), -1, dtype=torch.int32, device=dev)
    return s


def _prepare_prefix(case, gen, dev):
    dt, hq, hk, d, page = _dtype(case), case["q_heads"], case["kv_heads"], case["d"], case["page"]
    q_lens, kv_lens, prefixes, sequences = (_lens(case[k]) for k in ("q_lens", "kv_lens", "prefixes", "sequences"))

    def normal(*shape, by=1.0):
        return (torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32) * by).to(dt)

    s = {"case": dict(case), "op": "prefix", "max_q": max(q_lens), "max_kv": max(kv_lens), "max_prefix": max(1, max(prefixes)),
         "cu_q": _offsets(q_lens, dev), "kv_len": _ints(kv_lens, dev), "cu_group": _offsets(sequences, dev), "prefix_len": _ints(prefixes, dev),
         "status": torch.zeros(1, dtype=torch.int32, device=dev)}
    at, most = 0, 1
    for n in sequences:
        most, at = max(most, sum(q_lens[at:at + n])), at + n
    s["max_group_q"] = most
    s["ps"], s["cols"], s["pages"] = _pool(page, kv_lens)
    s["pps"], s["pcols"], s["ppages"] = _pool(page, prefixes)
    if page:  # one pool for both
        s["pages"] = s["ppages"] = s["pages"] + s["ppages"]
        order = torch.randperm(s["pages"], generator=gen, device=dev).to(torch.int32)
        s["table"] = _table(order, kv_lens, page, s["cols"])
        s["ptable"] = _table(order, prefixes, page, s["pcols"], skip=sum(-(-n // page) for n in kv_lens))
    else:
        s["table"] = s["ptable"] = None
    s["keys"], s["values"] = normal(s["pages"], hk, s["ps"], d), normal(s["pages"], hk, s["ps"], d)
    if page:
        s["pkeys"], s["pvalues"] = s["keys"], s["values"]
    else:
        s["pkeys"], s["pvalues"] = normal(s["ppages"], hk, s["pps"], d), normal(s["ppages"], hk, s["pps"], d)
    s["q"] = normal(sum(q_lens), hq, d, by=1.5)
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(sum(q_lens), hq, dtype=torch.float32, device=dev)
    return s


def _prepare_rotate(case, gen, dev):
    hk, d, page, rot = case["kv_heads"], case["d"], case["page"], case["rot"]
    kv = _lens(case["kv_lens"])
    ps, cols, pages = _pool(page, kv)
    s = {"case": dict(case), "op": "rotate", "ps": ps, "cols": cols, "pages": pages, "max_kv": max(kv), "kv_len": _ints(kv, dev),
         "table": _table(torch.randperm(pages, generator=gen, device=dev).to(torch.int32), kv, page, cols) if page else None,
         "keys": (torch.randn(pages, hk, ps, d, generator=gen, device=dev) * 1.5).to(_dtype(case)),
         "status": torch.zeros(1, dtype=torch.int32, device=dev), "from_positions": None, "to_positions": None, "scale": 1.0}
    half = torch.arange(rot // 2, device=dev, dtype=torch.float64)
    s["from_freq"], s["to_freq"] = THETA ** (-2.0 * half / rot), None
    if case["kind"] == "evicted":  # the kept slots of a cache eight times as long, ascending; they become 0, 1, ...
        step = torch.rand(len(kv), hk, max(kv), generator=gen, device=dev) * 14 + 1
        s["from_positions"] = torch.cumsum(step, -1).to(torch.int32)
    elif case["kind"] == "scaled":
        # low frequencies are divided by four, high ones stay, those between by part; as a longer context is served
        turns = 8192 * s["from_freq"] / (2 * math.pi)
        part = ((turns - 1) / 31).clamp(0, 1)
        s["to_freq"] = s["from_freq"] * (part + (1 - part) / 4)
        s["scale"] = 1.0 + 0.1 * math.log(4.0) * 0.01  # keeps the size of keys that are turned a thousand times
    else:
        start = torch.randint(0, 100000, (2, len(kv), 1, 1), generator=gen, device=dev)
        slot = torch.arange(max(kv), device=dev)
        s["from_positions"], s["to_positions"] = ((start[i] + slot).to(torch.int32).contiguous() for i in range(2))
    return s


def work(case):
    if case["op"] == "plan":
        # of the sequences, by the shares of what they do: their numbers, the rows and the pages they take
        batch, kinds = case["batch"], [k / 100 for k in _lens(case["kinds"])]
        rows = batch * (kinds[0] + kinds[1] * (case["prompt"] + 1) / 2)
        moved = batch * kinds[3] * (case["low"] + case["high"]) / 2 + rows
        return {"bytes": int(20 * batch + 12 * rows + 8 * moved / case["page"]), "flops": int(8 * batch + 4 * rows)}
    es, d = 2 if case["dtype"] == "bf16" else 4, case["d"]
    kv_lens = _lens(case["kv_lens"])
    if case["op"] == "rotate":
        # a key's rotated part in and out, its position where one is given; four products and two sums a pair
        heads = {"evicted": case["kv_heads"], "scaled": 0, "moved": 2}[case["kind"]]
        return {"bytes": sum(kv_lens) * (2 * case["kv_heads"] * case["rot"] * es + 4 * heads), "flops": 3 * sum(kv_lens) * case["kv_heads"] * case["rot"]}
    q_lens, prefixes, sequences = (_lens(case[k]) for k in ("q_lens", "prefixes", "sequences"))
    hq, hk, total = case["q_heads"], case["kv_heads"], sum(q_lens)
    pairs, at = sum(m * n - m * (m - 1) // 2 for m, n in zip(q_lens, kv_lens)), 0
    for n, p in zip(sequences, prefixes):
        pairs, at = pairs + p * sum(q_lens[at:at + n]), at + n
    return {"bytes": 2 * total * hq * d * es + 4 * total * hq + 2 * (sum(kv_lens) + sum(prefixes)) * hk * d * es, "flops": 4 * d * hq * pairs}


# ----------------------------------------------------------------------------------
# plain forms
# ----------------------------------------------------------------------------------

def _dense(table, pool, cols, n):
    """[batch, kv_heads, n, d] of a pool's pages in the order of the sequences."""
    if table is None:
        return pool[:, :, :n]
    hk, ps, d = pool.shape[1:]
    return pool[table.long()].transpose(1, 2).reshape(table.shape[0], hk, cols * ps, d)[:, :, :n]


def _plain_plan(s):
    ps, cols, batch = s["ps"], s["cols"], s["change"].numel()
    n, change, dev = s["kv_len"].long(), s["change"].long(), s["kv_len"].device

    def pages(x):
        return (x + ps - 1) // ps

    grow = change.clamp(min=0)
    grow = torch.where(n + grow > cols * ps, torch.zeros_like(grow), grow)
    left = (n + change.clamp(max=0)).clamp(min=0)
    col = torch.arange(cols, device=dev)
    freed = s["table"][(col >= pages(left)[:, None]) & (col < pages(n)[:, None])]
    n_free = s["n_free"].long()
    available = n_free + freed.numel()
    # the free pages with those given back behind them
    stack = torch.cat((s["free"], freed))
    i = torch.arange(stack.numel(), device=dev)
    stack = stack[torch.where(i < n_free, i, i - n_free + s["free"].numel()).clamp(max=stack.numel() - 1)]
    need = pages(n + grow) - pages(n)
    served = (torch.cumsum(need, 0) <= available) & (torch.cumsum(grow, 0) <= s["max_rows"])
    grow, need = grow * served, need * served
    taken = torch.cumsum(need, 0)
    # column c of a sequence that grows is its page c - pages(n), counted behind those of the sequences before
    new = (col >= pages(n)[:, None]) & (col < pages(n + grow)[:, None])
    index = available - 1 - ((taken - need)[:, None] + col - pages(n)[:, None])
    s["table"] = torch.where(new, stack[index.clamp(0, stack.numel() - 1)], s["table"])
    end = available - taken[-1]
    i = torch.arange(s["free"].numel(), device=dev)
    s["free"] = torch.where((i >= n_free) & (i < end), stack[:i.numel()], s["free"])
    s["new_free"] = end.to(torch.int32)
    s["new_len"] = (left + grow).to(torch.int32)
    s["cu_q"] = torch.cat((torch.zeros(1, dtype=torch.int64, device=dev), torch.cumsum(grow, 0))).to(torch.int32)
    r = torch.arange(s["max_rows"], device=dev)
    live = r < s["cu_q"][-1]
    b = torch.searchsorted(s["cu_q"][1:].long(), r, right=True).clamp(max=batch - 1)
    slot = torch.where(live, n[b] + r - s["cu_q"].long()[b], torch.zeros_like(r))
    where = s["table"][b, slot // ps].long() * ps + slot % ps
    for name, value in (("positions", slot + s["base"][b]), ("slots", where), ("row_seq", b)):
        s[name] = torch.where(live, value.to(torch.int32), s[name])
    return {k: s[k] for k in ("new_len", "new_free", "cu_q", "table", "free", "positions", "slots", "row_seq")}


def _weights(x, seen, v):
    """Of logits x [.., rows, n]: the highest, the sum of exp(x - highest) over the seen and that sum with v."""
    x = x.masked_fill(~seen, -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=-3e38)
    p = (x - top).exp_()
    return top[..., 0], p.sum(-1), torch.matmul(p, v)


def _plain_prefix(s):
    c = s["case"]
    hq, hk, d, m, n = c["q_heads"], c["kv_heads"], c["d"], s["max_q"], s["max_kv"]
    g, dev, total = hq // hk, s["q"].device, s["q"].shape[0]
    cu, kv = s["cu_q"].long(), s["kv_len"].long()
    row = torch.arange(total, device=dev)
    b = torch.searchsorted(cu[1:], row, right=True)
    i = row - cu[b]
    # their own slots, the rows of each sequence padded to the longest
    at = (cu[:-1, None] + torch.arange(m, device=dev)).clamp(max=total - 1)
    q = s["q"][at].float().unflatten(2, (hk, g)).permute(0, 2, 3, 1, 4).flatten(2, 3)
    k, v = _dense(s["table"], s["keys"], s["cols"], n).float(), _dense(s["table"], s["values"], s["cols"], n).float()
    slot = torch.arange(n, device=dev)
    v = torch.where((slot < kv[:, None])[:, None, :, None], v, torch.zeros((), device=dev))
    j = torch.arange(m, device=dev)
    seen = slot <= (kv - cu[1:] + cu[:-1])[:, None, None] + j[:, None]
    seen = (seen & (slot < kv[:, None])[:, None])[:, None, None].expand(-1, 1, g, -1, -1).flatten(2, 3)
    top, total_p, o = _weights(torch.matmul(q, k.transpose(2, 3)) * (1.0 / math.sqrt(d)), seen, v)

    def packed(x):  # [batch, kv_heads, group * max_q, ..] to [rows, q_heads, ..]
        x = x.unflatten(2, (g, m)).transpose(2, 3)
        return x[b, :, i].flatten(1, 2)

    top, total_p, o = packed(top), packed(total_p), packed(o)
    # the prefixes, one after the other, each with all rows of its group
    sequences, prefixes = _lens(c["sequences"]), _lens(c["prefixes"])
    q_lens, first, r0 = _lens(c["q_lens"]), 0, 0
    for w, (count, p) in enumerate(zip(sequences, prefixes)):
        r1 = r0 + sum(q_lens[first:first + count])
        if p > 0:
            table = None if s["ptable"] is None else s["ptable"][w:w + 1]
            pool = [x if table is not None else x[w:w + 1] for x in (s["pkeys"], s["pvalues"])]
            k, v = (_dense(table, x, s["pcols"], p)[0].float() for x in pool)
            x = s["q"][r0:r1].float().unflatten(1, (hk, g)).permute(1, 2, 0, 3).flatten(1, 2)
            x = torch.matmul(x, k.transpose(1, 2)).mul_(1.0 / math.sqrt(d))
            t = x.amax(-1, keepdim=True)
            x = x.sub_(t).exp_()
            y = torch.matmul(x, v)
            t, l, y = (z.unflatten(1, (g, r1 - r0)).permute(2, 0, 1, *range(3, z.dim() + 1)).flatten(1, 2) for z in (t[..., 0], x.sum(-1), y))
            high = torch.maximum(t, top[r0:r1])
            f0, f1 = (top[r0:r1] - high).exp(), (t - high).exp()
            top[r0:r1], total_p[r0:r1] = high, total_p[r0:r1] * f0 + l * f1
            o[r0:r1] = o[r0:r1] * f0[..., None] + y * f1[..., None]
        first, r0 = first + count, r1
    o = o / total_p.clamp(min=1e-38)[..., None]
    return {"out": o.to(s["q"].dtype), "lse": total_p.log() + top}


def _plain_rotate(s):
    c, keys = s["case"], s["keys"]
    rot, ps, n, batch = c["rot"], s["ps"], s["max_kv"], s["kv_len"].numel()
    slot = torch.arange(n, device=keys.device)
    start = slot.expand(batch, 1, n) if s["from_positions"] is None else s["from_positions"]
    to = slot.expand(batch, 1, n) if s["to_positions"] is None else s["to_positions"]
    to_freq = s["from_freq"] if s["to_freq"] is None else s["to_freq"]
    angle = to.double()[..., None] * to_freq - start.double()[..., None] * s["from_freq"]
    cos, sin = angle.cos().float() * s["scale"], angle.sin().float() * s["scale"]
    x = _dense(s["table"], keys, s["cols"], n).float()
    if c["interleaved"]:
        x1, x2 = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((x1 * cos - x2 * sin, x2 * cos + x1 * sin), -1).flatten(-2)
    else:
        x1, x2 = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat((x1 * cos - x2 * sin, x2 * cos + x1 * sin), -1)
    y = torch.cat((y, x[..., rot:]), -1).to(keys.dtype)
    b, at = torch.nonzero(slot < s["kv_len"][:, None], as_tuple=True)
    page = b if s["table"] is None else s["table"].long()[b, at // ps]
    keys[page, :, at % ps] = y[b, :, at]
    return {"keys": keys}


# ----------------------------------------------------------------------------------
# the library's calls
# ----------------------------------------------------------------------------------

def _own_run(s):
    import lsh_sampled_sparse_centered_gb300 as mp
    c, op = s["case"], s["op"]
    cfg = s.get("cfg")
    if cfg is None:  # the configurations and the workspace that a program makes once
        kv_heads = c.get("kv_heads", 1)
        shape = dict(kv_heads=kv_heads, q_heads=c.get("q_heads", kv_heads), head_dim=c.get("d", 128), dtype=c.get("dtype", "bf16"))
        cfg = s["cfg"] = mp.make_cache_config(batch=s["kv_len"].numel(), page_size=s["ps"], n_pages=s["pages"], max_pages=s["cols"], **shape)
        if op == "prefix":
            s["pcfg"] = mp.make_cache_config(batch=s["prefix_len"].numel(), page_size=s["pps"], n_pages=s["ppages"], max_pages=s["pcols"], **shape)
            size = mp.mp_prefix_workspace_bytes(cfg, s["pcfg"], s["q"].shape[0], s["max_q"], s["max_kv"], s["max_group_q"], s["max_prefix"])
            s["workspace"] = torch.empty(size, dtype=torch.uint8, device=s["q"].device)
        if op == "rotate":
            s["rotary"] = mp.make_rotary(rot_dim=c["rot"], interleaved=c["interleaved"])
    if op == "plan":
        mp.mp_cache_plan(cfg, s["change"], s["base"], s["kv_len"], s["n_free"], s["max_rows"], s["table"], s["free"], s["new_len"],
                         s["new_free"], s["cu_q"], s["positions"], s["slots"], s["row_seq"], s["status"])
        return {k: s[k] for k in ("new_len", "new_free", "cu_q", "table", "free", "positions", "slots", "row_seq")}
    if op == "prefix":
        mp.mp_prefix_attention(cfg, s["pcfg"], s["q"], s["cu_q"], s["kv_len"], s["max_q"], s["max_kv"], s["keys"], s["values"], s["table"],
                               s["cu_group"], s["prefix_len"], s["max_group_q"], s["max_prefix"], s["pkeys"], s["pvalues"], s["ptable"],
                               s["out"], s["lse"], s["workspace"], s["status"])
        return {"out": s["out"], "lse": s["lse"]}
    mp.mp_cache_rotate(cfg, s["rotary"], s["keys"], s["table"], s["kv_len"], s["max_kv"], s["from_freq"], s["to_freq"], s["from_positions"],
                       s["to_positions"], s["scale"], s["status"])
    return {"keys": s["keys"]}


def run(state):
    if own:
        return _own_run(state)
    return {"plan": _plain_plan, "prefix": _plain_prefix, "rotate": _plain_rotate}[state["op"]](state)


# ----------------------------------------------------------------------------------
# the definitions in 64 bits
# ----------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "plan":  # whole numbers: a loop over the sequences
        return None if case["batch"] > 2000 else _exact_plan(s)
    hk, d, ps = case["kv_heads"], case["d"], s["ps"]
    kv_lens = _lens(case["kv_lens"])

    def pages(table, b, n, per):
        return torch.tensor([b], device="cuda") if table is None else table[b, :-(-n // per)].long()

    def rows(pool, numbers, h, n):
        return pool[numbers, h].flatten(0, 1)[:n].double()

    if case["op"] == "rotate":
        keys, rot = s["keys"].double(), case["rot"]
        first = torch.arange(0, rot, 2, device="cuda") if case["interleaved"] else torch.arange(rot // 2, device="cuda")
        second = first + (1 if case["interleaved"] else rot // 2)
        for b, n in enumerate(kv_lens):
            numbers = pages(s["table"], b, n, ps)
            for h in range(hk):
                def positions(p):
                    return torch.arange(n, device="cuda").double() if p is None else p[b, h if p.shape[1] > 1 else 0, :n].double()
                turn = torch.outer(positions(s["to_positions"]), s["from_freq"] if s["to_freq"] is None else s["to_freq"])
                turn = torch.polar(torch.full_like(turn, s["scale"]), turn - torch.outer(positions(s["from_positions"]), s["from_freq"]))
                x = rows(s["keys"], numbers, h, n)
                z = torch.complex(x[:, first], x[:, second]) * turn
                x[:, first], x[:, second] = z.real, z.imag
                whole = keys[numbers, h].flatten(0, 1)
                whole[:n] = x
                keys[numbers, h] = whole.unflatten(0, (numbers.numel(), ps))
        return {"keys": keys}

    hq, q_lens, prefixes, sequences = case["q_heads"], *(_lens(case[k]) for k in ("q_lens", "prefixes", "sequences"))
    total = sum(q_lens)
    out = torch.zeros(total, hq, d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(total, hq, dtype=torch.float64, device="cuda")
    group = [g for g, n in enumerate(sequences) for _ in range(n)]
    owners = [b for b, m in enumerate(q_lens) for _ in range(m)]
    for h in range(hk):
        heads = slice(h * (hq // hk), (h + 1) * (hq // hk))
        for g in [None] + list(range(len(sequences))):
            mine = [r for r in range(total) if (group[owners[r]] if owners[r] < len(group) else None) == g]
            if not mine:
                continue
            at = torch.tensor(mine, device="cuda")
            q = s["q"][at, heads].double() / d ** 0.5  # [rows, heads, d]
            zs, os = [], []
            if g is not None and prefixes[g]:
                numbers = pages(s["ptable"], g, prefixes[g], s["pps"])
                k, v = rows(s["pkeys"], numbers, h, prefixes[g]), rows(s["pvalues"], numbers, h, prefixes[g])
                x = q @ k.T
                z = torch.logsumexp(x, -1)
                zs.append(z)
                os.append(torch.exp(x - z[..., None]) @ v)
            z, o = torch.zeros_like(q[..., 0]), torch.zeros_like(q)
            for b in sorted(set(owners[r] for r in mine)):
                local = torch.tensor([i for i, r in enumerate(mine) if owners[r] == b], device="cuda")
                m, n = q_lens[b], kv_lens[b]
                numbers = pages(s["table"], b, n, ps)
                x = q[local] @ rows(s["keys"], numbers, h, n).T
                limit = torch.arange(n - m, n, device="cuda")
                x = x + torch.where(torch.arange(n, device="cuda") > limit[:, None], -math.inf, 0.0).double()[:, None]
                z[local] = torch.logsumexp(x, -1)
                o[local] = torch.exp(x - z[local][..., None]) @ rows(s["values"], numbers, h, n)
            zs.append(z)
            os.append(o)
            both = torch.logsumexp(torch.stack(zs), 0)
            lse[at, heads] = both
            out[at, heads] = sum(torch.exp(z - both)[..., None] * o for z, o in zip(zs, os))
    return {"out": out, "lse": lse}


def _exact_plan(s):
    ps, cols = s["ps"], s["cols"]
    change, kv, base, table, free = (s[k].tolist() for k in ("change", "kv_len", "base", "table", "free"))
    n_free = int(s["n_free"])
    stack = free[:n_free]
    for b, (x, n) in enumerate(zip(change, kv)):
        if x < 0:
            stack += table[b][-(-max(0, n + x) // ps):-(-n // ps)]
    back = len(stack)
    lengths, cu, positions, slots, owner, open_ = [], [0], s["positions"].tolist(), s["slots"].tolist(), s["row_seq"].tolist(), True
    for b, (x, n) in enumerate(zip(change, kv)):
        if x <= 0 or n + x > cols * ps:
            lengths.append(max(0, n + min(x, 0)))
            cu.append(cu[-1])
            continue
        need = -(-(n + x) // ps) - -(-n // ps)
        open_ = open_ and need <= len(stack) and cu[-1] + x <= s["max_rows"]
        m = x if open_ else 0
        for j in range(need if open_ else 0):
            table[b][-(-n // ps) + j] = stack.pop()
        for i in range(m):
            r, at = cu[-1] + i, n + i
            positions[r], slots[r], owner[r] = base[b] + at, table[b][at // ps] * ps + at % ps, b
        lengths.append(n + m)
        cu.append(cu[-1] + m)
    for i in range(n_free, min(len(stack), back)):
        free[i] = stack[i]
    made = {"new_len": lengths, "new_free": [len(stack)], "cu_q": cu, "table": table, "free": free, "positions": positions, "slots": slots,
            "row_seq": owner}
    return {k: torch.tensor(v, dtype=torch.int32, device="cuda") for k, v in made.items()}
