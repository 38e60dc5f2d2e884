"""The cache operators on the GPU against plain float64 forms, at the sizes, masks, pages
and lengths where they can go wrong.

Tolerances, with h = half a step of a type relative to the value (fp32 2^-24, bf16 2^-8):
- append: one final rounding, h |y|, plus fp32 arithmetic on the pair (a, b): the mean of
  d squares through chains of at most 8 + 5 additions, its root and quotient, two products,
  a sine and cosine good to 2^-22 and three roundings of the rotation: below 2^-18 of the
  pair's norm.
- attention: a logit is off by at most (d + 8) 2^-24 slack with slack = sum |q k| / sqrt(d)
  (a chain of d products, the scale and the reference's subtraction), a weight relatively by
  that and 2^-21 of the exponential, numerator and sum alike, and sums of n terms by n 2^-24;
  in bf16 a weight is rounded by 2^-8 more. All of it weighs sum p |v|; the result is rounded
  once. lse is off by the logits' part, n 2^-24 and its own rounding.
- weights: as the exponentials above, on a sum of at most rows terms.
- eviction copies and compares: equal bits.
"""
import math

import pytest
import torch

import cache_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def mp():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import lsh_sampled_sparse_centered_gb300 as m
    return m


DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


class Cache:
    """A pool with pages in no order; everything behind the sequences' ends is NaN."""

    def __init__(self, mp, dtype, hq, hk, d, page, kv, seed=0, cap=None, fill="normal"):
        g = torch.Generator().manual_seed(seed)
        self.gen, self.kv, self.dtype, self.hq, self.hk, self.d = g, list(kv), DT[dtype], hq, hk, d
        batch = len(kv)
        cap = cap or max(1, max(kv))
        if page == 0:
            self.ps, self.cols, self.pages, self.table = cap, 1, batch, None
        else:
            self.ps, self.cols = page, -(-cap // page)
            self.pages = batch * self.cols + 2
            order = torch.randperm(self.pages, generator=g)[:batch * self.cols].view(batch, self.cols).to(torch.int32)
            for b, n in enumerate(kv):
                order[b, -(-n // page):] = -7  # never looked at
            self.table = order.to(DEV)
        shape = (self.pages, hk, self.ps, d)
        self.keys = torch.full(shape, math.nan, dtype=self.dtype, device=DEV)
        self.values = torch.full(shape, math.nan, dtype=self.dtype, device=DEV)
        if fill == "normal":
            for b, n in enumerate(kv):
                for i, p in enumerate(R.pages_of(self.table, b, n, self.ps)):
                    e = min(self.ps, n - i * self.ps)
                    for pool in (self.keys, self.values):
                        pool[p, :, :e] = torch.randn(hk, e, d, generator=g).to(DEV, self.dtype)
        self.cfg = mp.make_cache_config(batch=batch, kv_heads=hk, q_heads=hq, head_dim=d, page_size=self.ps, n_pages=self.pages,
                                        max_pages=self.cols, dtype=dtype)
        self.kv_len = torch.tensor(kv, dtype=torch.int32, device=DEV)
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def randn(self, *shape, by=1.0):
        return (torch.randn(*shape, generator=self.gen) * by).to(DEV, self.dtype)


def offsets(q_lens):
    cu = [0]
    for m in q_lens:
        cu.append(cu[-1] + m)
    return cu, torch.tensor(cu, dtype=torch.int32, device=DEV)


def attend(mp, c, q, cu_t, max_q, max_kv=None, lse=True, stream=None, workspace=None):
    max_kv = max_kv or max(1, max(c.kv))
    out = torch.full_like(q, 77.0)
    z = torch.full(q.shape[:2], 77.0, device=DEV) if lse else None
    size = mp.mp_chunk_workspace_bytes(c.cfg, q.shape[0], max_q, max_kv)
    ws = torch.full((max(1, size),), 0xFF, dtype=torch.uint8, device=DEV) if workspace is None else workspace
    mp.mp_chunk_attention(c.cfg, q, cu_t, c.kv_len, max_q, max_kv, c.keys, c.values, c.table, out, z, ws, c.status, stream=stream)
    return out, z


def check_attention(c, dtype, q, cu, out, lse):
    want, z, spread, slack = R.attention(q, cu, c.kv, c.keys, c.values, c.table, c.hk)
    n = cu[-1]
    eps_x = (c.d + 8) * 2.0 ** -24 * slack[:n]
    rel = 2 * eps_x + max(c.kv) * 2.0 ** -24 + 2.0 ** -20 + (2.0 ** -8 if dtype == "bf16" else 0.0)
    tol = HALF[dtype] * want[:n].abs() + (1 + HALF[dtype]) * rel[..., None] * spread[:n]
    err = (out[:n].double() - want[:n]).abs()
    assert torch.isfinite(out[:n]).all()
    assert (err <= tol).all(), (err - tol).max().item()
    if lse is not None:
        empty = torch.isinf(z[:n])
        assert torch.equal(torch.isinf(lse[:n]) & (lse[:n] < 0), empty)
        ztol = eps_x + (max(c.kv) + 8) * 2.0 ** -24 + 2.0 ** -21 * (1 + z[:n].abs())
        assert ((lse[:n].double() - z[:n]).abs()[~empty] <= ztol[~empty]).all()
    assert (out[n:] == 77.0).all() and (lse is None or (lse[n:] == 77.0).all())  # rows behind the last sequence


ATTEND = [
    # dtype, q heads, kv heads, d, page, chunk lengths, cache lengths
    ("bf16", 4, 2, 64, 0, [1], [1]),
    ("bf16", 8, 2, 128, 16, [1, 1, 1], [1, 17, 300]),
    ("bf16", 8, 1, 128, 64, [1, 1], [64, 4097]),                    # one token over a long cache, and exactly a page
    ("bf16", 7, 7, 64, 0, [1, 1], [129, 1000]),                     # no grouping
    ("bf16", 12, 1, 128, 48, [1, 2], [777, 50]),                    # a group of 12, pages that end inside a tile
    ("bf16", 40, 1, 64, 32, [1], [500]),                            # a group of more than 32
    ("bf16", 6, 2, 64, 16, [3, 2, 5], [3, 1000, 77]),               # groups of 3, a few tokens
    ("bf16", 4, 2, 128, 128, [128], [128]),
    ("bf16", 4, 2, 128, 128, [129, 1, 127], [129, 640, 1000]),
    ("bf16", 28, 4, 128, 64, [37, 100], [37, 411]),                 # groups of 7
    ("bf16", 16, 2, 64, 256, [200], [1111]),
    ("bf16", 8, 8, 64, 0, [300, 10], [700, 333]),
    ("bf16", 8, 2, 128, 16, [0, 5, 0, 40, 1], [9, 5, 0, 300, 0]),    # empty chunks, empty caches
    ("bf16", 8, 2, 64, 16, [9, 70], [4, 33]),                       # chunks longer than their caches: rows that see nothing
    ("bf16", 32, 8, 128, 0, [513], [2500]),
    ("bf16", 64, 1, 128, 96, [5], [900]),
    ("bf16", 136, 1, 64, 32, [3, 1], [100, 40]),                    # a group of more than 128
    ("bf16", 300, 1, 64, 16, [2, 1], [50, 7]),                      # and of more than 256
    ("bf16", 4, 4, 64, 64, [20, 8, 32], [500, 1300, 32]),
    ("f32", 4, 2, 64, 0, [1], [1]),
    ("f32", 8, 2, 128, 16, [1, 1, 3], [17, 2000, 64]),
    ("f32", 6, 2, 64, 48, [65, 1, 0], [200, 1500, 9]),
    ("f32", 8, 8, 128, 0, [100, 3], [333, 400]),
    ("f32", 8, 1, 64, 32, [9, 70], [4, 33]),
]


@pytest.mark.parametrize("dtype,hq,hk,d,page,q_lens,kv", ATTEND)
def test_attention(mp, dtype, hq, hk, d, page, q_lens, kv):
    c = Cache(mp, dtype, hq, hk, d, page, kv)
    cu, cu_t = offsets(q_lens)
    q = c.randn(cu[-1] + 3, hq, d, by=1.5)  # three rows that belong to no sequence
    out, lse = attend(mp, c, q, cu_t, max(q_lens))
    check_attention(c, dtype, q, cu, out, lse)
    assert c.status.item() == 0
    # the same bits again, without lse, and with wider limits (another split of the same slots is
    # another order of sums, so that one is held to the tolerance)
    again, _ = attend(mp, c, q, cu_t, max(q_lens), lse=False)
    assert torch.equal(again[:cu[-1]], out[:cu[-1]])
    cap = c.ps * c.cols
    wide, z = attend(mp, c, q, cu_t, max(q_lens) + 50, max_kv=cap)
    check_attention(c, dtype, q, cu, wide, z)


def test_attention_of_large_logits(mp):
    """Logits of both signs and several hundred: the reference of the softmax has to move."""
    for dtype in ("bf16", "f32"):
        c = Cache(mp, dtype, 8, 2, 128, 64, [700, 300])
        c.keys.mul_(6.0)
        cu, cu_t = offsets([40, 1])
        q = c.randn(41, 8, 128, by=8.0)
        out, lse = attend(mp, c, q, cu_t, 40)
        check_attention(c, dtype, q, cu, out, lse)


def test_attention_of_equal_and_constant_keys(mp):
    c = Cache(mp, "bf16", 4, 2, 64, 32, [333])
    c.keys[~c.keys.isnan()] = 0.0
    cu, cu_t = offsets([20])
    q = c.randn(20, 4, 64)
    out, lse = attend(mp, c, q, cu_t, 20)
    check_attention(c, "bf16", q, cu, out, lse)
    want = torch.log(torch.arange(314, 334, device=DEV).double())[:, None]
    assert ((lse.double() - want).abs() <= 2.0 ** -20 * want).all()


def test_attention_over_offsets_past_32_bits(mp):
    """A pool of more than 2^32 elements: the pages in use lie at its end."""
    ps, hk, d = 4096, 4, 128
    pages = 2 ** 31 // (ps * hk * d) * 2 + 3
    cfg = mp.make_cache_config(batch=1, kv_heads=hk, q_heads=8, head_dim=d, page_size=ps, n_pages=pages, max_pages=2, dtype="bf16")
    keys = torch.empty(pages, hk, ps, d, dtype=torch.bfloat16, device=DEV)
    values = torch.empty_like(keys)
    assert keys.numel() > 2 ** 32
    g = torch.Generator(device=DEV).manual_seed(3)
    for pool in (keys, values):
        pool[-2:] = torch.randn(2, hk, ps, d, generator=g, device=DEV).to(torch.bfloat16)
    table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32, device=DEV)
    for m, n in ((1, 5000), (150, 5000)):
        kv_len = torch.tensor([n], dtype=torch.int32, device=DEV)
        cu, cu_t = offsets([m])
        q = torch.randn(m, 8, d, generator=g, device=DEV).to(torch.bfloat16)
        out, lse = torch.empty_like(q), torch.empty(m, 8, device=DEV)
        ws = torch.empty(max(1, mp.mp_chunk_workspace_bytes(cfg, m, m, n)), dtype=torch.uint8, device=DEV)
        mp.mp_chunk_attention(cfg, q, cu_t, kv_len, m, n, keys, values, table, out, lse, ws)

        class C:
            pass
        c = C()
        c.kv, c.keys, c.values, c.table, c.hk, c.d = [n], keys, values, table, hk, d
        check_attention(c, "bf16", q, cu, out, lse)


def test_append_weights_and_evict_over_offsets_past_32_bits(mp):
    ps, hk, d, n = 4096, 4, 128, 5000
    pages = 2 ** 31 // (ps * hk * d) * 2 + 3
    cfg = mp.make_cache_config(batch=1, kv_heads=hk, q_heads=hk, head_dim=d, page_size=ps, n_pages=pages, max_pages=2, dtype="bf16")
    keys = torch.zeros(pages, hk, ps, d, dtype=torch.bfloat16, device=DEV)
    values = torch.zeros_like(keys)
    assert keys.numel() > 2 ** 32
    table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(5)
    q, k, v = (torch.randn(n, hk, d, generator=g, device=DEV).to(torch.bfloat16) for _ in range(3))
    cu, cu_t = offsets([n])
    kv_len = torch.tensor([n], dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    q_out = torch.empty_like(q)
    mp.mp_cache_append(cfg, mp.make_rotary(rot_dim=0), q, k, v, None, None, None, None, cu_t, kv_len, keys, values, table, q_out, status)
    for pool, x in ((keys, k), (values, v)):
        assert torch.equal(R.gather(pool, table, 0, 3, n), x[:, 3].double())
    assert not keys[:-2].any() and not values[:-2].any() and torch.equal(q_out, q)
    cu, cu_t = offsets([2])
    lse = R.attention(q[:2], cu, [n], keys, values, table, hk)[1].float()
    scores = torch.zeros(1, hk, 2 * ps, device=DEV)
    mp.mp_cache_weights(cfg, q[:2], lse, cu_t, kv_len, 2, n, keys, table, scores, status)
    want = R.weights(q[:2], lse, cu, [n], keys, table, torch.zeros_like(scores))[0]
    assert ((scores.double() - want).abs() <= 2.0 ** -14 * want + 1e-30).all()
    dst = mp.make_cache_config(batch=1, kv_heads=hk, q_heads=hk, head_dim=d, page_size=100, n_pages=1, dtype="bf16")
    dk, dv = (torch.zeros(1, hk, 100, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    dlen, kept = torch.zeros(1, dtype=torch.int32, device=DEV), torch.zeros(1, hk, 100, dtype=torch.int32, device=DEV)
    ws = torch.empty(mp.mp_evict_workspace_bytes(cfg, n, 100), dtype=torch.uint8, device=DEV)
    mp.mp_cache_evict(cfg, dst, keys, values, table, kv_len, n, scores, 4, 16, 100, dk, dv, None, None, dlen, kept, ws, status)
    for h in range(hk):
        keep = R.keep(scores[0, h], n, 4, 16, 100)
        assert kept[0, h].tolist() == keep
        at = torch.tensor(keep, device=DEV)
        assert torch.equal(dk[0, h], k[at, h]) and torch.equal(dv[0, h], v[at, h])
    assert status.item() == 0


def test_attention_of_more_sequences_than_one_launch_takes(mp):
    """The tensor-core path plans 1024 sequences at a time."""
    batch = 1100
    kv = [(7 * b) % 40 for b in range(batch)]
    q_lens = [min(n, 1 + b % 5) for b, n in enumerate(kv)]
    c = Cache(mp, "bf16", 5, 1, 64, 16, kv)
    cu, cu_t = offsets(q_lens)
    q = c.randn(cu[-1] + 1, 5, 64)
    out, lse = attend(mp, c, q, cu_t, 5)
    check_attention(c, "bf16", q, cu, out, lse)
    assert c.status.item() == 0


def test_two_calls_at_once_with_a_workspace_each(mp):
    """Two streams, both kinds of the attention, a shared page that both sequences read."""
    for m in (1, 50):
        c = Cache(mp, "bf16", 8, 2, 128, 64, [3000, 2500])
        c.table[1, 0] = c.table[0, 0]
        cu, cu_t = offsets([m, m])
        qs = [c.randn(2 * m, 8, 128) for _ in range(2)]
        streams = [torch.cuda.Stream() for _ in range(2)]
        size = max(1, mp.mp_chunk_workspace_bytes(c.cfg, 2 * m, m, 3000))
        ws = [torch.empty(size, dtype=torch.uint8, device=DEV) for _ in range(2)]
        outs = [(torch.empty_like(q), torch.empty(2 * m, 8, device=DEV)) for q in qs]
        torch.cuda.synchronize()
        for _ in range(20):
            for q, (out, lse), w, st in zip(qs, outs, ws, streams):
                mp.mp_chunk_attention(c.cfg, q, cu_t, c.kv_len, m, 3000, c.keys, c.values, c.table, out, lse, w, c.status, stream=st)
        torch.cuda.synchronize()
        for q, (out, lse) in zip(qs, outs):
            check_attention(c, "bf16", q, cu, out, lse)


def test_bad_lengths_and_pages_set_their_bits_and_leave_the_rest(mp):
    c = Cache(mp, "bf16", 8, 2, 128, 32, [200, 100, 150])
    cu, cu_t = offsets([5, 40, 1])
    q = c.randn(46, 8, 128)
    want, _ = attend(mp, c, q, cu_t, 40)
    c.table[1, 1] = c.pages + 5
    c.table[1, 2] = -1
    # what the bad numbers read instead must be finite for the others to stay comparable
    out, lse = attend(mp, c, q, cu_t, 40)
    assert c.status.item() == mp.MP_STATUS_BAD_PAGE
    assert torch.equal(out[:5], want[:5]) and torch.equal(out[45:], want[45:])
    c.status.zero_()
    sc = torch.zeros(3, 2, c.ps * c.cols, device=DEV)
    mp.mp_cache_weights(c.cfg, q, lse, cu_t, c.kv_len, 40, 200, c.keys, c.table, sc, c.status)
    assert c.status.item() == mp.MP_STATUS_BAD_PAGE and torch.isfinite(sc[0]).all()
    c.status.zero_()
    c.table[1, 1:3] = 0
    c.kv_len[0] = 10 ** 9
    cu_t[3] = 10 ** 6
    attend(mp, c, q, cu_t, 40)
    assert c.status.item() & mp.MP_STATUS_BAD_LENGTH
    # a limit of the host's below a device length cuts it
    c.kv_len[0] = 200
    cu_t[3] = 46
    c.status.zero_()
    attend(mp, c, q, cu_t, 40, max_kv=150)
    assert c.status.item() == mp.MP_STATUS_BAD_LENGTH


def test_attention_captured_follows_the_lengths(mp):
    """One captured call over a growing cache, on a stream of its own, with two graphs that
    have a workspace each."""
    for q_len in (1, 33):
        c = Cache(mp, "bf16", 8, 2, 128, 64, [1500, 900])
        cu, cu_t = offsets([q_len, q_len])
        st = torch.cuda.Stream()
        graphs = []
        for i in range(2):
            q = c.randn(2 * q_len, 8, 128)
            out, lse = torch.empty_like(q), torch.empty(2 * q_len, 8, device=DEV)
            ws = torch.empty(max(1, mp.mp_chunk_workspace_bytes(c.cfg, 2 * q_len, q_len, 1500)), dtype=torch.uint8, device=DEV)
            call = lambda: mp.mp_chunk_attention(c.cfg, q, cu_t, c.kv_len, q_len, 1500, c.keys, c.values, c.table, out, lse, ws, c.status)
            torch.cuda.synchronize()
            with torch.cuda.stream(st):
                call()
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g, stream=st):
                    call()
            graphs.append((g, q, out, lse, ws))
        for lens in ([1500, 900], [64, 65], [q_len, 870]):
            c.kv = lens
            c.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
            torch.cuda.synchronize()
            for g, *_ in graphs:
                g.replay()
            torch.cuda.synchronize()
            for _, q, out, lse, _ in graphs:
                check_attention(c, "bf16", q, cu, out, lse)
        assert c.status.item() == 0


# ---- weights ----

@pytest.mark.parametrize("dtype,hq,hk,d,page,q_lens,kv", ATTEND)
def test_weights(mp, dtype, hq, hk, d, page, q_lens, kv):
    c = Cache(mp, dtype, hq, hk, d, page, kv)
    cu, cu_t = offsets(q_lens)
    q = c.randn(cu[-1] + 3, hq, d, by=1.5)
    lse = R.attention(q, cu, c.kv, c.keys, c.values, c.table, hk)[1].float()
    lse[cu[-1]:] = math.nan
    sc0 = torch.rand(len(kv), hk, c.ps * c.cols, generator=c.gen).to(DEV) * 0.01
    for b, n in enumerate(kv):
        sc0[b, :, n:] = math.nan
    want, slack = R.weights(q, lse, cu, c.kv, c.keys, c.table, sc0)
    got = []
    for _ in range(2):
        sc = sc0.clone()
        mp.mp_cache_weights(c.cfg, q, lse, cu_t, c.kv_len, max(q_lens), max(1, max(kv)), c.keys, c.table, sc, c.status)
        got.append(sc)
    assert c.status.item() == 0
    assert torch.equal(got[0].view(torch.int32), got[1].view(torch.int32))
    for b, n in enumerate(kv):
        assert torch.isnan(got[0][b, :, n:]).all()
        if n == 0:
            continue
        w = want[b, :, :n]
        top = (lse[cu[b]:cu[b + 1]][~torch.isinf(lse[cu[b]:cu[b + 1]])]).abs().max() if cu[b + 1] > cu[b] and (n > 0) else torch.zeros((), device=DEV)
        rel = (d + 8) * 2.0 ** -24 * slack[b, :, :n] + 2.0 ** -21 * (1 + top.double()) + (hq // hk * max(q_lens) + 2) * 2.0 ** -24
        assert ((got[0][b, :, :n].double() - w).abs() <= rel * w).all()


def test_weights_sum_to_the_number_of_queries(mp):
    """What attention hands out is one per query head and token: also through bf16 tensors."""
    c = Cache(mp, "bf16", 8, 2, 128, 64, [1000, 77])
    cu, cu_t = offsets([60, 1])
    q = c.randn(61, 8, 128)
    _, lse = attend(mp, c, q, cu_t, 60)
    sc = torch.zeros(2, 2, c.ps * c.cols, device=DEV)
    mp.mp_cache_weights(c.cfg, q, lse, cu_t, c.kv_len, 60, 1000, c.keys, c.table, sc, c.status)
    total = sc.double().sum(-1)
    want = torch.tensor([[60 * 4.0], [4.0]], device=DEV).double()
    assert ((total - want).abs() <= 2.0 ** -14 * want).all()


# Enough tiles of rows and blocks of keys that a CTA has several of them, shares some with
# others, and passes from one sequence to the next.
WIDE = [
    ("bf16", 40, 40, 128, 64, [1000], [1100]),
    ("bf16", 32, 8, 128, 0, [1024], [2048]),
    ("bf16", 64, 8, 64, 16, [300, 200, 90], [2000, 900, 3000]),
    ("bf16", 16, 16, 128, 48, [33, 40, 65], [9000, 4000, 2500]),
    ("bf16", 17, 1, 64, 16, [1 + b % 2 for b in range(520)], [1 + (7 * b) % 40 for b in range(520)]),
]


@pytest.mark.parametrize("dtype,hq,hk,d,page,q_lens,kv", WIDE)
def test_attention_of_many_tiles(mp, dtype, hq, hk, d, page, q_lens, kv):
    test_attention(mp, dtype, hq, hk, d, page, q_lens, kv)


@pytest.mark.parametrize("dtype,hq,hk,d,page,q_lens,kv", WIDE)
def test_weights_of_many_blocks(mp, dtype, hq, hk, d, page, q_lens, kv):
    test_weights(mp, dtype, hq, hk, d, page, q_lens, kv)


def test_weights_captured_and_on_two_streams(mp):
    """One captured call per stream, replayed at once, that follows the lengths."""
    c = Cache(mp, "bf16", 8, 2, 128, 64, [3000, 2500])
    cu, cu_t = offsets([50, 20])
    parts = []
    for _ in range(2):
        st = torch.cuda.Stream()
        q = c.randn(70, 8, 128)
        lse = R.attention(q, cu, [2000, 2500], c.keys, c.values, c.table, 2)[1].float()
        sc = torch.zeros(2, 2, c.ps * c.cols, device=DEV)
        call = lambda: mp.mp_cache_weights(c.cfg, q, lse, cu_t, c.kv_len, 50, 3000, c.keys, c.table, sc, c.status)
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            call()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=st):
                call()
        parts.append((g, st, q, lse, sc))
    torch.cuda.synchronize()
    c.kv_len.copy_(torch.tensor([2000, 2500], dtype=torch.int32))
    for _, _, _, _, sc in parts:
        sc.zero_()
    torch.cuda.synchronize()
    for g, st, *_ in parts:
        with torch.cuda.stream(st):
            g.replay()
    torch.cuda.synchronize()
    assert c.status.item() == 0
    for _, _, q, lse, sc in parts:
        want, slack = R.weights(q, lse, cu, [2000, 2500], c.keys, c.table, torch.zeros_like(sc))
        for b, n in enumerate([2000, 2500]):
            # as in test_weights
            rel = 136 * 2.0 ** -24 * slack[b, :, :n] + 2.0 ** -21 * (1 + lse.abs().max().double()) + 202 * 2.0 ** -24
            assert ((sc[b, :, :n].double() - want[b, :, :n]).abs() <= rel * want[b, :, :n]).all()
            assert not sc[b, :, n:].any()


# ---- append ----

APPEND = [
    # dtype, q heads, kv heads, d, page, chunk lengths, cache lengths, rot, interleaved, norms
    ("bf16", 4, 2, 128, 16, [1, 3, 0, 20], [1, 50, 9, 20], 128, False, True),
    ("bf16", 32, 8, 128, 64, [1] * 5, [100, 64, 65, 1, 4000], 128, False, True),
    ("bf16", 8, 8, 64, 0, [70, 1], [70, 200], 64, True, True),
    ("bf16", 3, 1, 64, 48, [33, 17], [100, 17], 32, False, True),
    ("bf16", 5, 5, 128, 32, [9], [9], 0, False, False),
    ("bf16", 4, 4, 64, 16, [10], [20], 10, True, True),              # pairs that end inside a vector
    ("bf16", 4, 4, 128, 16, [10, 4], [20, 3], 16, False, False),     # a token in no slot
    ("f32", 4, 2, 128, 16, [1, 3, 0, 20], [1, 50, 9, 20], 128, False, True),
    ("f32", 6, 2, 64, 0, [70, 1], [70, 200], 8, False, True),
    ("f32", 7, 1, 64, 32, [33], [40], 62, True, False),
    ("bf16", 3, 1, 64, 16, [1225, 0, 6, 3], [1300, 5, 6, 200], 64, False, True),  # enough rows for several tokens a block
    ("f32", 1, 1, 128, 64, [1250], [1250], 128, True, True),
]


@pytest.mark.parametrize("dtype,hq,hk,d,page,q_lens,kv,rot,inter,norms", APPEND)
def test_append(mp, dtype, hq, hk, d, page, q_lens, kv, rot, inter, norms):
    c = Cache(mp, dtype, hq, hk, d, page, kv, fill="none")
    cu, cu_t = offsets(q_lens)
    rows = cu[-1] + 2
    qkv = c.randn(rows, (hq + 2 * hk) * d + 16, by=2.0)[:, 8:-8] if dtype == "bf16" else c.randn(rows, (hq + 2 * hk) * d + 8, by=2.0)[:, 4:-4]
    q, k, v = qkv[:, :hq * d].unflatten(1, (hq, d)), qkv[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d)), qkv[:, (hq + hk) * d:].unflatten(1, (hk, d))
    qn, kn = (c.randn(d), c.randn(d)) if norms else (None, None)
    inv = (500000.0 ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64) / max(1, rot))).to(DEV) if rot else None
    eps = 1e-5
    slots = torch.cat([torch.arange(n - m, n) for m, n in zip(q_lens, kv)] + [torch.zeros(2, dtype=torch.int64)]).to(DEV)
    negative = any(m > n for m, n in zip(q_lens, kv))
    for positions in (None, torch.randint(0, 1 << 20, (rows,), generator=c.gen).to(DEV, torch.int32)):
        c.keys.fill_(5.0)
        c.values.fill_(5.0)
        q_out = torch.full((rows, hq, d), 77.0, dtype=c.dtype, device=DEV)
        mp.mp_cache_append(c.cfg, mp.make_rotary(rot_dim=rot, interleaved=inter, eps=eps), q, k, v, qn, kn, inv, positions, cu_t, c.kv_len,
                           c.keys, c.values, c.table, q_out, c.status)
        assert c.status.item() == (mp.MP_STATUS_BAD_LENGTH if negative else 0)
        c.status.zero_()
        pos = slots if positions is None else positions
        f = inv if inv is not None else torch.zeros(0, dtype=torch.float64, device=DEV)
        wq, sq = R.rotate(q, qn, eps, f, pos, rot, inter)
        wk, sk = R.rotate(k, kn, eps, f, pos, rot, inter)
        ok = lambda got, want, size: ((got.double() - want).abs() <= HALF[dtype] * want.abs() + (1 + HALF[dtype]) * 2.0 ** -18 * size).all()
        assert ok(q_out[:cu[-1]], wq[:cu[-1]], sq[:cu[-1]])
        assert (q_out[cu[-1]:] == 77.0).all()
        touched = torch.zeros(c.pages, c.ps, dtype=torch.bool, device=DEV)
        for b, (m, n) in enumerate(zip(q_lens, kv)):
            for i in range(m):
                s = n - m + i
                if s < 0:
                    continue
                p = b if c.table is None else int(c.table[b, s // c.ps])
                touched[p, s % c.ps] = True
                r = cu[b] + i
                assert ok(c.keys[p, :, s % c.ps], wk[r], sk[r])
                assert torch.equal(c.values[p, :, s % c.ps], v[r])
        for pool in (c.keys, c.values):
            assert (pool.transpose(1, 2)[~touched] == 5.0).all()


def test_append_past_the_end_of_the_cache(mp):
    """Tokens behind the cache's last slot are left out, the others stand where they belong."""
    c = Cache(mp, "bf16", 2, 1, 64, 16, [48], fill="none")
    c.keys.fill_(5.0)
    c.values.fill_(5.0)
    _, cu_t = offsets([6])
    c.kv_len[0] = 51  # three more than the table has room for: slots 45 to 50
    q, k, v = c.randn(6, 2, 64), c.randn(6, 1, 64), c.randn(6, 1, 64)
    q_out = torch.empty_like(q)
    mp.mp_cache_append(c.cfg, mp.make_rotary(rot_dim=0), q, k, v, None, None, None, None, cu_t, c.kv_len, c.keys, c.values, c.table, q_out,
                       c.status)
    assert c.status.item() == mp.MP_STATUS_BAD_LENGTH
    last = int(c.table[0, 2])
    assert torch.equal(c.keys[last, 0, 13:], k[:3, 0]) and torch.equal(c.values[last, 0, 13:], v[:3, 0])
    c.keys[last, 0, 13:] = 5.0
    assert (c.keys == 5.0).all() and torch.equal(q_out, q)


def test_append_far_positions_and_bad_pages(mp):
    """Angles of hundreds of millions of radians, negative positions, and a page outside the pool."""
    c = Cache(mp, "f32", 2, 1, 64, 16, [40], fill="none")
    _, cu_t = offsets([40])
    q, k, v = c.randn(40, 2, 64), c.randn(40, 1, 64), c.randn(40, 1, 64)
    inv = (10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32)).to(DEV)
    pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (40,), generator=c.gen).to(DEV, torch.int32)
    q_out = torch.empty_like(q)
    c.keys.fill_(5.0)
    c.values.fill_(5.0)
    c.table[0, 1] = c.pages
    mp.mp_cache_append(c.cfg, mp.make_rotary(rot_dim=64), q, k, v, None, None, inv, pos, cu_t, c.kv_len, c.keys, c.values, c.table, q_out,
                       c.status)
    assert c.status.item() == mp.MP_STATUS_BAD_PAGE
    want, size = R.rotate(q, None, 0.0, inv, pos, 64, False)
    # the product position * inv_freq is rounded in both: 2^31 * 2^-53 * 2 radians at most
    assert ((q_out.double() - want).abs() <= 2.0 ** -18 * size + 2.0 ** -20 * size).all()
    p0, p2 = int(c.table[0, 0]), int(c.table[0, 2])
    used = torch.zeros(c.pages, dtype=torch.bool)
    used[p0] = used[p2] = True
    assert torch.equal(c.values[p0, 0], v[:16, 0]) and torch.equal(c.values[p2, 0, :8], v[32:, 0])
    assert (c.keys[~used.to(DEV)] == 5.0).all() and (c.values[p2, 0, 8:] == 5.0).all()


# ---- eviction ----

EVICT = [
    # dtype, kv heads, d, page, destination page, cache lengths, budget, sinks, window, scores
    ("bf16", 2, 128, 16, 16, [100, 40, 64], 50, 4, 16, "normal"),
    ("bf16", 3, 64, 0, 0, [5000], 700, 4, 64, "heavy"),
    ("bf16", 1, 128, 64, 0, [1025, 1], 1024, 0, 0, "normal"),
    ("f32", 2, 64, 0, 32, [300, 0, 299], 299, 1, 0, "ties"),
    ("f32", 2, 128, 48, 16, [2049, 2048], 64, 4, 60, "normal"),     # nothing wanted between sinks and window
    ("bf16", 2, 64, 32, 32, [513, 77], 1, 0, 0, "ties"),
    ("bf16", 2, 64, 16, 16, [333], 100, 0, 1, "odd"),
    ("bf16", 1, 64, 0, 0, [40000], 33000, 4, 64, "ties"),
    ("bf16", 1, 64, 0, 0, [300001], 2000, 4, 64, "normal"),          # more scores than shared memory holds
]


def make_scores(kind, shape, gen):
    x = torch.randn(shape, generator=gen)
    if kind == "heavy":
        x = (x * 3).exp()
    if kind == "ties":
        x = (x * 2).round().abs() * 0.5
    if kind == "odd":  # both zeros, infinities, NaN, the smallest numbers, negative ones
        pick = torch.randint(0, 8, shape, generator=gen)
        special = torch.tensor([0.0, -0.0, math.inf, -math.inf, math.nan, 1e-45, -1e-45, -2.0])
        x = torch.where(torch.rand(shape, generator=gen) < 0.7, special[pick], x)
    return x.to(DEV)


@pytest.mark.parametrize("dtype,hk,d,page,dpage,kv,budget,sink,window,kind", EVICT)
def test_evict(mp, dtype, hk, d, page, dpage, kv, budget, sink, window, kind):
    c = Cache(mp, dtype, hk, hk, d, page, kv)
    t = Cache(mp, dtype, hk, hk, d, dpage, [min(n, budget) for n in kv], seed=5, cap=budget + 3, fill="none")
    t.keys.fill_(9.0)
    t.values.fill_(9.0)
    sc = make_scores(kind, (len(kv), hk, c.ps * c.cols), c.gen)
    for full in (True, False):
        dsc = torch.full((len(kv), hk, t.ps * t.cols), 9.0, device=DEV) if full else None
        kept = torch.full((len(kv), hk, budget), -5, dtype=torch.int32, device=DEV) if full else None
        dlen = torch.full((len(kv),), -1, dtype=torch.int32, device=DEV)
        ws = torch.full((mp.mp_evict_workspace_bytes(c.cfg, max(1, max(kv)), budget),), 0xFF, dtype=torch.uint8, device=DEV)
        t.keys.fill_(9.0)
        t.values.fill_(9.0)
        mp.mp_cache_evict(c.cfg, t.cfg, c.keys, c.values, c.table, c.kv_len, max(1, max(kv)), sc, sink, window, budget, t.keys, t.values,
                          t.table, dsc, dlen, kept, ws, c.status)
        assert c.status.item() == 0
        want_keys, want_values = torch.full_like(t.keys, 9.0), torch.full_like(t.values, 9.0)
        for b, n in enumerate(kv):
            for h in range(hk):
                want = R.keep(sc[b, h], n, sink, window, budget)
                m = len(want)
                assert int(dlen[b]) == m == min(n, budget)
                at = torch.tensor(want, dtype=torch.int64, device=DEV)
                if full:
                    assert kept[b, h, :m].tolist() == want
                    assert (kept[b, h, m:] == -5).all()
                    assert torch.equal(dsc[b, h, :m].view(torch.int32), sc[b, h][at].view(torch.int32))
                    assert (dsc[b, h, m:] == 9.0).all()
                k, v = (pool_rows(pool, c, b, h, n)[at] for pool in (c.keys, c.values))
                for i, p in enumerate(R.pages_of(t.table, b, m, t.ps)):
                    e = min(t.ps, m - i * t.ps)
                    want_keys[p, h, :e], want_values[p, h, :e] = k[i * t.ps:i * t.ps + e], v[i * t.ps:i * t.ps + e]
        assert torch.equal(t.keys, want_keys) and torch.equal(t.values, want_values)


def pool_rows(pool, c, b, h, n):
    parts = [pool[p, h, :min(c.ps, n - i * c.ps)] for i, p in enumerate(R.pages_of(c.table, b, n, c.ps))]
    return torch.cat(parts) if parts else pool.new_zeros(0, c.d)


def test_evict_skips_bad_destination_pages(mp):
    c = Cache(mp, "bf16", 2, 2, 64, 16, [100])
    t = Cache(mp, "bf16", 2, 2, 64, 16, [48], cap=48, fill="none")
    t.keys.fill_(9.0)
    t.values.fill_(9.0)
    t.table[0, 1] = -3
    sc = make_scores("normal", (1, 2, c.ps * c.cols), c.gen)
    dlen = torch.zeros(1, dtype=torch.int32, device=DEV)
    ws = torch.empty(mp.mp_evict_workspace_bytes(c.cfg, 100, 48), dtype=torch.uint8, device=DEV)
    mp.mp_cache_evict(c.cfg, t.cfg, c.keys, c.values, c.table, c.kv_len, 100, sc, 4, 8, 48, t.keys, t.values, t.table, None, dlen, None, ws,
                      c.status)
    assert c.status.item() == mp.MP_STATUS_BAD_PAGE
    used = [int(t.table[0, 0]), int(t.table[0, 2])]
    for p in range(t.pages):
        assert bool((t.keys[p] != 9.0).all()) == (p in used)


# ---- together ----

def test_a_captured_step_follows_the_lengths(mp):
    """One generated token's append, attention, weights and eviction in one graph, replayed
    while the sequence grows (what a serving loop captures once), in fp32 and bf16."""
    for dtype in ("bf16", "f32"):
        c = Cache(mp, dtype, 4, 2, 64, 16, [0, 0], cap=200, fill="none")
        c.keys.zero_()
        c.values.zero_()
        full = torch.arange(2 * c.cols, dtype=torch.int32, device=DEV).view(2, c.cols)
        c.table.copy_(full)
        cu, cu_t = offsets([1, 1])
        q, k, v = c.randn(2, 4, 64), c.randn(2, 2, 64), c.randn(2, 2, 64)
        q_out, out, lse = torch.empty_like(q), torch.empty_like(q), torch.empty(2, 4, device=DEV)
        inv = (10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32)).to(DEV)
        scores = torch.zeros(2, 2, c.ps * c.cols, device=DEV)
        ws = torch.empty(max(1, mp.mp_chunk_workspace_bytes(c.cfg, 2, 1, 200)), dtype=torch.uint8, device=DEV)
        t = Cache(mp, dtype, 4, 2, 64, 0, [20, 20], cap=20, fill="none")
        dlen, kept = torch.zeros(2, dtype=torch.int32, device=DEV), torch.zeros(2, 2, 20, dtype=torch.int32, device=DEV)
        ews = torch.empty(mp.mp_evict_workspace_bytes(c.cfg, 200, 20), dtype=torch.uint8, device=DEV)

        def step():
            mp.mp_cache_append(c.cfg, mp.make_rotary(rot_dim=64), q, k, v, None, None, inv, None, cu_t, c.kv_len, c.keys, c.values, c.table,
                               q_out, c.status)
            mp.mp_chunk_attention(c.cfg, q_out, cu_t, c.kv_len, 1, 200, c.keys, c.values, c.table, out, lse, ws, c.status)
            mp.mp_cache_weights(c.cfg, q_out, lse, cu_t, c.kv_len, 1, 200, c.keys, c.table, scores, c.status)
            mp.mp_cache_evict(c.cfg, t.cfg, c.keys, c.values, c.table, c.kv_len, 200, scores, 2, 4, 20, t.keys, t.values, None, None, dlen,
                              kept, ews, c.status)

        st = torch.cuda.Stream()
        c.kv_len.fill_(1)
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            step()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=st):
                step()
        scores.zero_()
        want = torch.zeros(2, 2, c.ps * c.cols, dtype=torch.float64, device=DEV)
        for n in range(1, 60):
            c.kv = [n, max(1, n - 5)]
            c.kv_len.copy_(torch.tensor(c.kv, dtype=torch.int32))
            q.copy_(c.randn(2, 4, 64))
            k.copy_(c.randn(2, 2, 64))
            v.copy_(c.randn(2, 2, 64))
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            check_attention(c, dtype, q_out, cu, out, lse)
            want = R.weights(q_out, lse, cu, c.kv, c.keys, c.table, want)[0]
        # each step adds one exponential's error (2^-21 and the logits'), weighted as the sum is
        assert ((scores.double() - want).abs() <= 2.0 ** -16 * want).all()
        assert c.status.item() == 0 and dlen.tolist() == [20, 20]
        for b, n in enumerate(c.kv):
            for h in range(2):
                keep = R.keep(scores[b, h], n, 2, 4, 20)
                assert kept[b, h].tolist() == keep
                assert torch.equal(t.keys[b, h], pool_rows(c.keys, c, b, h, n)[torch.tensor(keep, device=DEV)])


def test_a_prompt_in_chunks_then_eviction_then_sampled_decode(mp):
    """The operators as a serving loop uses them on one dense layer: a prompt arrives in
    chunks (append, attention, weights), the cache is cut to its budget, the hash tables are
    built over what is left, and generation goes on with mp_cache_append and mp_decode_step
    (K = 0: every key is sampled, so the sampled attention is exact and comparable)."""
    import workloads as WL
    hq, hk, d, prompt, budget, steps = 8, 2, 128, 1000, 400, 3
    g = torch.Generator().manual_seed(11)
    rnd = lambda *s: torch.randn(*s, generator=g).to(DEV, torch.bfloat16)
    inv = (500000.0 ** (-torch.arange(64, dtype=torch.float64) / 64)).to(DEV)
    rotary = mp.make_rotary(rot_dim=d)
    qn, kn = rnd(d).abs() + 0.5, rnd(d).abs() + 0.5
    shape = dict(batch=1, kv_heads=hk, q_heads=hq, head_dim=d, n_pages=1, dtype="bf16")
    cfg = mp.make_cache_config(page_size=prompt, **shape)
    keys, values = (torch.full((1, hk, prompt, d), math.nan, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    scores = torch.zeros(1, hk, prompt, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    kv_len = torch.zeros(1, dtype=torch.int32, device=DEV)
    want_scores = torch.zeros(1, hk, prompt, dtype=torch.float64, device=DEV)
    at = 0
    for m in (300, 500, 200):
        cu, cu_t = offsets([m])
        q, k, v = rnd(m, hq, d), rnd(m, hk, d), rnd(m, hk, d)
        kv_len.fill_(at + m)
        q_out, out, lse = torch.empty_like(q), torch.empty_like(q), torch.empty(m, hq, device=DEV)
        mp.mp_cache_append(cfg, rotary, q, k, v, qn, kn, inv, None, cu_t, kv_len, keys, values, None, q_out, status)
        ws = torch.empty(max(1, mp.mp_chunk_workspace_bytes(cfg, m, m, prompt)), dtype=torch.uint8, device=DEV)
        mp.mp_chunk_attention(cfg, q_out, cu_t, kv_len, m, prompt, keys, values, None, out, lse, ws, status)
        mp.mp_cache_weights(cfg, q_out, lse, cu_t, kv_len, m, prompt, keys, None, scores, status)
        at += m

        class C:
            pass
        c = C()
        c.kv, c.keys, c.values, c.table, c.hk, c.d = [at], keys, values, None, hk, d
        check_attention(c, "bf16", q_out, cu, out, lse)
        want_scores = R.weights(q_out, lse, cu, [at], keys, None, want_scores)[0]
    assert ((scores.double() - want_scores).abs() <= 2.0 ** -10 * want_scores).all()

    capacity = budget + steps
    dst = mp.make_cache_config(page_size=capacity, **shape)
    dk, dv = (torch.zeros(1, hk, capacity, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    dlen, kept = torch.zeros(1, dtype=torch.int32, device=DEV), torch.zeros(1, hk, budget, dtype=torch.int32, device=DEV)
    ws = torch.empty(mp.mp_evict_workspace_bytes(cfg, prompt, budget), dtype=torch.uint8, device=DEV)
    mp.mp_cache_evict(cfg, dst, keys, values, None, kv_len, prompt, scores, 4, 64, budget, dk, dv, None, None, dlen, kept, ws, status)
    assert int(dlen) == budget
    for h in range(hk):
        want = R.keep(scores[0, h], prompt, 4, 64, budget)
        assert kept[0, h].tolist() == want
        assert torch.equal(dk[0, h, :budget], keys[0, h][torch.tensor(want, device=DEV)])

    lsh = mp.make_config(layers=1, batch=1, kv_heads=hk, q_heads=hq, head_dim=d, K=0, L=4, n_sink=4, window=64, capacity=capacity, dtype="bf16")
    tables = torch.empty(mp.mp_tables_layout_get(lsh).total_bytes, dtype=torch.uint8, device=DEV)
    scratch = torch.empty(mp.mp_decode_layout_get(lsh).total_bytes, dtype=torch.uint8, device=DEV)
    mp.mp_build_tables(lsh, dk, budget, None, tables)
    for i in range(steps):
        cu, cu_t = offsets([1])
        q, k, v = rnd(1, hq, d), rnd(1, hk, d), rnd(1, hk, d)
        kv_len.fill_(budget + i + 1)
        pos = torch.tensor([prompt + i], dtype=torch.int32, device=DEV)  # where the token stands, not its slot
        q_out = torch.empty_like(q)
        mp.mp_cache_append(dst, rotary, q, k, v, qn, kn, inv, pos, cu_t, kv_len, dk, dv, None, q_out, status)
        sampled = torch.empty(1, 1, hq, d, dtype=torch.float32, device=DEV)
        mp.mp_decode_step(lsh, tables, dk, dv, budget + i, q_out, sampled, scratch)
        out, lse = torch.empty_like(q), torch.empty(1, hq, device=DEV)
        ws = torch.empty(max(1, mp.mp_chunk_workspace_bytes(dst, 1, 1, capacity)), dtype=torch.uint8, device=DEV)
        mp.mp_chunk_attention(dst, q_out, cu_t, kv_len, 1, capacity, dk, dv, None, out, lse, ws, status)
        c = C()
        c.kv, c.keys, c.values, c.table, c.hk, c.d = [budget + i + 1], dk, dv, None, hk, d
        check_attention(c, "bf16", q_out, cu, out, lse)
        exact = R.attention(q_out, cu, c.kv, dk, dv, None, hk)[0]
        assert (sampled[0].double() - exact).norm() <= 2e-3 * exact.norm()
    assert status.item() == 0
    assert mp.mp_get_status(tables) == 0
