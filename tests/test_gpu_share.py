"""Planning a step, attention over shared prefixes and the rotation of cached keys on the GPU against
plain forms, at the sizes, masks, pages and lengths where they can go wrong.

Tolerances, with h = half a step of a type relative to the value (fp32 2^-24, bf16 2^-8):
- planning: whole numbers, equal.
- attention: that of the chunk's (test_gpu_cache.py) over prefix and own slots together: the join of the two
  passes is part of the sums of n terms and of the exponentials counted there.
- rotation: one final rounding, h |y|, plus fp32 arithmetic on the pair (a, b): sine and cosine off by
  2^-20 in bf16 (2^-23 in fp32) each, so sqrt(2) times that of the pair's size, the scale's rounding, two
  products and a sum: below 2^-18 of the size in bf16 and 2^-20 in fp32. The reference's own angle is a double
  of up to 2^31 positions and is off by 2^-53 of it: 2^-22 of a turn at most, for positions below 2^20 2^-33.
"""
import math
import os
import random
import subprocess
import sys

import pytest
import torch

import cache_reference as R
import share_reference as S
from test_gpu_cache import DEV, DT, HALF, Cache, offsets

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mp():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import lsh_sampled_sparse_centered_gb300 as m
    return m


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


# ----------------------------------------------------------------------------------
# planning
# ----------------------------------------------------------------------------------

class Plan:
    """A pool whose pages are dealt to sequences of the lengths `kv` in no order."""

    def __init__(self, mp, kv, page, cols, spare, seed=0, table=True):
        rng = random.Random(seed)
        self.mp, self.kv, self.page, self.cols, self.batch = mp, list(kv), page, cols, len(kv)
        used = [-(-n // page) for n in kv]
        self.pages = sum(used) + spare if table else self.batch
        order = list(range(self.pages))
        rng.shuffle(order)
        self.table = [[-9] * cols for _ in kv] if table else None
        if table:
            for b, u in enumerate(used):
                self.table[b][:u] = [order.pop() for _ in range(u)]
        self.free = order + [-5] * (self.pages - len(order))
        self.n_free = len(order) if table else 0
        self.base = [rng.randint(0, 10 ** 6) for _ in kv]
        self.cfg = mp.make_cache_config(batch=self.batch, kv_heads=1, q_heads=1, head_dim=64, page_size=page, n_pages=self.pages, max_pages=cols)
        self.d_table, self.d_free = (ints(self.table), ints(self.free)) if table else (None, None)
        self.d_kv, self.d_n, self.status = ints(self.kv), ints([self.n_free]), ints([0])

    def step(self, change, max_rows, in_place=True, rows=(True, True, True), base=True, stream=None):
        """One call and its plain form; both states go on. The status bits that the call has set."""
        mp = self.mp
        lens, left = (self.d_kv, self.d_n) if in_place else (torch.full_like(self.d_kv, -1), torch.full_like(self.d_n, -1))
        cu = torch.full((self.batch + 1,), -1, dtype=torch.int32, device=DEV)
        out = [torch.full((max_rows + 2,), 77, dtype=torch.int32, device=DEV) if r else None for r in rows]
        paged = self.table is not None
        mp.mp_cache_plan(self.cfg, ints(change), ints(self.base) if base else None, self.d_kv, self.d_n if paged else None, max_rows, self.d_table,
                         self.d_free, lens, left if paged else None, cu, *out, self.status, stream=stream)
        self.d_kv, self.d_n = lens, left
        want = S.plan(change, self.kv, self.base if base else [0] * self.batch, self.table, self.free, self.n_free, self.page, self.cols, max_rows)
        self.kv, self.n_free, cu_want, self.table, self.free, named = want
        assert lens.tolist() == self.kv and cu.tolist() == cu_want
        if paged:
            assert left.tolist() == [self.n_free]
            assert self.d_table.tolist() == self.table and self.d_free.tolist() == self.free
        for i, x in enumerate(out):
            if x is not None:
                assert x.tolist() == [r[i] for r in named] + [77] * (max_rows + 2 - len(named)), i
        bits = self.status.item()
        self.status.zero_()
        return bits


@pytest.mark.parametrize("batch,page,cols,max_rows", [(1, 16, 1, 1), (1, 16, 40, 300), (5, 48, 7, 30), (33, 16, 20, 64), (64, 64, 30, 64), (1024, 16, 9, 500),
                                                      (1025, 32, 5, 4000), (3000, 16, 3, 1)])
def test_plan_over_many_steps(mp, batch, page, cols, max_rows):
    """Growth, rollback, ends and pauses by chance over a pool that sometimes runs out."""
    rng = random.Random(batch)
    cap = page * cols
    p = Plan(mp, [rng.randint(0, cap) if rng.random() < 0.8 else rng.choice((0, page, cap)) for _ in range(batch)], page, cols,
             spare=max(1, batch * cols // 4), seed=batch)
    seen = 0
    for step in range(12):
        change = [rng.choice((0, 1, 1, 1, rng.randint(1, 2 * page), -rng.randint(1, 8), -n, -n - 3, page, -page)) for n in p.kv]
        change = [min(x, cap - n) for x, n in zip(change, p.kv)]  # none outgrows its table here
        bits = p.step(change, max_rows, in_place=step % 2 == 0, rows=[(True, True, True), (True, False, False), (False, True, False), (False, False, True)][step % 4],
                      base=step % 3 != 0)
        assert bits & ~mp.MP_STATUS_NO_ROOM == 0
        seen |= bits
        assert sum(-(-n // page) for n in p.kv) + p.n_free == p.pages  # no page is lost
    assert seen or max_rows >= 64


def test_plan_takes_back_before_it_gives(mp):
    """A full pool: what one sequence drops, another takes in the same step, the last page first."""
    p = Plan(mp, [64, 100, 16], 16, 20, spare=0)
    mine = p.table[1][5:7]
    assert p.step([20, -20, 0], 100) == 0
    assert p.table[0][4:6] == mine[::-1] and p.n_free == 0
    assert p.step([13, 0, 0], 100) == mp.MP_STATUS_NO_ROOM and p.kv == [84, 80, 16]


def test_plan_leaves_the_last_sequences_waiting(mp):
    p = Plan(mp, [16, 16, 16, 5, 16], 16, 20, spare=2)
    # the third needs a page that is not there, and the ones behind it wait too, need a page or not
    assert p.step([1, 1, 1, 1, 1], 100) == mp.MP_STATUS_NO_ROOM and p.kv == [17, 17, 16, 5, 16]
    # rows run out: two of three tokens would fit, none is given
    assert p.step([1, 2, 0, 1, -16], 2) == mp.MP_STATUS_NO_ROOM and p.kv == [18, 17, 16, 5, 0]
    # a drop is done wherever the sequence stands
    assert p.step([1, 2, 0, 1, 0], 4) == 0 and p.kv == [19, 19, 16, 6, 0]
    assert p.step([0, 0, 0, 0, 0], 0) == 0 and p.step([-1, 0, -30, -6, 0], 0) == 0 and p.kv == [18, 19, 0, 0, 0]


def test_plan_of_a_sequence_that_outgrows_its_table(mp):
    p = Plan(mp, [30, 7, 64], 16, 4, spare=9)
    assert p.step([35, 3, 1], 100) == mp.MP_STATUS_BAD_LENGTH and p.kv == [30, 10, 64]
    assert p.step([34, 2 ** 31 - 1, 0], 100) == mp.MP_STATUS_BAD_LENGTH and p.kv == [64, 10, 64]
    assert p.step([0, -2 ** 31, -1], 100) == 0 and p.kv == [64, 0, 63]


def test_plan_of_a_dense_cache(mp):
    for batch in (1, 40, 1500):
        rng = random.Random(batch)
        p = Plan(mp, [rng.randint(0, 77) for _ in range(batch)], 77, 1, spare=0, table=False)
        for _ in range(4):
            bits = p.step([rng.choice((0, 1, 5, -3)) for _ in range(batch)], 6 * batch)
            assert bits & ~mp.MP_STATUS_BAD_LENGTH == 0


def test_plan_of_the_most_sequences_and_long_chunks(mp):
    rng = random.Random(5)
    p = Plan(mp, [rng.randint(0, 40) for _ in range(mp.MP_PLAN_SEQUENCES)], 16, 8, spare=30000)
    assert p.step([rng.choice((1, 1, 60, -4)) for _ in p.kv], 200000) == 0
    q = Plan(mp, [100, 3, 0], 64, 4000, spare=9000)
    assert q.step([200000, 1, 55555], 300000) == 0


def test_plan_with_damaged_lengths_and_pages(mp):
    """Whatever the arrays hold, the bits are set and nothing outside them is written."""
    p = Plan(mp, [40, 50, 60, 70], 16, 8, spare=10)
    p.d_table[1, 3] = 10 ** 9  # moved as it is, as a page given back and as an old page that rows go to
    p.d_table[2, 3] = -1
    lens, left, cu = torch.zeros_like(p.d_kv), torch.zeros_like(p.d_n), torch.zeros(5, dtype=torch.int32, device=DEV)
    rows = [torch.full((100,), 77, dtype=torch.int32, device=DEV) for _ in range(3)]
    mp.mp_cache_plan(p.cfg, ints([0, -20, 2, 1]), None, p.d_kv, p.d_n, 100, p.d_table, p.d_free, lens, left, cu, *rows, p.status)
    assert p.status.item() == mp.MP_STATUS_BAD_PAGE
    assert lens.tolist() == [40, 30, 62, 71] and left.tolist() == [12] and p.d_free.tolist()[10:12] == [p.table[1][2], 10 ** 9]
    assert rows[1].tolist()[:3] == [-1, -1, p.table[3][4] * 16 + 6] and rows[0].tolist()[:3] == [60, 61, 70]
    p.status.zero_()
    # lengths and the count of free pages outside their limits; pages given back beyond the pool's number
    for kv, n, bits in (([-4, 10 ** 9, 20, 30], 5, mp.MP_STATUS_BAD_LENGTH), ([1, 2, 3, 4], 10 ** 8, mp.MP_STATUS_BAD_LENGTH), ([1, 2, 3, 4], -3, mp.MP_STATUS_BAD_LENGTH),
                        ([40, 50, 60, 70], p.pages - 1, mp.MP_STATUS_BAD_LENGTH)):
        p = Plan(mp, [40, 50, 60, 70], 16, 8, spare=10)
        p.d_free[:] = 0
        p.d_table[:] = 1
        mp.mp_cache_plan(p.cfg, ints([-9, -100, 5, -30]), None, ints(kv), ints([n]), 100, p.d_table, p.d_free, lens, left, cu, *rows, p.status)
        assert p.status.item() & bits, (kv, n)
        assert 0 <= left.item() <= p.pages and all(0 <= x <= 128 for x in lens.tolist()) and cu.tolist() == sorted(cu.tolist())
        assert set(p.d_free.tolist()) <= {0, 1}


def test_plan_captured_runs_a_loop(mp):
    """A captured step that updates lengths and free pages in place, on a stream of its own."""
    for batch, page in ((6, 16), (1200, 16)):
        p = Plan(mp, [10] * batch, page, 6, spare=3 * batch)
        change, base = ints([1] * batch), ints(p.base)
        cu = torch.zeros(batch + 1, dtype=torch.int32, device=DEV)
        rows = [torch.zeros(2 * batch, dtype=torch.int32, device=DEV) for _ in range(3)]
        st = torch.cuda.Stream()
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=st):
            mp.mp_cache_plan(p.cfg, change, base, p.d_kv, p.d_n, 2 * batch, p.d_table, p.d_free, p.d_kv, p.d_n, cu, *rows, p.status)
        kv, n_free, table, free = p.kv, p.n_free, p.table, p.free
        for step in range(9):
            x = [(1, 2, -5)[(b + step) % 3] for b in range(batch)]
            change.copy_(ints(x))
            g.replay()
            torch.cuda.synchronize()
            kv, n_free, cu_want, table, free, named = S.plan(x, kv, p.base, table, free, n_free, page, 6, 2 * batch)
            assert p.d_kv.tolist() == kv and p.d_n.tolist() == [n_free] and p.d_table.tolist() == table and p.d_free.tolist() == free
            assert cu.tolist() == cu_want and rows[1].tolist()[:len(named)] == [r[1] for r in named]


def test_plans_on_two_streams(mp):
    """Two layers' pools planned at once share nothing."""
    ps = [Plan(mp, [10 + i] * 1500, 16, 30, spare=9000, seed=i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    args = []
    for p in ps:
        args.append((ints([3] * 1500), [torch.zeros(9000, dtype=torch.int32, device=DEV) for _ in range(3)], torch.zeros(1501, dtype=torch.int32, device=DEV)))
    torch.cuda.synchronize()
    for _ in range(20):
        for p, (change, rows, cu), st in zip(ps, args, streams):
            mp.mp_cache_plan(p.cfg, change, None, p.d_kv, p.d_n, 9000, p.d_table, p.d_free, p.d_kv, p.d_n, cu, *rows, p.status, stream=st)
    torch.cuda.synchronize()
    for p, (_, rows, cu) in zip(ps, args):
        kv, n_free, table, free = p.kv, p.n_free, p.table, p.free
        for _ in range(20):
            kv, n_free, cu_want, table, free, named = S.plan([3] * 1500, kv, [0] * 1500, table, free, n_free, 16, 30, 9000)
        assert p.d_kv.tolist() == kv and p.d_n.tolist() == [n_free] and p.d_table.tolist() == table and p.d_free.tolist() == free
        assert cu.tolist() == cu_want and [r.tolist()[:4500] for r in rows] == [[r[i] for r in named] for i in range(3)]


# ----------------------------------------------------------------------------------
# prefixes
# ----------------------------------------------------------------------------------

class Shared(Cache):
    """The sequences' own slots and the prefixes of their groups, in one pool where there are pages.
    Everything behind their ends is NaN."""

    def __init__(self, mp, dtype, hq, hk, d, page, kv, groups, prefixes, seed=0, cap=None, pcap=None, ppage=None):
        super().__init__(mp, dtype, hq, hk, d, page, kv, seed=seed, cap=cap)
        self.groups, self.prefixes = list(groups), list(prefixes)
        ppage = page if ppage is None else ppage
        self.pre = Cache(mp, dtype, hq, hk, d, ppage, prefixes, seed=seed + 1, cap=pcap)
        if page and page == ppage:  # one pool
            n = self.pages
            self.keys, self.values = (torch.cat((x, y)) for x, y in ((self.keys, self.pre.keys), (self.values, self.pre.values)))
            self.pages = n + self.pre.pages
            self.pre.table = torch.where(self.pre.table >= 0, self.pre.table + n, self.pre.table)
            self.pre.keys, self.pre.values, self.pre.pages = self.keys, self.values, self.pages
            for c in (self, self.pre):
                c.cfg = mp.make_cache_config(batch=len(c.kv), kv_heads=hk, q_heads=hq, head_dim=d, page_size=page, n_pages=self.pages, max_pages=c.cols, dtype=dtype)
        cg = offsets(self.groups)
        self.cu_group = cg[1]
        assert cg[0][-1] <= len(kv)

    def limits(self, cu):
        most, at = 1, 0
        for n in self.groups:
            most, at = max(most, cu[at + n] - cu[at]), at + n
        return most, max(1, max(self.prefixes))


def attend_prefix(mp, c, q, cu, cu_t, max_q, max_kv=None, group_q=None, max_prefix=None, lse=True, stream=None, workspace=None):
    max_kv = max_kv or max(1, max(c.kv))
    g, l = c.limits(cu)
    g, l = group_q or g, max_prefix or l
    out = torch.full_like(q, 77.0)
    z = torch.full(q.shape[:2], 77.0, device=DEV) if lse else None
    size = mp.mp_prefix_workspace_bytes(c.cfg, c.pre.cfg, q.shape[0], max_q, max_kv, g, l)
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device=DEV) if workspace is None else workspace
    mp.mp_prefix_attention(c.cfg, c.pre.cfg, q, cu_t, c.kv_len, max_q, max_kv, c.keys, c.values, c.table, c.cu_group, c.pre.kv_len, g, l,
                           c.pre.keys, c.pre.values, c.pre.table, out, z, ws, c.status, stream=stream)
    return out, z


def check_prefix(c, dtype, q, cu, out, lse):
    want, z, spread, slack = S.prefix_attention(q, cu, c.kv, c.keys, c.values, c.table, c.groups, c.prefixes, c.pre.keys, c.pre.values,
                                                c.pre.table, c.hk)
    n, slots = cu[-1], max(c.kv) + max(c.prefixes)
    eps_x = (c.d + 8) * 2.0 ** -24 * slack[:n]
    rel = 2 * eps_x + slots * 2.0 ** -24 + 2.0 ** -20 + (2.0 ** -8 if dtype == "bf16" else 0.0)
    tol = HALF[dtype] * want[:n].abs() + (1 + HALF[dtype]) * rel[..., None] * spread[:n]
    assert torch.isfinite(out[:n]).all()
    err = (out[:n].double() - want[:n]).abs()
    assert (err <= tol).all(), (err - tol).max().item()
    if lse is not None:
        empty = torch.isinf(z[:n])
        assert torch.equal(torch.isinf(lse[:n]) & (lse[:n] < 0), empty)
        ztol = eps_x + (slots + 8) * 2.0 ** -24 + 2.0 ** -21 * (1 + z[:n].abs())
        assert ((lse[:n].double() - z[:n]).abs()[~empty] <= ztol[~empty]).all()
    assert (out[n:] == 77.0).all() and (lse is None or (lse[n:] == 77.0).all())  # rows behind the last sequence


PREFIX = [
    # dtype, q heads, kv heads, d, page, chunk lengths, own lengths, groups, prefixes
    ("bf16", 4, 2, 64, 0, [1], [1], [1], [1]),
    ("bf16", 8, 2, 128, 16, [1, 1, 1], [1, 17, 300], [3], [333]),
    ("bf16", 8, 2, 128, 64, [1, 1], [64, 100], [2], [5000]),                      # few rows over a long prefix
    ("bf16", 32, 8, 128, 64, [1] * 5, [1, 2, 3, 4, 5], [5], [130]),                # more than 16 rows of a group, few of a sequence
    ("bf16", 8, 1, 128, 16, [1] * 33, [1 + 7 * i for i in range(33)], [33], [777]),  # 264 rows: two tiles
    ("bf16", 8, 1, 64, 48, [1] * 40, [1 + 3 * i for i in range(40)], [40], [1000]),
    ("bf16", 7, 7, 64, 0, [1] * 20, [5 + i for i in range(20)], [20], [257]),        # no grouping of heads
    ("bf16", 12, 1, 128, 48, [1, 2, 1], [777, 50, 3], [2], [100]),                 # a sequence without a prefix
    ("bf16", 40, 1, 64, 32, [1, 1], [500, 2], [1, 1], [64, 65]),
    ("bf16", 6, 2, 64, 16, [3, 2, 5, 1], [3, 1000, 77, 1], [2, 0, 2], [129, 50, 128]),  # a group of no sequences
    ("bf16", 4, 2, 128, 128, [129, 1, 127], [129, 640, 1000], [3], [300]),          # chunks of both passes on large tiles
    ("bf16", 28, 4, 128, 64, [37, 100], [37, 411], [1, 1], [0, 900]),               # an empty prefix
    ("bf16", 16, 2, 64, 256, [200, 1], [1111, 4], [2], [2000]),
    ("bf16", 8, 2, 128, 16, [0, 5, 0, 40, 1], [9, 5, 0, 300, 0], [2, 3], [77, 40]),  # empty chunks, a token of an empty cache
    ("bf16", 8, 2, 64, 16, [9, 70], [4, 33], [2], [45]),                           # tokens at negative slots see the prefix alone
    ("bf16", 8, 2, 64, 16, [9, 70], [4, 33], [2], [0]),                            # and nothing at all
    ("bf16", 32, 8, 128, 0, [513, 20], [2500, 20], [2], [1500]),
    ("bf16", 136, 1, 64, 32, [3, 1], [100, 40], [2], [333]),                       # a group of heads of more than 128
    ("bf16", 4, 4, 128, 16, [1, 2, 3, 4, 5, 6], [9, 9, 9, 9, 9, 9], [1, 2, 1], [700, 16, 1]),
    ("f32", 4, 2, 64, 0, [1], [1], [1], [1]),
    ("f32", 8, 2, 128, 16, [1, 1, 3], [17, 2000, 64], [3], [1500]),
    ("f32", 6, 2, 64, 48, [65, 1, 0, 2], [200, 1500, 9, 3], [1, 2], [129, 64]),
    ("f32", 8, 8, 128, 0, [100, 3], [333, 400], [2], [70]),
    ("f32", 8, 1, 64, 32, [9, 70], [4, 33], [1, 1], [3, 0]),
]


@pytest.mark.parametrize("dtype,hq,hk,d,page,q_lens,kv,groups,prefixes", PREFIX)
def test_prefix_attention(mp, dtype, hq, hk, d, page, q_lens, kv, groups, prefixes):
    c = Shared(mp, dtype, hq, hk, d, page, kv, groups, prefixes)
    cu, cu_t = offsets(q_lens)
    q = c.randn(cu[-1] + 3, hq, d, by=1.5)  # three rows that belong to no sequence
    out, lse = attend_prefix(mp, c, q, cu, cu_t, max(q_lens))
    check_prefix(c, dtype, q, cu, out, lse)
    assert c.status.item() == 0
    # the same bits again, without lse; and wider limits, which may split the same slots otherwise
    again, _ = attend_prefix(mp, c, q, cu, cu_t, max(q_lens), lse=False)
    assert torch.equal(again[:cu[-1]], out[:cu[-1]])
    wide, z = attend_prefix(mp, c, q, cu, cu_t, max(q_lens) + 50, max_kv=c.ps * c.cols, group_q=c.limits(cu)[0] + 70, max_prefix=c.pre.ps * c.pre.cols)
    check_prefix(c, dtype, q, cu, wide, z)
    assert c.status.item() == 0


@pytest.mark.parametrize("hq,hk,d,page,q_lens,groups,prefixes", [
    (32, 8, 128, 64, [1] * 20, [20], [9000]),          # 80 rows: several steps of each half
    (40, 40, 64, 16, [1] * 20, [20], [12000]),         # many steps of each half
    (16, 16, 128, 0, [1] * 24, [24], [7777]),
    (32, 8, 64, 48, [1] * 11, [5, 6], [5000, 900]),    # pieces of two prefixes in one CTA
    (16, 2, 128, 16, [1] * 40, [40], [6000]),          # 320 rows: two tiles side by side
    (16, 2, 64, 0, [3] * 30, [30], [6001]),
    (40, 40, 128, 32, [1] * 300, [300], [700]),        # more tiles than half of the SMs: equal runs
    # own rows in eights, sixteens and more beside one half's rows and beside whole tiles
    (32, 8, 128, 64, [4, 1, 3, 4, 2, 4, 4, 4], [8], [12001]),
    (32, 8, 64, 16, [4, 1, 3, 4, 2, 4, 4, 4], [8], [12001]),
    (32, 8, 128, 48, [8, 1, 3, 4, 2, 6, 4, 4], [8], [9999]),
    (32, 8, 64, 0, [8, 1, 3, 4, 2, 6, 4, 4], [8], [20000]),
    (16, 2, 128, 0, [4, 3, 2, 1] * 10, [40], [9000]),
    (16, 2, 128, 16, [2, 1] * 20, [40], [8001]),
    (16, 2, 64, 64, [2, 1] * 20, [38], [8001]),
    (16, 2, 128, 64, [1] * 40, [33], [6000]),           # a long cache among the own ones
])
def test_prefix_attention_of_long_prefixes(mp, hq, hk, d, page, q_lens, groups, prefixes):
    own = [m + (37 * i) % 400 for i, m in enumerate(q_lens)]
    own[1] += 5000 if groups == [33] else 0
    c = Shared(mp, "bf16", hq, hk, d, page, own, groups, prefixes)
    cu, cu_t = offsets(q_lens)
    q = c.randn(cu[-1], hq, d, by=1.5)
    first = None
    for _ in range(20):  # many at once, so that they load the memory
        out, lse = attend_prefix(mp, c, q, cu, cu_t, max(q_lens))
        first = first if first is not None else out
        assert torch.equal(out, first)
    check_prefix(c, "bf16", q, cu, out, lse)
    assert c.status.item() == 0


@pytest.mark.parametrize("hq,hk,d,page,q_lens,groups,prefixes", [
    (40, 40, 128, 0, [1] * 30, [], []),                       # a row per KV head, no prefix at all
    (8, 8, 64, 16, [1, 2, 3, 4, 1, 1], [4, 1], [333, 0]),     # up to four rows, both passes
    (8, 2, 64, 48, [1, 2, 1, 0, 2], [1, 1, 1], [5000, 17, 3]),  # up to eight
    (8, 2, 128, 16, [2, 1, 2, 1], [1, 0, 2], [2999, 5, 16]),
    (7, 1, 128, 32, [1, 2, 1], [2], [9000]),                  # up to sixteen
    (16, 1, 64, 0, [1, 1, 1], [1, 1], [31, 4097]),
    (5, 5, 128, 0, [1, 3, 7, 2], [1, 2], [64, 1500]),        # own slots by warps, a group's prefix in tiles
    (4, 1, 64, 64, [1, 1, 30], [2], [700]),                   # and the other way round
    (12, 1, 128, 256, [1] * 9, [9], [777]),
])
def test_prefix_attention_of_few_rows_in_fp32(mp, hq, hk, d, page, q_lens, groups, prefixes):
    own = [m + (173 * i) % 900 for i, m in enumerate(q_lens)]
    own[-1] = q_lens[-1]
    c = Shared(mp, "f32", hq, hk, d, page, own, groups or [0], prefixes or [0])
    cu, cu_t = offsets(q_lens)
    q = c.randn(cu[-1] + 2, hq, d, by=1.5)
    group_q = max(c.limits(cu)[0], 1)
    out, lse = attend_prefix(mp, c, q, cu, cu_t, max(q_lens), group_q=group_q)
    check_prefix(c, "f32", q, cu, out, lse)
    wide, z = attend_prefix(mp, c, q, cu, cu_t, max(q_lens), max_kv=c.ps * c.cols, group_q=group_q + 2, max_prefix=c.pre.ps * c.pre.cols)
    check_prefix(c, "f32", q, cu, wide, z)
    assert c.status.item() == 0
    again, _ = attend_prefix(mp, c, q, cu, cu_t, max(q_lens), group_q=group_q)
    assert torch.equal(again[:cu[-1]], out[:cu[-1]])


def test_prefix_attention_over_pages_of_another_size(mp):
    """The prefixes' cache is another one: short pages here, a dense one there."""
    for page, ppage in ((16, 128), (64, 0), (0, 48)):
        c = Shared(mp, "bf16", 8, 2, 128, page, [100, 7, 300], [2, 1], [500, 130], ppage=ppage)
        cu, cu_t = offsets([3, 1, 20])
        q = c.randn(24, 8, 128, by=1.5)
        out, lse = attend_prefix(mp, c, q, cu, cu_t, 20)
        check_prefix(c, "bf16", q, cu, out, lse)
        assert c.status.item() == 0


def test_prefix_attention_of_large_logits(mp):
    """The prefix holds nearly all of the softmax for some rows and nearly nothing for others."""
    for dtype in ("bf16", "f32"):
        for m in (1, 40):
            c = Shared(mp, dtype, 8, 2, 128, 64, [100, 70, 300], [2, 1], [700, 300])
            c.keys.mul_(6.0)
            c.pre.keys = c.keys
            cu, cu_t = offsets([m, 1, m])
            q = c.randn(cu[-1], 8, 128, by=8.0)
            out, lse = attend_prefix(mp, c, q, cu, cu_t, m)
            check_prefix(c, dtype, q, cu, out, lse)


def test_prefix_attention_is_the_chunk_attention_over_both(mp):
    """The same slots behind one page table per sequence: what mp_chunk_attention gives for them."""
    for m in (1, 3, 30):
        c = Shared(mp, "bf16", 8, 2, 128, 16, [40, 3 * m, 200], [3], [160])
        cu, cu_t = offsets([m, m, m])
        q = c.randn(cu[-1], 8, 128, by=1.5)
        out, lse = attend_prefix(mp, c, q, cu, cu_t, m)
        pages = 160 // 16
        table = torch.cat((c.pre.table[:1, :pages].expand(3, -1), c.table), 1).contiguous()
        cfg = mp.make_cache_config(batch=3, kv_heads=2, q_heads=8, head_dim=128, page_size=16, n_pages=c.pages, max_pages=table.shape[1])
        both, z = torch.empty_like(q), torch.empty_like(lse)
        ws = torch.empty(max(1, mp.mp_chunk_workspace_bytes(cfg, cu[-1], m, 360)), dtype=torch.uint8, device=DEV)
        mp.mp_chunk_attention(cfg, q, cu_t, c.kv_len + 160, m, 360, c.keys, c.values, table, both, z, ws)
        # each is within its tolerance of the exact result: compared with it, not with each other
        check_prefix(c, "bf16", q, cu, out, lse)
        check_prefix(c, "bf16", q, cu, both, z)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prefix_attention_of_more_groups_than_one_launch_takes(mp, dtype):
    groups = [(i * 3) % 4 for i in range(1100)]
    batch = sum(groups) + 2
    c = Shared(mp, dtype, 8, 1, 64, 16, [(7 * b) % 20 + 1 for b in range(batch)], groups, [(11 * g) % 50 for g in range(1100)])
    cu, cu_t = offsets([1] * batch)
    q = c.randn(batch, 8, 64)
    out, lse = attend_prefix(mp, c, q, cu, cu_t, 1, group_q=3)
    check_prefix(c, dtype, q, cu, out, lse)
    assert c.status.item() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prefix_attention_of_more_tiles_than_one_launch_takes(mp, dtype):
    """Chunks of 1350 sequences and 1000 groups on tiles: three launches, whose cut tiles are joined at once. Two
    long caches and a long prefix among short ones."""
    groups = [1 + g % 2 if g % 3 else 0 for g in range(1000)]
    batch = sum(groups) + 351
    q_lens = [(5 * b) % 7 for b in range(batch)]
    q_lens[1200] = 300
    own = [max(1, m) + (7 * b) % 20 for b, m in enumerate(q_lens)]
    own[3], own[1201] = 3000, 900
    prefixes = [(11 * g) % 50 for g in range(1000)]
    prefixes[700] = 2000
    c = Shared(mp, dtype, 8, 1, 64, 16, own, groups, prefixes)
    cu, cu_t = offsets(q_lens)
    q = c.randn(cu[-1], 8, 64)
    out, lse = attend_prefix(mp, c, q, cu, cu_t, 300)
    check_prefix(c, dtype, q, cu, out, lse)
    assert c.status.item() == 0


@pytest.mark.parametrize("seqs", [5, 20])
def test_prefix_attention_of_many_groups_in_slices(mp, seqs):
    """1030 groups, planned 1024 at a time and most of them without a sequence, next to own slots."""
    groups = [seqs if g % 103 == 1 or g == 1027 else 0 for g in range(1030)]
    batch = sum(groups) + 1
    c = Shared(mp, "bf16", 8, 1, 64, 16, [(7 * b) % 90 + 1 for b in range(batch)], groups, [(11 * g) % 300 for g in range(1030)], cap=100, pcap=4800)
    cu, cu_t = offsets([1] * batch)
    q = c.randn(batch, 8, 64)
    out, lse = attend_prefix(mp, c, q, cu, cu_t, 1, max_prefix=300 * 16)
    check_prefix(c, "bf16", q, cu, out, lse)
    assert c.status.item() == 0


def test_prefix_attention_over_offsets_past_32_bits(mp):
    ps, hk, d = 4096, 4, 128
    pages = 2 ** 31 // (ps * hk * d) * 2 + 4
    shape = dict(kv_heads=hk, q_heads=8, head_dim=d, page_size=ps, n_pages=pages, dtype="bf16")
    keys = torch.empty(pages, hk, ps, d, dtype=torch.bfloat16, device=DEV)
    values = torch.empty_like(keys)
    assert keys.numel() > 2 ** 32
    g = torch.Generator(device=DEV).manual_seed(3)
    for pool in (keys, values):
        pool[-3:] = torch.randn(3, hk, ps, d, generator=g, device=DEV).to(torch.bfloat16)

    class C:
        pass
    c, c.pre = C(), C()
    c.cfg, c.pre.cfg = (mp.make_cache_config(batch=1, max_pages=n, **shape) for n in (1, 2))
    c.kv, c.prefixes, c.groups, c.hk, c.d = [300], [5000], [1], hk, d
    c.keys, c.values, c.pre.keys, c.pre.values = keys, values, keys, values
    c.table, c.pre.table = ints([[pages - 3]]), ints([[pages - 1, pages - 2]])
    c.kv_len, c.pre.kv_len, c.cu_group, c.status = ints([300]), ints([5000]), ints([0, 1]), ints([0])
    c.limits = lambda cu: (cu[-1], 5000)
    for m in (1, 150):
        cu, cu_t = offsets([m])
        q = torch.randn(m, 8, d, generator=g, device=DEV).to(torch.bfloat16)
        out, lse = attend_prefix(mp, c, q, cu, cu_t, m)
        check_prefix(c, "bf16", q, cu, out, lse)


def test_prefix_attention_with_bad_lengths_groups_and_pages(mp):
    c = Shared(mp, "bf16", 8, 2, 128, 32, [100, 60, 90, 20], [2, 1], [200, 150])
    cu, cu_t = offsets([1, 30, 1, 5])
    q = c.randn(37, 8, 128)
    want, _ = attend_prefix(mp, c, q, cu, cu_t, 30)
    keep = c.pre.table.clone()
    c.pre.table[1, 1], c.pre.table[1, 2] = c.pages + 5, -1
    c.keys[0], c.values[0] = c.keys[0].nan_to_num(0.0), c.values[0].nan_to_num(0.0)  # what is read in their place
    out, _ = attend_prefix(mp, c, q, cu, cu_t, 30)
    assert c.status.item() == mp.MP_STATUS_BAD_PAGE
    assert torch.equal(out[:31], want[:31]) and torch.equal(out[32:], want[32:])
    c.pre.table.copy_(keep)
    for change in (lambda: c.cu_group.copy_(ints([0, 2, 10 ** 9])), lambda: c.cu_group.copy_(ints([-5, 2, 3])), lambda: c.pre.kv_len.copy_(ints([10 ** 9, -1]))):
        c.status.zero_()
        change()
        attend_prefix(mp, c, q, cu, cu_t, 30)
        assert c.status.item() == mp.MP_STATUS_BAD_LENGTH
        c.cu_group.copy_(ints([0, 2, 3]))
        c.pre.kv_len.copy_(ints([200, 150]))
    # rows of a group behind the limit do not see the prefix, the others do
    c.status.zero_()
    out, lse = attend_prefix(mp, c, q, cu, cu_t, 30, group_q=20)
    assert c.status.item() == mp.MP_STATUS_BAD_LENGTH
    c.groups, c.prefixes = [0], [0]
    alone = S.prefix_attention(q, cu, c.kv, c.keys, c.values, c.table, [0], [0], None, None, None, 2)
    assert ((lse[20:31].double() - alone[1][20:31]).abs() <= 2.0 ** -12).all()
    assert ((out[20:31].double() - alone[0][20:31]).abs() <= 2.0 ** -5 * alone[2][20:31]).all()
    err = (out[31:].double() - want[31:].double()).abs()
    assert (err <= 2.0 ** -6 * want[31:].abs() + 2.0 ** -6).all()


def test_prefix_attention_captured_and_on_two_streams(mp):
    """Captured calls follow lengths and groups; two graphs with a workspace each at once."""
    for m in (1, 33):
        c = Shared(mp, "bf16", 8, 2, 128, 64, [300, 170, 90], [2, 1], [1500, 900])
        cu, cu_t = offsets([m] * 3)
        graphs, streams = [], [torch.cuda.Stream() for _ in range(2)]
        for st in streams:
            q = c.randn(3 * m, 8, 128)
            out, lse = torch.empty_like(q), torch.empty(3 * m, 8, device=DEV)
            ws = torch.empty(mp.mp_prefix_workspace_bytes(c.cfg, c.pre.cfg, 3 * m, m, 300, 3 * m, 1500), dtype=torch.uint8, device=DEV)
            call = lambda: mp.mp_prefix_attention(c.cfg, c.pre.cfg, q, cu_t, c.kv_len, m, 300, c.keys, c.values, c.table, c.cu_group, c.pre.kv_len,
                                                  3 * m, 1500, c.pre.keys, c.pre.values, c.pre.table, out, lse, ws, c.status)
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=st):
                call()
            graphs.append((g, q, out, lse, ws))
        for kv, groups, prefixes in (([300, 170, 90], [2, 1], [1500, 900]), ([m, m, m], [1, 2], [64, 65]), ([120, 44, 90], [3, 0], [0, 5]), ([120, 44, 90], [0, 3], [7, 700])):
            c.kv, c.groups, c.prefixes = kv, groups, prefixes
            c.kv_len.copy_(ints(kv))
            c.cu_group.copy_(offsets(groups)[1])
            c.pre.kv_len.copy_(ints(prefixes))
            torch.cuda.synchronize()
            for _ in range(3):
                for (g, *_), st in zip(graphs, streams):
                    with torch.cuda.stream(st):
                        g.replay()
            torch.cuda.synchronize()
            assert c.status.item() == 0
            for _, q, out, lse, _ in graphs:
                check_prefix(c, "bf16", q, cu, out, lse)


def test_prefix_queries_of_another_shape_are_refused(mp):
    c = Shared(mp, "bf16", 8, 2, 128, 64, [30, 17], [2], [150])
    cu, cu_t = offsets([1, 1])
    q, ws = c.randn(2, 8, 128), torch.empty(1 << 24, dtype=torch.uint8, device=DEV)
    call = lambda q, out: mp.mp_prefix_attention(c.cfg, c.pre.cfg, q, cu_t, c.kv_len, 1, 30, c.keys, c.values, c.table, c.cu_group, c.pre.kv_len, 2, 150,
                                                 c.pre.keys, c.pre.values, c.pre.table, out, None, ws)
    call(q, torch.empty_like(q))
    for bad_q, bad_out in ((q[None], torch.empty_like(q)), (q, torch.empty(3, 8, 128, dtype=torch.bfloat16, device=DEV)), (q.float(), q.clone()),
                           (q.transpose(1, 2), q.clone())):
        with pytest.raises(ValueError):
            call(bad_q, bad_out)


# ----------------------------------------------------------------------------------
# rotation
# ----------------------------------------------------------------------------------

def freq(rot, theta=500000.0):
    return theta ** (-2.0 * torch.arange(rot // 2, device=DEV, dtype=torch.float64) / max(1, rot))


def check_rotate(c, dtype, before, after, kv, start, at, f0, f1, rot, inter, scale):
    """Every slot of the pool after the call: turned, or the bits that were there."""
    eps = 2.0 ** -18 if dtype == "bf16" else 2.0 ** -20
    want, tol = before.double(), torch.zeros_like(before, dtype=torch.float64)
    turned = torch.zeros(before.shape[:3], dtype=torch.bool, device=DEV)
    for b, n in enumerate(kv):
        slot = torch.arange(n, device=DEV)
        for h in range(c.hk):
            pick = lambda p: slot if p is None else p[b, h if p.shape[1] > 1 else 0, :n]
            y, size = S.turned(R.gather(before, c.table, b, h, n), pick(at), pick(start), f0 if f1 is None else f1, f0, rot, inter, scale)
            t = HALF[dtype] * y.abs() + (1 + HALF[dtype]) * eps * size + 2.0 ** -126
            for i, p in enumerate(R.pages_of(c.table, b, n, c.ps)):
                e = min(c.ps, n - i * c.ps)
                want[p, h, :e], tol[p, h, :e] = y[i * c.ps:i * c.ps + e], t[i * c.ps:i * c.ps + e]
                turned[p, h, :e] = True
    bits = lambda x: x.view(torch.int16 if dtype == "bf16" else torch.int32)
    assert torch.equal(bits(after)[~turned], bits(before)[~turned])            # what lies behind the lengths
    assert torch.equal(bits(after)[..., rot:], bits(before)[..., rot:])        # elements that do not turn
    err = (after.double() - want).abs()[turned]
    assert (err <= tol[turned]).all(), (err - tol[turned]).max().item()


ROTATE = [
    # dtype, kv heads, d, page, lengths, rot, interleaved
    ("bf16", 2, 128, 0, [1, 300], 128, False),
    ("bf16", 8, 128, 64, [1000, 64, 0, 7], 128, True),
    ("bf16", 3, 64, 16, [77, 500, 16], 64, False),
    ("bf16", 1, 64, 48, [1, 333], 32, False),
    ("bf16", 5, 128, 16, [100], 16, False),
    ("bf16", 9, 128, 96, [200, 95], 96, False),      # six lanes of eight
    ("bf16", 2, 128, 32, [65], 20, True),            # a lane that turns a part of its pairs
    ("bf16", 4, 64, 0, [129, 12], 2, True),
    ("f32", 2, 128, 0, [1, 300], 128, False),
    ("f32", 4, 64, 16, [100, 0, 33], 64, True),
    ("f32", 3, 128, 48, [333], 24, False),
    ("f32", 7, 64, 0, [50, 9], 6, True),
]


@pytest.mark.parametrize("dtype,hk,d,page,kv,rot,inter", ROTATE)
@pytest.mark.parametrize("kind", ["slots", "one", "heads", "scaled"])
def test_rotate(mp, dtype, hk, d, page, kv, rot, inter, kind):
    c = Cache(mp, dtype, hk, hk, d, page, kv, seed=rot)
    cols, batch = c.ps * c.cols + 3, len(kv)
    at = lambda heads, top: torch.randint(0, top, (batch, heads, cols), generator=c.gen).to(torch.int32).to(DEV)
    f0, f1, start, to, scale = freq(rot), None, None, None, 1.0
    if kind == "slots":
        start = at(1, 2 ** 20)                        # to the slot's own place
    elif kind == "one":
        to, f1 = at(1, 2 ** 20) - 2 ** 19, freq(rot, 1e6)
    elif kind == "heads":
        start, to, scale = at(hk, 2 ** 20), at(hk, 5000), -0.75
    else:
        f1, scale = f0 / 8, 1.25
    before = c.keys.clone()
    rotary = mp.make_rotary(rot_dim=rot, interleaved=inter)
    mp.mp_cache_rotate(c.cfg, rotary, c.keys, c.table, c.kv_len, max(1, max(kv)), f0, f1, start, to, scale, c.status)
    check_rotate(c, dtype, before, c.keys, kv, start, to, f0, f1, rot, inter, scale)
    assert c.status.item() == 0


def test_rotate_many_slots(mp):
    """More slots than one pass of the CTAs takes, of one position for all heads and of one for each."""
    for heads in (1, 2):
        c = Cache(mp, "bf16", 2, 2, 64, 16, [70000, 1, 30001])
        c.keys = torch.randn(c.keys.shape, device=DEV).to(torch.bfloat16)
        start = torch.randint(0, 2 ** 18, (3, heads, 70000), dtype=torch.int32, device=DEV)
        before = c.keys.clone()
        mp.mp_cache_rotate(c.cfg, mp.make_rotary(rot_dim=64), c.keys, c.table, c.kv_len, 70000, freq(64), None, start, None, 1.0, c.status)
        check_rotate(c, "bf16", before, c.keys, c.kv, start, None, freq(64), None, 64, False, 1.0)


def test_rotate_gives_what_the_append_gives_at_the_new_place(mp):
    """A key appended at one position and turned to another is the key appended there, but for its rounding at
    the first: h |y| of the pair once more."""
    for dtype, inter in (("f32", False), ("bf16", True), ("bf16", False)):
        n, hk, d = 40, 2, 128
        c, t = (Cache(mp, dtype, hk, hk, d, 16, [n]) for _ in range(2))
        q = torch.randn(n, hk, d, device=DEV).to(DT[dtype])
        cu, cu_t = offsets([n])
        here, there = (torch.randint(0, 100000, (1, 1, n), dtype=torch.int32, device=DEV) for _ in range(2))
        rotary, f = mp.make_rotary(rot_dim=d, interleaved=inter), freq(d)
        for x, p in ((c, here), (t, there)):
            mp.mp_cache_append(x.cfg, rotary, q, q, q, None, None, f, p.flatten(), cu_t, x.kv_len, x.keys, x.values, x.table, torch.empty_like(q), x.status)
        mp.mp_cache_rotate(c.cfg, rotary, c.keys, c.table, c.kv_len, n, f, None, here, there, 1.0, c.status)
        i = torch.arange(d // 2, device=DEV)
        a, b = (2 * i, 2 * i + 1) if inter else (i, i + d // 2)
        for h in range(hk):
            got, want = R.gather(c.keys, c.table, 0, h, n), R.gather(t.keys, t.table, 0, h, n)
            size = torch.zeros_like(want)
            size[:, a] = size[:, b] = torch.hypot(want[:, a], want[:, b])
            # first rounding (of both elements, so sqrt(2) of the size), last rounding, the other side's
            assert ((got - want).abs() <= (1.5 + 1.05 + 1.05) * HALF[dtype] * size + 2.0 ** -17 * size).all()


def test_rotate_leaves_bad_pages_and_cut_lengths(mp):
    c = Cache(mp, "bf16", 2, 2, 128, 32, [200, 100])
    before = c.keys.clone()
    keep = c.table.clone()
    c.table[0, 2], c.table[0, 3] = -1, c.pages
    f = freq(128)
    start = torch.full((2, 1, 300), 9, dtype=torch.int32, device=DEV)
    mp.mp_cache_rotate(c.cfg, mp.make_rotary(rot_dim=128), c.keys, c.table, c.kv_len, 200, f, None, start, None, 1.0, c.status)
    assert c.status.item() == mp.MP_STATUS_BAD_PAGE
    changed = (c.keys != before).flatten(1).any(1) & ~c.keys.isnan().flatten(1).all(1)
    named = set(keep[0, [0, 1, 4, 5, 6]].tolist() + keep[1, :4].tolist())
    assert all(not changed[p] for p in range(c.pages) if p not in named)
    # a length behind the limit is cut to it
    c.table.copy_(keep)
    c.status.zero_()
    before = c.keys.clone()
    mp.mp_cache_rotate(c.cfg, mp.make_rotary(rot_dim=128), c.keys, c.table, c.kv_len, 150, f, None, start, None, 1.0, c.status)
    assert c.status.item() == mp.MP_STATUS_BAD_LENGTH
    check_rotate(c, "bf16", before, c.keys, [150, 100], start, None, f, None, 128, False, 1.0)


def test_rotate_over_offsets_past_32_bits(mp):
    ps, hk, d, n = 4096, 4, 128, 5000
    pages = 2 ** 31 // (ps * hk * d) * 2 + 3
    cfg = mp.make_cache_config(batch=1, kv_heads=hk, q_heads=hk, head_dim=d, page_size=ps, n_pages=pages, max_pages=2, dtype="bf16")
    keys = torch.zeros(pages, hk, ps, d, dtype=torch.bfloat16, device=DEV)
    assert keys.numel() > 2 ** 32
    keys[-2:] = torch.randn(2, hk, ps, d, device=DEV).to(torch.bfloat16)
    before = keys[-2:].clone()
    for heads in (1, hk):
        start = torch.randint(0, 10 ** 6, (1, heads, n), dtype=torch.int32, device=DEV)
        mp.mp_cache_rotate(cfg, mp.make_rotary(rot_dim=d), keys, ints([[pages - 1, pages - 2]]), ints([n]), n, freq(d), None, start, None)

        class C:
            pass
        c = C()
        c.hk, c.ps, c.table = hk, ps, ints([[1, 0]])
        check_rotate(c, "bf16", before, keys[-2:], [n], start, None, freq(d), None, d, False, 1.0)
        before = keys[-2:].clone()
    assert not keys[:-2].any()


def test_rotate_keeps_infinities_in_their_pairs(mp):
    c = Cache(mp, "bf16", 1, 1, 64, 0, [3])
    c.keys[0, 0, 1, 5], c.keys[0, 0, 1, 40] = math.inf, math.nan
    start = torch.full((1, 1, 3), 7, dtype=torch.int32, device=DEV)
    for inter, rot, hit in ((False, 32, {5, 21}), (True, 64, {4, 5, 40, 41})):
        k = c.keys.clone()
        mp.mp_cache_rotate(c.cfg, mp.make_rotary(rot_dim=rot, interleaved=inter), k, None, c.kv_len, 3, freq(rot), None, start, None)
        odd = {i for i in range(64) if not math.isfinite(k[0, 0, 1, i].item())}
        assert hit <= odd <= hit | {40} and torch.isfinite(k[0, 0, [0, 2]]).all()


def test_rotate_leaves_the_bits_of_what_does_not_turn(mp):
    """NaN of any bits behind rot_dim, interleaved pairs that end inside a lane's vectors among them."""
    for dtype, word, bits in (("bf16", torch.int16, -3), ("f32", torch.int32, -5)):
        for rot in (2, 6, 8, 14, 18, 32, 54, 64):
            c = Cache(mp, dtype, 2, 2, 64, 16, [20, 3])
            c.keys[:] = torch.randn(c.keys.shape, device=DEV).to(DT[dtype])
            c.keys.view(word)[..., rot:] = bits
            start = torch.full((2, 1, 20), 11, dtype=torch.int32, device=DEV)
            before = c.keys.clone()
            mp.mp_cache_rotate(c.cfg, mp.make_rotary(rot_dim=rot, interleaved=True), c.keys, c.table, c.kv_len, 20, freq(rot), None, start, None, 1.0, c.status)
            assert (c.keys.view(word)[..., rot:] == bits).all() and torch.isfinite(c.keys[..., :rot]).all()
            assert not torch.equal(c.keys.view(word), before.view(word))


def test_rotate_captured_follows_lengths_and_positions(mp):
    c = Cache(mp, "bf16", 2, 2, 128, 64, [500, 90])
    start = torch.zeros(2, 2, 500, dtype=torch.int32, device=DEV)
    f, rotary = freq(128), mp.make_rotary(rot_dim=128)
    st, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=st):
        mp.mp_cache_rotate(c.cfg, rotary, c.keys, c.table, c.kv_len, 500, f, None, start, None, 1.0, c.status)
    for kv in ([500, 90], [1, 0], [64, 65]):
        start.copy_(torch.randint(0, 9000, start.shape, dtype=torch.int32))
        c.kv_len.copy_(ints(kv))
        before = c.keys.clone()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        check_rotate(c, "bf16", before, c.keys, kv, start, None, f, None, 128, False, 1.0)


# ----------------------------------------------------------------------------------
# all of them, as a serving loop calls them
# ----------------------------------------------------------------------------------

def test_a_serving_loop_plans_shares_cuts_and_moves(mp):
    """Two groups of sequences behind a shared prefix each: their steps are planned (prompts, single tokens, a rejected
    draft, an end), appended behind the prefix's positions and attended; then the longest caches are cut, their keys
    moved up to their new places, and the sequences go on over the destination."""
    hq, hk, d, page, cap = 8, 2, 128, 16, 160
    g = torch.Generator().manual_seed(9)
    prefixes, groups = [200, 75], [2, 2]
    pre = Cache(mp, "f32", hq, hk, d, page, prefixes, seed=4)
    batch, cols = 5, cap // page
    pages = batch * cols - 8
    cfg = mp.make_cache_config(batch=batch, kv_heads=hk, q_heads=hq, head_dim=d, page_size=page, n_pages=pages, max_pages=cols, dtype="f32")
    keys, values = (torch.full((pages, hk, page, d), math.nan, device=DEV) for _ in range(2))
    table = torch.full((batch, cols), -1, dtype=torch.int32, device=DEV)
    free, n_free, kv_len, status = ints(list(range(pages))), ints([pages]), ints([0] * batch), ints([0])
    base, cu_group = ints([200, 200, 75, 75, 0]), ints([0, 2, 4])
    cu_q, positions = ints([0] * (batch + 1)), ints([0] * 400)
    scores = torch.zeros(batch, hk, cap, device=DEV)
    f, rotary = freq(d), mp.make_rotary(rot_dim=d)
    ws = torch.empty(mp.mp_prefix_workspace_bytes(cfg, pre.cfg, 400, 100, cap, 200, 200), dtype=torch.uint8, device=DEV)
    lengths = [0] * batch

    def step(change, cfg, keys, values, table, free, n_free, kv_len, scores, cap):
        nonlocal lengths
        lengths = [max(0, n + x) for n, x in zip(lengths, change)]
        m = [max(0, x) for x in change]
        mp.mp_cache_plan(cfg, ints(change), base, kv_len, n_free, 400, table, free, kv_len, n_free, cu_q, positions, None, None, status)
        rows = sum(m)
        cu, _ = offsets(m)
        assert cu_q.tolist() == cu and kv_len.tolist() == lengths
        if not rows:
            return
        x, k, v = (torch.randn(rows, h, d, generator=g).to(DEV) for h in (hq, hk, hk))
        q = torch.empty_like(x)
        mp.mp_cache_append(cfg, rotary, x, k, v, None, None, f, positions[:rows].contiguous(), cu_q, kv_len, keys, values, table, q, status)
        out, lse = torch.full_like(q, 77.0), torch.full((rows, hq), 77.0, device=DEV)
        mp.mp_prefix_attention(cfg, pre.cfg, q, cu_q, kv_len, max(m), cap, keys, values, table, cu_group, pre.kv_len, max(1, sum(m[:2]), sum(m[2:4])),
                               200, pre.keys, pre.values, pre.table, out, lse, ws, status)

        class C:
            pass
        c = C()
        c.kv, c.keys, c.values, c.table, c.groups, c.prefixes, c.pre, c.hk, c.d = lengths, keys, values, table, groups, prefixes, pre, hk, d
        check_prefix(c, "f32", q, cu, out, lse)
        mp.mp_cache_weights(cfg, q, lse, cu_q, kv_len, max(m), cap, keys, table, scores, status)

    args = (cfg, keys, values, table, free, n_free, kv_len, scores, cap)
    for change in ([30, 100, 17, 1, 60], [1, 1, 1, 1, 1], [4, 4, 0, 4, 4], [-3, -4, 0, -1, 0], [1, 1, 1, 1, -65], [1, 40, 70, 1, 8]):
        step(change, *args)
    assert status.item() == 0 and sum(-(-n // page) for n in lengths) + n_free.item() == pages
    # cut to 48 slots a sequence, into a dense cache of 64
    budget, old = 48, list(lengths)
    dense = mp.make_cache_config(batch=batch, kv_heads=hk, q_heads=hq, head_dim=d, page_size=64, n_pages=batch, dtype="f32")
    dk, dv = (torch.full((batch, hk, 64, d), math.nan, device=DEV) for _ in range(2))
    ds, kept = torch.zeros(batch, hk, 64, device=DEV), torch.zeros(batch, hk, budget, dtype=torch.int32, device=DEV)
    ews = torch.empty(mp.mp_evict_workspace_bytes(cfg, cap, budget), dtype=torch.uint8, device=DEV)
    mp.mp_cache_evict(cfg, dense, keys, values, table, kv_len, cap, scores, 4, 16, budget, dk, dv, None, ds, kv_len, kept, ews, status)
    lengths = [min(n, budget) for n in lengths]
    # a kept key stands where its slot says, behind the same prefix: its text position was base + old slot and becomes base + new slot
    before = dk.clone()
    mp.mp_cache_rotate(dense, rotary, dk, None, kv_len, budget, f, None, kept, None, 1.0, status)

    class D:
        pass
    c = D()
    c.hk, c.ps, c.table = hk, 64, None
    check_rotate(c, "f32", before, dk, lengths, kept, None, f, None, d, False, 1.0)
    for change in ([1, 1, 1, 1, 1], [5, -2, 1, 3, 1]):
        step(change, dense, dk, dv, None, None, None, kv_len, ds, 64)
    assert status.item() == 0 and kv_len.tolist() == lengths


FIRST = '''
import sys
import torch
sys.path.insert(0, {root!r})
import lsh_sampled_sparse_centered_gb300 as mp
dev, d, hk, hq, n, prefix, m = "cuda:0", {d}, 2, 8, 700, {prefix}, {m}
dt = {{"bf16": torch.bfloat16, "f32": torch.float32}}[{dtype!r}]
g = torch.Generator(device=dev).manual_seed(1)
rnd = lambda *s: torch.randn(*s, generator=g, device=dev).to(dt)
ints = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
cfg = mp.make_cache_config(batch=2, kv_heads=hk, q_heads=hq, head_dim=d, page_size=16, n_pages=96, max_pages=44, dtype={dtype!r})
pre = mp.make_cache_config(batch=1, kv_heads=hk, q_heads=hq, head_dim=d, page_size=prefix, n_pages=1, dtype={dtype!r})
keys, values, pk, pv = rnd(96, hk, 16, d), rnd(96, hk, 16, d), rnd(1, hk, prefix, d), rnd(1, hk, prefix, d)
table, free = ints([list(range(44)), list(range(44, 88))]), ints(list(range(88, 96)) + [0] * 88)
q, out, lse = rnd(2 * m, hq, d), torch.empty(2 * m, hq, d, dtype=dt, device=dev), torch.empty(2 * m, hq, device=dev)
kv, change, n_free, new_len, new_free, cu, group, pl = ints([640, 600]), ints([m, m]), ints([8]), ints([0, 0]), ints([0]), ints([0, 0, 0]), ints([0, 2]), ints([prefix])
f, at = torch.ones(d // 2, dtype=torch.float64, device=dev), ints([[[i + 1 for i in range(700)]]] * 2)
ws = torch.empty(mp.mp_prefix_workspace_bytes(cfg, pre, 2 * m, m, 700, 2 * m, prefix), dtype=torch.uint8, device=dev)
status = ints([0])
first = keys.clone()
def step():
    mp.mp_cache_plan(cfg, change, None, kv, n_free, 2 * m, table, free, new_len, new_free, cu, None, None, None, status)
    mp.mp_prefix_attention(cfg, pre, q, cu, new_len, m, 700, keys, values, table, group, pl, 2 * m, prefix, pk, pv, None, out, lse, ws, status)
    mp.mp_cache_rotate(cfg, mp.make_rotary(rot_dim=d), keys, table, new_len, 700, f, None, at, None, 1.0, status)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    step()
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in (out, lse, new_len, new_free, cu, keys)]
keys.copy_(first)
step()
torch.cuda.synchronize()
assert status.item() == 0 and new_len.tolist() == [640 + m, 600 + m]
assert all(torch.equal(a, b) for a, b in zip(got, (out, lse, new_len, new_free, cu, keys)))
print("same")
'''


@pytest.mark.parametrize("dtype,d,m,prefix", [("bf16", 128, 1, 500), ("bf16", 64, 12, 40000), ("bf16", 128, 12, 40000), ("bf16", 128, 40, 1000),
                                              ("f32", 64, 1, 700), ("f32", 128, 30, 300)])
def test_a_first_call_may_be_captured(dtype, d, m, prefix):
    """Kernels are loaded and their shared memory set under the capture; equal bits afterwards."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST.format(root=root, dtype=dtype, d=d, m=m, prefix=prefix)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("same"), (r.stdout[-500:], r.stderr[-2000:])
