"""Calls at the edges of what the cache operators allow, on the GPU: lengths that pass a limit,
infinities, buffers used in place, few-row attention of 9 to 16 rows, workspaces sized once.

Tolerances are those of test_gpu_cache.py, with h = half a step of a type relative to the
value (fp32 2^-24, bf16 2^-8). Few rows (at most 16 per KV head) take their weights as two bf16
terms: the second is off by 2^-8 of itself, and it is at most 2^-8 of the weight, so that a weight
is off by 2^-16 where other chunks have 2^-8.
"""
import math
import os
import shutil
import subprocess
import threading
import time

import pytest
import torch

import cache_reference as R
from test_gpu_cache import DEV, HALF, Cache, attend, check_attention, make_scores, offsets, pool_rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mp():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import lsh_sampled_sparse_centered_gb300 as m
    return m


# ---- append: infinities stay in their own elements ----

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rot,inter", [(0, False), (32, False), (16, True), (0, True)])
def test_append_keeps_infinities_out_of_other_elements(mp, dtype, rot, inter):
    """Without a norm an element that is not rotated goes through unchanged, whatever it or the
    element next to it holds; with one, x / sqrt(inf) is 0 for every finite x."""
    hq, hk, d = 3, 1, 64
    c = Cache(mp, dtype, hq, hk, d, 16, [5], fill="none")
    _, cu_t = offsets([5])
    q, k, v = c.randn(5, hq, d), c.randn(5, hk, d), c.randn(5, hk, d)
    q[1, 0, 40], q[2, 2, 63], q[3, 1, 50] = math.inf, -math.inf, math.nan
    k[4, 0, 41] = math.inf
    inv = torch.ones(max(1, rot // 2), dtype=torch.float64, device=DEV)
    q_out = torch.empty_like(q)
    mp.mp_cache_append(c.cfg, mp.make_rotary(rot_dim=rot, interleaved=inter), q, k, v, None, None, inv, None, cu_t, c.kv_len, c.keys,
                       c.values, c.table, q_out, c.status)
    same = lambda a, b: torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(5.0, math.inf, -math.inf), b.nan_to_num(5.0, math.inf, -math.inf))
    page = int(c.table[0, 0])
    assert same(q_out[..., rot:], q[..., rot:])
    assert same(c.keys[page, 0, :5, rot:], k[:, 0, rot:])
    assert torch.isfinite(q_out[..., :rot]).all()
    w = c.randn(d)
    mp.mp_cache_append(c.cfg, mp.make_rotary(rot_dim=rot, interleaved=inter), q, k, v, w, w, inv, None, cu_t, c.kv_len, c.keys, c.values,
                       c.table, q_out, c.status)
    for r, h, e in ((1, 0, 40), (2, 2, 63)):
        want = torch.zeros(d, device=DEV, dtype=c.dtype)
        want[e] = math.nan
        assert same(q_out[r, h], want), q_out[r, h]
    assert c.status.item() == 0


# ---- lengths that pass a limit: every token stays in its own slot ----

CUT = [
    # dtype, q heads, kv heads, d, page, slots filled, kv_len, cu_q's end, rows of q, max_q, max_kv
    ("bf16", 4, 2, 64, 16, 48, 51, 6, 6, 6, 48),        # three tokens behind the table's last slot
    ("bf16", 4, 1, 128, 16, 48, 50, 4, 4, 4, 48),       # (at most 16 rows per KV head)
    ("bf16", 8, 2, 128, 16, 400, 390, 40, 40, 40, 300),  # a limit that no token's own slot is below
    ("bf16", 8, 2, 64, 16, 400, 390, 200, 200, 200, 300),  # and one that falls inside the chunk
    ("bf16", 8, 2, 128, 16, 400, 390, 40, 40, 30, 400),  # more tokens than max_q
    ("bf16", 4, 2, 128, 16, 400, 390, 50, 42, 50, 400),  # more tokens than rows
    ("bf16", 4, 2, 64, 16, 400, 390, 8, 8, 5, 400),
    ("bf16", 4, 2, 64, 16, 300, 20, 60, 60, 50, 300),    # chunk longer than the cache, and cut: the first 40 slots are negative
    ("bf16", 4, 2, 64, 16, 300, 2 ** 31 - 1, 60, 60, 60, 300),
    ("f32", 4, 2, 64, 16, 48, 51, 6, 6, 6, 48),
    ("f32", 8, 2, 128, 16, 400, 390, 200, 200, 150, 300),
    ("f32", 4, 2, 64, 16, 300, 20, 60, 60, 50, 300),
]


@pytest.mark.parametrize("dtype,hq,hk,d,page,fill,kv,end,rows,max_q,max_kv", CUT)
def test_cut_lengths_leave_tokens_in_their_slots(mp, dtype, hq, hk, d, page, fill, kv, end, rows, max_q, max_kv):
    c = Cache(mp, dtype, hq, hk, d, page, [fill])
    c.kv_len.fill_(kv)
    cu_t = torch.tensor([0, end], dtype=torch.int32, device=DEV)
    q = c.randn(rows, hq, d, by=1.5)
    live = min(rows, end, max_q)  # rows that the call takes
    out, lse = attend(mp, c, q, cu_t, max_q, max_kv=max_kv)
    assert c.status.item() == mp.MP_STATUS_BAD_LENGTH
    n = min(kv, max_kv, c.ps * c.cols)
    x = torch.full((live, hq, n), -math.inf, dtype=torch.float64, device=DEV)
    ab, p_v, p_av = torch.zeros_like(x), torch.zeros(live, hq, d, dtype=torch.float64, device=DEV), None
    p_av = torch.zeros_like(p_v)
    seen = torch.arange(n, device=DEV)[None] <= (kv - end + torch.arange(live, device=DEV))[:, None]
    for j in range(hq):
        k = R.gather(c.keys, c.table, 0, j // (hq // hk), n)
        x[:, j] = (q[:live, j].double() @ k.T / math.sqrt(d)).masked_fill(~seen, -math.inf)
        ab[:, j] = (q[:live, j].double().abs() @ k.abs().T / math.sqrt(d)).masked_fill(~seen, 0)
    z = torch.logsumexp(x, -1)
    p = torch.where(seen[:, None], torch.exp(x - z[..., None]), torch.zeros_like(x))
    p = torch.where(torch.isinf(z)[..., None], torch.zeros_like(p), p)
    for j in range(hq):
        v = R.gather(c.values, c.table, 0, j // (hq // hk), n)
        p_v[:, j], p_av[:, j] = p[:, j] @ v, p[:, j] @ v.abs()
    eps_x = (d + 8) * 2.0 ** -24 * ab.amax(-1)
    rel = 2 * eps_x + n * 2.0 ** -24 + 2.0 ** -20 + (2.0 ** -8 if dtype == "bf16" else 0.0)
    tol = HALF[dtype] * p_v.abs() + (1 + HALF[dtype]) * rel[..., None] * p_av
    assert ((out[:live].double() - p_v).abs() <= tol).all()
    empty = torch.isinf(z)
    assert torch.equal(torch.isinf(lse[:live]), empty)
    ztol = eps_x + (n + 8) * 2.0 ** -24 + 2.0 ** -21 * (1 + z.abs())
    assert ((lse[:live].double() - z).abs()[~empty] <= ztol[~empty]).all()
    assert (out[live:] == 77.0).all() and (lse[live:] == 77.0).all()  # rows that the limits leave out
    # the weights see the same slots
    c.status.zero_()
    given = torch.full((rows, hq), math.nan, device=DEV)
    given[:live] = z.float()
    sc0 = torch.rand(1, hk, c.ps * c.cols, generator=c.gen).to(DEV) * 0.01
    sc = sc0.clone()
    mp.mp_cache_weights(c.cfg, q, given, cu_t, c.kv_len, max_q, max_kv, c.keys, c.table, sc, c.status)
    assert c.status.item() == mp.MP_STATUS_BAD_LENGTH
    zz = torch.where(empty, torch.zeros_like(z), given[:live].double())
    w = torch.where(seen[:, None] & ~empty[..., None], torch.exp(x - zz[..., None]), torch.zeros_like(x))
    want = sc0.double()
    want[0, :, :n] += w.unflatten(1, (hk, hq // hk)).sum((0, 2))
    top = zz.abs().max()
    rel = (d + 8) * 2.0 ** -24 * ab.amax() + 2.0 ** -21 * (1 + top) + (hq // hk * live + 2) * 2.0 ** -24
    assert ((sc.double() - want).abs() <= rel * want).all()


def test_append_and_attention_agree_where_a_cut_token_stands(mp):
    """A token that the append has put into the last slots attends to its own key there."""
    c = Cache(mp, "f32", 2, 1, 64, 16, [48])
    c.keys.zero_()
    c.values.zero_()
    c.kv_len.fill_(51)  # three more than the table has room for: the tokens stand in slots 45 to 50
    _, cu_t = offsets([6])
    q, k, v = c.randn(6, 2, 64), c.randn(6, 1, 64), c.randn(6, 1, 64)
    q_out = torch.empty_like(q)
    mp.mp_cache_append(c.cfg, mp.make_rotary(rot_dim=0), q, k, v, None, None, None, None, cu_t, c.kv_len, c.keys, c.values, c.table, q_out,
                       c.status)
    out, _ = attend(mp, c, 40.0 * k.expand(6, 2, 64).contiguous(), cu_t, 6)  # queries that see little but their own key
    assert (out[:3].double() - v[:3].double()).abs().max() <= 2.0 ** -20 * v.abs().max()


def test_append_of_more_rows_than_the_call_has(mp):
    """cu_q that ends behind the packed tensors: the rows that are there go where they belong."""
    c = Cache(mp, "bf16", 2, 1, 64, 16, [48], fill="none")
    c.keys.fill_(5.0)
    c.values.fill_(5.0)
    cu_t = torch.tensor([0, 9], dtype=torch.int32, device=DEV)
    q, k, v = c.randn(6, 2, 64), c.randn(6, 1, 64), c.randn(6, 1, 64)
    q_out = torch.empty_like(q)
    mp.mp_cache_append(c.cfg, mp.make_rotary(rot_dim=0), q, k, v, None, None, None, None, cu_t, c.kv_len, c.keys, c.values, c.table, q_out,
                       c.status)
    assert c.status.item() == mp.MP_STATUS_BAD_LENGTH
    assert torch.equal(pool_rows(c.keys, c, 0, 0, 48)[39:45], k[:, 0]) and torch.equal(pool_rows(c.values, c, 0, 0, 48)[39:45], v[:, 0])
    assert (pool_rows(c.keys, c, 0, 0, 48)[:39] == 5.0).all() and (pool_rows(c.keys, c, 0, 0, 48)[45:] == 5.0).all()


# ---- the binding: tensors that are not what the call takes ----

def test_queries_of_another_shape_are_refused(mp):
    """A leading dimension of one would pass for one row: the other tokens would be left out."""
    c = Cache(mp, "bf16", 8, 2, 128, 64, [300])
    _, cu_t = offsets([20])
    q = c.randn(20, 8, 128)
    out, lse = torch.full_like(q, 77.0), torch.zeros(20, 8, device=DEV)
    ws = torch.empty(max(1, mp.mp_chunk_workspace_bytes(c.cfg, 20, 20, 300)), dtype=torch.uint8, device=DEV)
    sc = torch.zeros(1, 2, c.ps * c.cols, device=DEV)
    for bad in (q[None], q.view(4, 5, 8, 128), q.view(2, 10 * 8, 128), q.flatten()):
        with pytest.raises(ValueError):
            mp.mp_chunk_attention(c.cfg, bad, cu_t, c.kv_len, 20, 300, c.keys, c.values, c.table, out, lse, ws, c.status)
        with pytest.raises(ValueError):
            mp.mp_cache_weights(c.cfg, bad, lse, cu_t, c.kv_len, 20, 300, c.keys, c.table, sc, c.status)
    assert (out == 77.0).all() and not sc.any()
    a, _ = attend(mp, c, q, cu_t, 20)
    b = torch.empty_like(q)
    mp.mp_chunk_attention(c.cfg, q.flatten(1), cu_t, c.kv_len, 20, 300, c.keys, c.values, c.table, b, None, ws, c.status)
    assert torch.equal(a, b)


# ---- few rows: 9 to 16 per KV head ----

FEW = [
    # q heads, kv heads, d, page, chunk lengths, cache lengths
    (12, 1, 128, 0, [1], [2000]),                    # a short cache, one cluster of slices
    (8, 2, 128, 64, [4, 3], [2000, 700]),
    (16, 1, 128, 16, [1, 1, 1], [300, 5, 500]),       # four slices
    (16, 1, 64, 0, [1], [200]),                      # two
    (9, 1, 128, 48, [1], [250]),
    (12, 1, 128, 64, [1], [20000]),                  # slices that a second kernel joins
    (8, 2, 128, 0, [4], [20000]),
    (8, 2, 64, 64, [4, 2], [20000, 13000]),
    (12, 1, 64, 0, [1, 1], [9000, 20000]),
    (16, 16, 128, 16, [16, 9, 1], [700, 3000, 40]),
    (16, 16, 64, 0, [13], [1000]),
    (24, 2, 128, 64, [1] * 40, [70 * (b + 1) for b in range(40)]),  # as many sequences as leave a slice each
    (8, 2, 128, 16, [4, 0, 3], [600, 50, 400]),      # a sequence without new tokens
    # and up to 8 rows
    (8, 1, 128, 0, [1], [20000]),
    (4, 1, 128, 64, [2, 0, 1], [600, 50, 400]),
    (8, 8, 64, 16, [8, 5], [500, 2000]),
    (4, 2, 64, 64, [4, 1], [9000, 200]),
]


@pytest.mark.parametrize("hq,hk,d,page,q_lens,kv", FEW)
def test_few_rows_keep_their_weights_exact(mp, hq, hk, d, page, q_lens, kv):
    assert hq // hk * max(q_lens) <= 16
    c = Cache(mp, "bf16", hq, hk, d, page, kv)
    cu, cu_t = offsets(q_lens)
    q = c.randn(cu[-1], hq, d, by=1.5)
    out, lse = attend(mp, c, q, cu_t, max(q_lens))
    assert c.status.item() == 0
    want, z, spread, slack = R.attention(q, cu, c.kv, c.keys, c.values, c.table, hk)
    eps_x = (d + 8) * 2.0 ** -24 * slack
    rel = 2 * eps_x + max(kv) * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -16
    tol = HALF["bf16"] * want.abs() + (1 + HALF["bf16"]) * rel[..., None] * spread
    assert ((out.double() - want).abs() <= tol).all()
    ztol = eps_x + (max(kv) + 8) * 2.0 ** -24 + 2.0 ** -21 * (1 + z.abs())
    assert ((lse.double() - z).abs() <= ztol).all()


# ---- workspaces ----

@pytest.mark.parametrize("dtype,hq,hk,page,total,max_q,max_kv", [
    ("bf16", 8, 2, 0, 90, 30, 4000), ("bf16", 8, 2, 64, 9, 3, 20000), ("f32", 8, 2, 64, 200, 70, 6000)])
def test_a_workspace_sized_for_the_largest_call_serves_smaller_ones(mp, dtype, hq, hk, page, total, max_q, max_kv):
    """One workspace for a serving loop's limits, and calls below them: other lengths, fewer rows,
    rows that belong to no sequence, each followed by a guard that nothing may touch."""
    d = 64
    lens = [max_kv, max_kv // 3, max_kv // 7]
    c = Cache(mp, dtype, hq, hk, d, page, lens)
    size = mp.mp_chunk_workspace_bytes(c.cfg, total, max_q, max_kv)
    buf = torch.full((size + 4096,), 0xA5, dtype=torch.uint8, device=DEV)
    ws = buf[:size]
    for m, n, rows in ((max_q, max_kv, total), (1, max_kv, 3), (1, max_kv, total), (2, max_kv // 2, 7), (1, 700, 3), (1, 300, 5), (2, 130, 6),
                       (max_q, 1000, total), (max_q // 2 + 1, 300, total), (1, 1, 3)):
        kv = [min(x, n) for x in lens]
        q_lens = [min(m, x) for x in kv]
        c.kv = kv
        c.kv_len.copy_(torch.tensor(kv, dtype=torch.int32))
        cu, cu_t = offsets(q_lens)
        if cu[-1] > rows:
            q_lens = [1, 1, 1]
            cu, cu_t = offsets(q_lens)
        q = c.randn(rows, hq, d, by=1.5)
        out, lse = attend(mp, c, q, cu_t, m, max_kv=n, workspace=ws)
        check_attention(c, dtype, q, cu, out, lse)
        assert (buf[size:] == 0xA5).all()
    assert c.status.item() == 0


# ---- eviction in place ----

def test_eviction_may_write_the_new_lengths_over_the_old(mp):
    """dst_len == kv_len: what a loop that keeps one length per sequence passes. Every head must
    have read the old length before it changes."""
    kv = [5000, 300, 2049, 1000, 4096, 0, 77, 3000]
    for rep in range(3):
        c = Cache(mp, "bf16", 8, 8, 64, 0, kv, seed=rep)
        t = Cache(mp, "bf16", 8, 8, 64, 0, [500] * 8, cap=500, fill="none")
        sc = make_scores("heavy", (8, 8, c.ps), c.gen)
        ws = torch.empty(mp.mp_evict_workspace_bytes(c.cfg, 5000, 500), dtype=torch.uint8, device=DEV)
        mp.mp_cache_evict(c.cfg, t.cfg, c.keys, c.values, None, c.kv_len, 5000, sc, 4, 16, 500, t.keys, t.values, None, None, c.kv_len, None,
                          ws, c.status)
        assert c.status.item() == 0 and c.kv_len.tolist() == [min(n, 500) for n in kv]
        for b, n in enumerate(kv):
            for h in range(8):
                at = torch.tensor(R.keep(sc[b, h], n, 4, 16, 500), dtype=torch.int64, device=DEV)
                assert torch.equal(t.keys[b, h, :len(at)], c.keys[b, h][at]) and torch.equal(t.values[b, h, :len(at)], c.values[b, h][at])


# ---- other threads run while a call is in the library ----

def test_calls_leave_the_interpreter_to_other_threads(mp, tmp_path):
    """A launch can wait for room in the device's queue. Stood in for by a library call that
    sleeps: Python code of another thread has to go on meanwhile."""
    import ctypes
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src, lib = tmp_path / "slow.c", str(tmp_path / "slow.so")
    src.write_text("#define _GNU_SOURCE\n#include <unistd.h>\nint slow(void) { usleep(400000); return 0; }\n")
    subprocess.run([cc, "-shared", "-fPIC", str(src), "-o", lib], check=True)
    slow = ctypes.cast(ctypes.CDLL(lib).slow, ctypes.c_void_p).value
    calls = mp._cache_calls()
    real = [ctypes.cast(getattr(mp._lib, f), ctypes.c_void_p).value
            for f in ("mp_cache_append", "mp_chunk_attention", "mp_cache_weights", "mp_cache_evict")]
    c = Cache(mp, "bf16", 2, 1, 64, 16, [20])
    _, cu_t = offsets([1])
    q, k = c.randn(1, 2, 64), c.randn(1, 1, 64)
    lse, sc = torch.zeros(1, 2, device=DEV), torch.zeros(1, 1, c.ps * c.cols, device=DEV)
    ws = torch.empty(1 << 16, dtype=torch.uint8, device=DEV)
    dlen = torch.zeros(1, dtype=torch.int32, device=DEV)
    four = [
        lambda: mp.mp_cache_append(c.cfg, mp.make_rotary(rot_dim=0), q, k, k, None, None, None, None, cu_t, c.kv_len, c.keys, c.values, c.table,
                                   q.clone(), c.status),
        lambda: mp.mp_chunk_attention(c.cfg, q, cu_t, c.kv_len, 1, 20, c.keys, c.values, c.table, q.clone(), lse, ws, c.status),
        lambda: mp.mp_cache_weights(c.cfg, q, lse, cu_t, c.kv_len, 1, 20, c.keys, c.table, sc, c.status),
        lambda: mp.mp_cache_evict(c.cfg, c.cfg, c.keys, c.values, c.table, c.kv_len, 20, sc, 0, 0, 4, c.keys, c.values, c.table, None, dlen, None,
                                  ws, c.status)]
    calls.bind(*[slow] * 4)
    try:
        for call in four:
            ticks, stop = [], threading.Event()

            def tick():
                while not stop.is_set():
                    ticks.append(time.perf_counter())
                    time.sleep(0.005)

            th = threading.Thread(target=tick)
            th.start()
            t0 = time.perf_counter()
            call()
            t1 = time.perf_counter()
            stop.set()
            th.join()
            assert t1 - t0 >= 0.35
            assert sum(t0 + 0.05 < t < t1 - 0.05 for t in ticks) >= 5
    finally:
        calls.bind(*real)


# ---- a process whose first call is a captured one ----

FIRST = '''
import sys
import torch
sys.path.insert(0, {root!r})
import lsh_sampled_sparse_centered_gb300 as mp
dev, d, hk, hq, n = "cuda:0", {d}, 2, 8, 3000
dt = {{"bf16": torch.bfloat16, "f32": torch.float32}}[{dtype!r}]
g = torch.Generator(device=dev).manual_seed(1)
rnd = lambda *s: torch.randn(*s, generator=g, device=dev).to(dt)
cfg = mp.make_cache_config(batch=1, kv_heads=hk, q_heads=hq, head_dim=d, page_size={cap}, n_pages=1, dtype={dtype!r})
dst = mp.make_cache_config(batch=1, kv_heads=hk, q_heads=hq, head_dim=d, page_size=100, n_pages=1, dtype={dtype!r})
m = {m}
keys, values = rnd(1, hk, {cap}, d), rnd(1, hk, {cap}, d)
q, k, v = rnd(m, hq, d), rnd(m, hk, d), rnd(m, hk, d)
cu = torch.tensor([0, m], dtype=torch.int32, device=dev)
kv = torch.tensor([{n}], dtype=torch.int32, device=dev)
inv = torch.ones(d // 2, dtype=torch.float64, device=dev)
ws = torch.empty(1 << 25, dtype=torch.uint8, device=dev)
status = torch.zeros(1, dtype=torch.int32, device=dev)
q_out, out, lse = torch.empty_like(q), torch.empty_like(q), torch.empty(m, hq, device=dev)
sc = torch.zeros(1, hk, {cap}, device=dev)
dk, dv = torch.zeros(1, hk, 100, d, dtype=dt, device=dev), torch.zeros(1, hk, 100, d, dtype=dt, device=dev)
dlen, kept = torch.zeros(1, dtype=torch.int32, device=dev), torch.zeros(1, hk, 100, dtype=torch.int32, device=dev)
def step():
    mp.mp_cache_append(cfg, mp.make_rotary(rot_dim=d), q, k, v, None, None, inv, None, cu, kv, keys, values, None, q_out, status)
    mp.mp_chunk_attention(cfg, q_out, cu, kv, m, {n}, keys, values, None, out, lse, ws, status)
    mp.mp_cache_weights(cfg, q_out, lse, cu, kv, m, {n}, keys, None, sc, status)
    mp.mp_cache_evict(cfg, dst, keys, values, None, kv, {n}, sc, 4, 16, 100, dk, dv, None, None, dlen, kept, ws, status)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    step()
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in (q_out, out, lse, sc, dk, dv, dlen, kept)]
sc.zero_()
step()
torch.cuda.synchronize()
assert status.item() == 0
assert all(torch.equal(a, b) for a, b in zip(got, (q_out, out, lse, sc, dk, dv, dlen, kept)))
print("same")
'''


@pytest.mark.parametrize("dtype,d,m,cap,n", [("bf16", 128, 1, 3000, 2000), ("bf16", 64, 3, 9000, 8000), ("bf16", 128, 50, 3000, 2500),
                                             ("f32", 64, 5, 3000, 2900)])
def test_a_first_call_may_be_captured(dtype, d, m, cap, n):
    """Kernels are loaded and occupancies asked for under the capture; equal bits afterwards."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import sys
    import __graft_entry__
    __graft_entry__.build()
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST.format(root=root, dtype=dtype, d=d, m=m, cap=cap, n=n)], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("same"), (r.stdout[-500:], r.stderr[-2000:])
