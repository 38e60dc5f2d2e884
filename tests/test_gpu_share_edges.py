"""Planning, attention over shared prefixes and rotation on the GPU where one call meets another: tiles of one CTA,
threads that call at once, a cache that goes on after it was turned. Tolerances as in test_gpu_share.py."""
import math
import os
import subprocess
import sys
import threading

import pytest
import torch

import cache_reference as R
import share_reference as S
from test_gpu_cache import DEV, HALF, Cache, offsets
from test_gpu_share import Plan, Shared, attend_prefix, check_prefix, freq, ints, mp  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hk,d,m,n,prefix", [
    (8, 64, 500, 2048, 40),     # 24 CTAs have a tile that sees none of its slots before one that sees some
    (16, 64, 700, 1000, 0),     # 91
    (32, 128, 640, 640, 300),
    (5, 128, 333, 4000, 64),
])
def test_fp32_tiles_behind_tiles_that_see_nothing(mp, hk, d, m, n, prefix):  # noqa: F811
    """The first tiles of a chunk see none of the pieces of its last slots. What such a piece asked for must not come
    over the next tile's rows of Q, however late it comes: Q is out of L2 in every call, and the bits are equal."""
    c = Shared(mp, "f32", hk, hk, d, 64, [n], [1], [prefix])
    cu, cu_t = offsets([m])
    q = c.randn(m, hk, d, by=1.5)
    other = torch.empty(1 << 26, device=DEV)
    first = None
    for i in range(30):
        other.fill_(float(i))
        out, lse = attend_prefix(mp, c, q, cu, cu_t, m)
        first = first if first is not None else (out, lse)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    check_prefix(c, "f32", q, cu, *first)
    assert c.status.item() == 0


@pytest.mark.parametrize("hq,hk,d,page,q_lens,own,groups,prefixes", [
    (8, 2, 128, 16, [1, 1, 1], [1, 17, 300], [3], [333]),                            # all rows few
    (16, 16, 64, 0, [3, 1, 2], [30, 700, 5], [2], [4000]),
    (8, 1, 128, 64, [1] * 20, [5 + 30 * i for i in range(20)], [20], [500]),         # 160 rows of a group over a short prefix
    (4, 1, 64, 16, [4] * 15, [20 + 9 * i for i in range(15)], [10, 5], [300, 900]),
    (8, 1, 128, 16, [1] * 90, [1 + 7 * i for i in range(90)], [80], [333]),          # 640 rows
    (16, 2, 64, 48, [2, 1, 3] * 20, [9 + 11 * i for i in range(60)], [50, 9], [200, 77]),  # 800 rows in blocks of 32
    (24, 6, 128, 0, [1] * 150, [1 + i % 50 for i in range(150)], [1, 149], [40, 64]),
])
def test_few_rows_have_weights_of_two_terms(mp, hq, hk, d, page, q_lens, own, groups, prefixes):  # noqa: F811
    """Where the header says so, in both passes: a weight is off by what two roundings to bf16 leave of it, 2^-16, where
    one leaves 2^-8."""
    c = Shared(mp, "bf16", hq, hk, d, page, own, groups, prefixes)
    cu, cu_t = offsets(q_lens)
    q = c.randn(cu[-1], hq, d, by=1.5)
    out, _ = attend_prefix(mp, c, q, cu, cu_t, max(q_lens))
    want, _, spread, slack = S.prefix_attention(q, cu, c.kv, c.keys, c.values, c.table, c.groups, c.prefixes, c.pre.keys, c.pre.values, c.pre.table, hk)
    rel = 2 * (d + 8) * 2.0 ** -24 * slack + (max(own) + max(prefixes)) * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -16
    assert ((out.double() - want).abs() <= HALF["bf16"] * want.abs() + (1 + HALF["bf16"]) * rel[..., None] * spread).all()


def together(*loops):
    """Runs the functions in a thread each, at once; the first exception of any is raised."""
    failed = []
    start = threading.Barrier(len(loops))

    def run(f):
        try:
            start.wait()
            f()
        except Exception as e:
            failed.append(e)

    threads = [threading.Thread(target=run, args=(f,)) for f in loops]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    if failed:
        raise failed[0]


KINDS = [  # one batch for each way the attention goes: dtype, q heads, kv heads, d, page, tokens, own lengths, groups, prefixes, limit of the prefixes
    ("bf16", 8, 2, 128, 16, [1] * 3, [40, 300, 7], [3], [500], 600),            # few rows for both
    ("bf16", 32, 8, 64, 64, [1] * 20, [30 + 9 * i for i in range(20)], [20], [9000], 12000),   # slices, a half each step
    ("bf16", 16, 2, 128, 0, [1] * 40, [30 + 9 * i for i in range(40)], [40], [9000], 12000),   # slices of two tiles
    ("bf16", 40, 40, 64, 32, [1] * 200, [9 + i % 70 for i in range(200)], [200], [900], 20000),  # few own rows, tiles for the prefix
    ("bf16", 8, 2, 128, 64, [100, 33], [100, 400], [2], [700], 5000),           # tiles for both
    ("f32", 8, 2, 128, 16, [1] * 3, [40, 300, 7], [3], [500], 600),             # few rows
    ("f32", 8, 2, 64, 16, [1] * 9, [40 + i for i in range(9)], [9], [500], 600),  # few own rows, tiles for the prefix
    ("f32", 8, 8, 64, 0, [50, 33], [100, 400], [2], [700], 5000),               # tiles for both
]


@pytest.mark.parametrize("kind", KINDS)
def test_prefix_attention_of_rows_that_see_nothing_at_all(mp, kind):  # noqa: F811
    """Every prefix and every cache is empty, whatever the limits let expect; then some of them are not."""
    dtype, hq, hk, d, page, q_lens, own, groups, prefixes, most = kind
    c = Shared(mp, dtype, hq, hk, d, page, own, groups, prefixes, cap=max(own) + 50, pcap=most)
    cu, cu_t = offsets(q_lens)
    q = c.randn(cu[-1] + 2, hq, d, by=1.5)
    for kv, pl in (([0] * len(own), [0] * len(groups)), ([0] * len(own), prefixes), ([0] * (len(own) - 1) + own[-1:], [0] * len(groups)), (own, prefixes)):
        c.kv, c.prefixes = kv, pl
        c.kv_len.copy_(ints(kv))
        c.pre.kv_len.copy_(ints(pl))
        out, lse = attend_prefix(mp, c, q, cu, cu_t, max(q_lens), max_kv=max(own) + 50, max_prefix=most)
        if not any(kv) and not any(pl):
            assert (out[:cu[-1]] == 0).all() and (lse[:cu[-1]] == -math.inf).all() and (out[cu[-1]:] == 77).all()
        else:
            check_prefix(c, dtype, q, cu, out, lse)
    assert c.status.item() == 0


@pytest.mark.parametrize("kind", KINDS)
def test_weights_behind_a_prefix(mp, kind):  # noqa: F811
    """The own slots' weights by the lse over prefix and own slots: what the formula gives for that lse, with the weights'
    own tolerance (test_gpu_cache.py), tokens in front of their cache's first slot among them."""
    dtype, hq, hk, d, page, q_lens, own, groups, prefixes, most = kind
    own = [max(1, own[0] // 3)] + own[1:]
    c = Shared(mp, dtype, hq, hk, d, page, own, groups, prefixes)
    cu, cu_t = offsets(q_lens)
    q = c.randn(cu[-1], hq, d, by=1.5)
    _, lse = attend_prefix(mp, c, q, cu, cu_t, max(q_lens))
    scores = torch.zeros(len(own), hk, c.ps * c.cols, device=DEV)
    want, slack = R.weights(q, lse, cu, own, c.keys, c.table, scores)
    mp.mp_cache_weights(c.cfg, q, lse, cu_t, c.kv_len, max(q_lens), max(own), c.keys, c.table, scores, c.status)
    for b, n in enumerate(own):
        rel = (d + 8) * 2.0 ** -24 * slack[b, :, :n] + 2.0 ** -21 * (1 + lse.abs().max().item()) + (hq // hk * max(q_lens) + 2) * 2.0 ** -24
        assert ((scores[b, :, :n].double() - want[b, :, :n]).abs() <= rel * want[b, :, :n] + 1e-30).all(), b
    assert c.status.item() == 0


@pytest.mark.parametrize("dtype,hq,hk,d,page,q_lens,own,groups,prefixes", [
    ("bf16", 300, 1, 64, 16, [1, 2], [40, 300], [2], [500]),        # more heads of a group than a tile has rows
    ("bf16", 600, 2, 128, 0, [1, 1, 1], [40, 1, 9], [1, 2], [5000, 33]),
    ("f32", 300, 1, 128, 32, [1, 2], [40, 300], [2], [500]),
    ("bf16", 1, 1, 128, 16, [1, 3, 40], [40, 300, 41], [3], [500]),  # a single head
    ("f32", 1, 1, 64, 0, [1, 3, 40], [40, 300, 41], [3], [500]),
    ("bf16", 65, 13, 64, 16, [1] * 7, [5, 16, 17, 31, 32, 33, 1], [3, 3], [15, 17]),
])
def test_prefix_attention_of_odd_heads(mp, dtype, hq, hk, d, page, q_lens, own, groups, prefixes):  # noqa: F811
    c = Shared(mp, dtype, hq, hk, d, page, own, groups, prefixes)
    cu, cu_t = offsets(q_lens)
    q = c.randn(cu[-1] + 1, hq, d, by=1.5)
    out, lse = attend_prefix(mp, c, q, cu, cu_t, max(q_lens))
    check_prefix(c, dtype, q, cu, out, lse)
    assert c.status.item() == 0


def test_prefix_attentions_from_several_threads(mp):  # noqa: F811
    """A thread, a stream and a workspace for each of the ways: the bits that each gives alone."""
    runs = []
    for dtype, hq, hk, d, page, q_lens, own, groups, prefixes, most in KINDS:
        c = Shared(mp, dtype, hq, hk, d, page, own, groups, prefixes)
        cu, cu_t = offsets(q_lens)
        q = c.randn(cu[-1], hq, d, by=1.5)
        want = attend_prefix(mp, c, q, cu, cu_t, max(q_lens))
        out, lse = torch.empty_like(q), torch.empty_like(want[1])
        g, l = c.limits(cu)
        ws = torch.empty(mp.mp_prefix_workspace_bytes(c.cfg, c.pre.cfg, cu[-1], max(q_lens), max(own), g, l), dtype=torch.uint8, device=DEV)
        runs.append((c, q, cu_t, max(q_lens), max(own), g, l, out, lse, ws, torch.cuda.Stream(), want))
    torch.cuda.synchronize()

    def loop(c, q, cu_t, m, n, g, l, out, lse, ws, st, want):
        def run():
            for _ in range(200):
                mp.mp_prefix_attention(c.cfg, c.pre.cfg, q, cu_t, c.kv_len, m, n, c.keys, c.values, c.table, c.cu_group, c.pre.kv_len, g, l,
                                       c.pre.keys, c.pre.values, c.pre.table, out, lse, ws, c.status, stream=st)
        return run

    together(*(loop(*r) for r in runs))
    torch.cuda.synchronize()
    for c, *_, out, lse, ws, st, want in runs:
        assert c.status.item() == 0 and torch.equal(out, want[0]) and torch.equal(lse, want[1])


def in_a_new_thread(call):
    """What `call` gives in a thread that has asked nothing of CUDA before."""
    got = []
    together(lambda: got.append(call()))
    torch.cuda.synchronize()
    return got[0]


@pytest.mark.parametrize("kind", KINDS)
def test_a_threads_first_call_is_a_prefix_attention(mp, kind):  # noqa: F811
    dtype, hq, hk, d, page, q_lens, own, groups, prefixes, most = kind
    c = Shared(mp, dtype, hq, hk, d, page, own, groups, prefixes)
    cu, cu_t = offsets(q_lens)
    q = c.randn(cu[-1], hq, d, by=1.5)
    out, lse = attend_prefix(mp, c, q, cu, cu_t, max(q_lens))
    g, l = c.limits(cu)
    ws = torch.empty(mp.mp_prefix_workspace_bytes(c.cfg, c.pre.cfg, cu[-1], max(q_lens), max(own), g, l), dtype=torch.uint8, device=DEV)
    o, z = torch.empty_like(out), torch.empty_like(lse)
    torch.cuda.synchronize()
    in_a_new_thread(lambda: mp.mp_prefix_attention(c.cfg, c.pre.cfg, q, cu_t, c.kv_len, max(q_lens), max(own), c.keys, c.values, c.table, c.cu_group,
                                                   c.pre.kv_len, g, l, c.pre.keys, c.pre.values, c.pre.table, o, z, ws, c.status))
    assert torch.equal(o, out) and torch.equal(z, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m", [1, 100])
def test_a_threads_first_call_is_one_of_the_cache(mp, dtype, m):  # noqa: F811
    """Attention and weights of a token and of a chunk, append, plan, rotation and eviction, each in a thread of its own."""
    c = Cache(mp, dtype, 8, 2, 128, 16, [300, m + 5])
    cu, cu_t = offsets([m, m])
    q, k = c.randn(2 * m, 8, 128), c.randn(2 * m, 2, 128)
    rotary, f = mp.make_rotary(rot_dim=128), freq(128)
    ws = torch.empty(1 << 24, dtype=torch.uint8, device=DEV)
    dst = mp.make_cache_config(batch=2, kv_heads=2, q_heads=8, head_dim=128, page_size=64, n_pages=2, dtype=dtype)
    shape = (2, 2, 64, 128)

    def calls():
        """[(call, what it writes)], each call with outputs of its own."""
        keys, values = c.keys.clone(), c.values.clone()
        out, lse, rotated = torch.zeros_like(q), torch.zeros(2 * m, 8, device=DEV), torch.zeros_like(q)
        scores = torch.zeros(2, 2, c.ps * c.cols, device=DEV)
        spread = torch.rand(scores.shape, generator=torch.Generator().manual_seed(1)).to(DEV)
        dk, dv, kept, length = torch.zeros(shape, dtype=c.dtype, device=DEV), torch.zeros(shape, dtype=c.dtype, device=DEV), ints([0] * 2 * 2 * 50), ints([0, 0])
        z = torch.full((2 * m, 8), 3.0, device=DEV)
        plan = [ints([0, 0, 0]), ints([0, 0])]
        return [
            (lambda: mp.mp_chunk_attention(c.cfg, q, cu_t, c.kv_len, m, 300, c.keys, c.values, c.table, out, lse, ws), (out, lse)),
            (lambda: mp.mp_cache_weights(c.cfg, q, z, cu_t, c.kv_len, m, 300, c.keys, c.table, scores), (scores[:, :, :m + 5],)),
            (lambda: mp.mp_cache_append(c.cfg, rotary, q, k, k, None, None, f, None, cu_t, c.kv_len, keys, values, c.table, rotated), (rotated,)),
            (lambda: mp.mp_cache_rotate(c.cfg, rotary, keys, c.table, c.kv_len, 300, f, f * 0.5), (keys.nan_to_num(0.0),)),
            (lambda: mp.mp_cache_evict(c.cfg, dst, c.keys, c.values, c.table, c.kv_len, 300, spread, 4, 8, 50, dk, dv, None, None, length, kept, ws), (dk, dv, length, kept)),
            (lambda: mp.mp_cache_plan(c.cfg, ints([0, -3]), None, c.kv_len, ints([0]), 8, c.table.clone(), torch.zeros(c.pages, dtype=torch.int32, device=DEV), plan[1],
                                      ints([0]), plan[0]), plan),
        ]

    for i, ((here, want), (there, got)) in enumerate(zip(calls(), calls())):
        here()
        torch.cuda.synchronize()
        in_a_new_thread(there)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i


def test_plans_of_two_sizes_from_two_threads(mp):  # noqa: F811
    """A batch of 8192 sequences needs more shared memory than one of 1500: neither thread's calls take it from the
    other's, and both pools are planned as if they were alone."""
    sizes, steps = (8192, 1500, 700), 2000
    pools = [Plan(mp, [10 + i] * n, 16, 8, spare=2 * n, seed=i) for i, n in enumerate(sizes)]
    cu = [torch.zeros(n + 1, dtype=torch.int32, device=DEV) for n in sizes]
    change = [(ints([1] * n), ints([-1] * n)) for n in sizes]
    streams = [torch.cuda.Stream() for _ in sizes]
    torch.cuda.synchronize()

    def loop(i):
        p, st = pools[i], streams[i]

        def run():
            for k in range(steps):
                mp.mp_cache_plan(p.cfg, change[i][k % 2], None, p.d_kv, p.d_n, 3 * p.batch, p.d_table, p.d_free, p.d_kv, p.d_n, cu[i], None, None, None,
                                 p.status, stream=st)
        return run

    together(*(loop(i) for i in range(len(sizes))))
    torch.cuda.synchronize()
    for p, c in zip(pools, cu):
        kv, n_free, table, free = p.kv, p.n_free, p.table, p.free
        for x in (1, -1):  # every two steps end where they began, the pages given back in another order once
            kv, n_free, cu_want, table, free, _ = S.plan([x] * p.batch, kv, [0] * p.batch, table, free, n_free, 16, 8, 3 * p.batch)
        assert p.d_kv.tolist() == kv == p.kv and p.d_n.tolist() == [n_free] and c.tolist() == cu_want and p.status.item() == 0


FIRST_PLAN = '''
import sys
import torch
sys.path.insert(0, {root!r})
import lsh_sampled_sparse_centered_gb300 as mp
ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda:0")
n = 3000
cfg = mp.make_cache_config(batch=n, kv_heads=1, q_heads=1, head_dim=64, page_size=16, n_pages=2 * n, max_pages=4)
table, free, n_free = torch.zeros(n, 4, dtype=torch.int32, device="cuda:0"), torch.arange(2 * n, dtype=torch.int32, device="cuda:0"), ints(2 * n)
change, kv, cu = torch.ones(n, dtype=torch.int32, device="cuda:0"), torch.zeros(n, dtype=torch.int32, device="cuda:0"), torch.zeros(n + 1, dtype=torch.int32, device="cuda:0")
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    mp.mp_cache_plan(cfg, change, None, kv, n_free, n, table, free, kv, n_free, cu)
graph.replay()
torch.cuda.synchronize()
assert (kv == 1).all() and n_free.item() == n and cu[-1].item() == n and table[:, 0].tolist() == list(range(2 * n - 1, n - 1, -1))
print("same")
'''


def test_a_first_plan_of_many_sequences_may_be_captured():
    """What it asks about its kernel, it may ask under a capture."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_PLAN.format(root=root)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("same"), (r.stdout[-500:], r.stderr[-2000:])


# ----------------------------------------------------------------------------------
# rotation
# ----------------------------------------------------------------------------------

def turn_unit_keys(mp, units, to_freq):  # noqa: F811
    """(-sine, cosine) that a bf16 key (0, 1) is turned by, for angles of so many 2^-32ths of a turn."""
    n = len(units)
    keys = torch.zeros(1, 1, n, 64, dtype=torch.bfloat16, device=DEV)
    keys[..., 1] = 1
    cfg = mp.make_cache_config(batch=1, kv_heads=1, q_heads=1, head_dim=64, page_size=n, n_pages=1, dtype="bf16")
    one = torch.tensor([2 * math.pi * 2.0 ** -32], dtype=torch.float64, device=DEV)
    at, zero = units.to(torch.int32).view(1, 1, n), torch.zeros(1, 1, n, dtype=torch.int32, device=DEV)
    status = ints([0])
    mp.mp_cache_rotate(cfg, mp.make_rotary(rot_dim=2, interleaved=True), keys, None, ints([n]), n, one, one.clone() if to_freq else None, zero, at, 1.0, status)
    assert status.item() == 0
    return keys[0, 0, :, 0].double(), keys[0, 0, :, 1].double()


@pytest.mark.parametrize("two", [False, True])
def test_bf16_sines_and_cosines_within_their_bound(mp, two):  # noqa: F811
    """2^-20, seen where they are small: next to a quarter of a turn the result's rounding, half a step of at most 2^-8
    of it, is a fraction of that. The angles are 2^-32ths of a turn; the phases' own rounding is two of them (2^-28).
    On average they are off by less than 2^-22: of the 3.7e-7 that the dropped bits are in the middle, at least 1.5e-7
    are put back; the sines' own errors do not all point one way. (All of it, one way, were 3.4e-7 to 4.9e-7.)"""
    near = torch.arange(-6000, 6000)
    for units in [near + q * 2 ** 30 for q in (-1, 0, 1)] + [-2 ** 31 + 1 + near.abs(), 2 ** 31 - 1 - near.abs()]:
        sine, cosine = turn_unit_keys(mp, units.to(DEV), two)
        t = units.double() * (2 * math.pi * 2.0 ** -32)  # on the host, whose sines are exact enough
        for name, got, want in (("sine", -sine.cpu(), torch.sin(t)), ("cosine", cosine.cpu(), torch.cos(t))):
            over = (got - want).abs() - 2.0 ** -8 * want.abs()
            assert over.max() <= 2.0 ** -20 + 2.0 ** -28, (name, over.max().item())
            if want.abs().max() < 2.0 ** -10:
                assert (got - want).mean().abs() <= 2.0 ** -22, (name, units[0].item(), (got - want).mean().item())


@pytest.mark.parametrize("rot,norm", [(128, True), (128, False), (64, True), (64, False)])
def test_a_scaled_cache_goes_on(mp, rot, norm):  # noqa: F811
    """Keys appended behind scaled ones, their k (or k_norm) multiplied in its first rot_dim elements, are the keys that
    the append and then the rotation would have given: each of the two is within 2^-20 of the size of an element's pair
    of it (the rotation's tolerance), and the factor's own rounding is a part of that."""
    n, m, hk, d, scale = 70, 23, 2, 128, 1.375 * math.sqrt(0.7)
    g = torch.Generator().manual_seed(rot)
    q, k, v = (torch.randn(n, hk, d, generator=g).to(DEV) for _ in range(3))
    w = 1 + 0.3 * torch.randn(d, generator=g).to(DEV)
    by = torch.ones(d, device=DEV)
    by[:rot] = scale
    rotary, f = mp.make_rotary(rot_dim=rot, eps=1e-6), freq(rot)

    def append(c, kv, rows, k, w):
        cu, cu_t = offsets([len(rows)])
        mp.mp_cache_append(c.cfg, rotary, q[rows], k[rows].contiguous(), v[rows], None, w, f, None, cu_t, ints([kv]), c.keys, c.values, c.table,
                           torch.empty_like(q[rows]), c.status)

    whole, on = (Cache(mp, "f32", hk, hk, d, 16, [n]) for _ in range(2))
    append(whole, n, list(range(n)), k, w if norm else None)
    mp.mp_cache_rotate(whole.cfg, rotary, whole.keys, whole.table, ints([n]), n, f, None, None, None, scale, whole.status)
    append(on, n - m, list(range(n - m)), k, w if norm else None)
    mp.mp_cache_rotate(on.cfg, rotary, on.keys, on.table, ints([n - m]), n, f, None, None, None, scale, on.status)
    append(on, n, list(range(n - m, n)), k if norm else k * by, w * by if norm else None)
    for h in range(hk):
        a, b = R.gather(whole.keys, whole.table, 0, h, n), R.gather(on.keys, on.table, 0, h, n)
        size = a.abs()
        size[:, :rot] = torch.hypot(a[:, :rot // 2], a[:, rot // 2:rot]).repeat(1, 2)
        assert torch.equal(a[:n - m], b[:n - m])
        assert ((a - b).abs() <= 2 * 2.0 ** -20 * size).all()
    assert whole.status.item() == 0 and on.status.item() == 0
