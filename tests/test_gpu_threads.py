"""Building tables and decoding from several threads: over tables of other sizes at once (kernels whose shared memory goes by
the call's sizes), and as a thread's first call. The results are those of the same calls alone."""
import pytest
import torch

import workloads as WL
from gpu_harness import DeviceRun
from test_gpu_share_edges import together

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mp():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import lsh_sampled_sparse_centered_gb300 as m
    return m


def workload(name, n, K, L, heads, dtype, seed):
    return WL.Workload(name, layers=1, batch=1, kv_heads=1, q_heads=heads, head_dim=128, n_prefill=n, steps=1, append=False, K=K, L=L, dtype=dtype, seed=seed)


@pytest.mark.parametrize("mode,threshold,small,large", [
    # the bucket walk's bitmaps, by the tokens; the buckets' offsets, by K
    ("MP_MATCH_CSR", 2, workload("csr-s", 30000, 8, 20, 2, "bf16", 1), workload("csr-l", 300000, 12, 40, 2, "bf16", 2)),
    ("MP_MATCH_CSR", 3, workload("csr3-s", 50000, 6, 20, 2, "f32", 3), workload("csr3-l", 150000, 11, 30, 2, "f32", 4)),
    # the scan's codes, by heads of a group times tables
    ("MP_MATCH_SCAN", 2, workload("scan-s", 3000, 4, 400, 64, "bf16", 5), workload("scan-l", 4000, 5, 1000, 64, "bf16", 6)),
    ("MP_MATCH_SCAN", 3, workload("scan3-s", 3000, 4, 200, 150, "bf16", 7), workload("scan3-l", 4000, 5, 250, 200, "bf16", 8)),
])
def test_two_threads_of_other_sizes(mp, mode, threshold, small, large):
    runs, alone, steps = [], [], 3000 if mode == "MP_MATCH_CSR" else 800
    for wl in (small, large):
        r = DeviceRun(mp, wl, WL.generate(wl), "cuda:0", threshold=threshold, match_mode=getattr(mp, mode))
        r.build()
        q = r.queries[0].contiguous()
        mp.mp_decode_attention(r.cfg, r.tables, r.keys, r.values, wl.n_prefill, q, r.out, r.scratch)
        torch.cuda.synchronize()
        runs.append((r, q, torch.cuda.Stream()))
        alone.append(r.out.clone())
    torch.cuda.synchronize()

    def loop(r, q, st):
        def run():
            for i in range(steps):
                if i % 100 == 0:
                    mp.mp_build_tables(r.cfg, r.keys, r.wl.n_prefill, r.W, r.tables, stream=st)
                mp.mp_decode_attention(r.cfg, r.tables, r.keys, r.values, r.wl.n_prefill, q, r.out, r.scratch, stream=st)
        return run

    together(*(loop(*x) for x in runs))
    torch.cuda.synchronize()
    for (r, _, _), want in zip(runs, alone):
        assert r.status() == 0 and torch.equal(r.out, want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_threads_first_call_builds_appends_or_decodes(mp, dtype):
    """Each call in a thread that has asked nothing of CUDA before gives what it gives in this one."""
    wl = WL.Workload("first", layers=1, batch=1, kv_heads=2, q_heads=8, head_dim=128, n_prefill=2000, steps=4, append=True, K=8, L=30, dtype=dtype, seed=9)
    t = WL.generate(wl)
    here, there = (DeviceRun(mp, wl, t, "cuda:0") for _ in range(2))
    torch.cuda.synchronize()
    calls = lambda r: [r.build, lambda: r.decode(0, 2000), lambda: r.append(2000), lambda: r.decode(1, 2001), lambda: r.step(2, 2002)]
    for i, (a, b) in enumerate(zip(calls(here), calls(there))):
        a()
        torch.cuda.synchronize()
        together(b)
        torch.cuda.synchronize()
        assert here.status() == there.status() == 0
        assert i in (0, 2) or torch.equal(here.out, there.out), i
