"""Waits that run out in the tensor-core kernels of the cache operators: one CTA stops half way
(MP_FAULT_INJECT=chunk_wait or weights_wait, in the bounds-checking build only), the others' bounded
waits for it expire, the call ends with MP_STATUS_WAIT_TIMEOUT, and the next call is right: nothing
of the first is left in flight. The cases run in a child process with that build."""
import os
import subprocess
import sys
import time

import pytest
import torch

import cache_reference as R
from test_gpu_cache import DEV, Cache, attend, check_attention, offsets

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CHILD = os.environ.get("MP_BOUNDS_CHECK") == "1"
LIMIT = 2.0  # seconds that a wait lasts at least


@pytest.fixture(scope="module")
def mp():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import lsh_sampled_sparse_centered_gb300 as m
    return m


def timed(call):
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    r = call()
    torch.cuda.synchronize()
    return r, time.perf_counter() - t0


@pytest.mark.skipif(not CHILD, reason="in the child process")
@pytest.mark.parametrize("d,page", [(128, 0), (64, 16)])
def test_child_attention(mp, monkeypatch, d, page):
    c = Cache(mp, "bf16", 8, 2, d, page, [1000])
    cu, cu_t = offsets([300])
    q = c.randn(300, 8, d)
    attend(mp, c, q, cu_t, 300)
    monkeypatch.setenv("MP_FAULT_INJECT", "chunk_wait")
    (out, lse), s = timed(lambda: attend(mp, c, q, cu_t, 300))
    assert c.status.item() == mp.MP_STATUS_WAIT_TIMEOUT and LIMIT <= s < 6 * LIMIT
    assert torch.isfinite(out[64:]).all()  # the other CTAs' tiles
    monkeypatch.delenv("MP_FAULT_INJECT")
    c.status.zero_()
    for _ in range(3):
        (out, lse), s = timed(lambda: attend(mp, c, q, cu_t, 300))
        assert c.status.item() == 0 and s < LIMIT / 4
        check_attention(c, "bf16", q, cu, out, lse)


@pytest.mark.skipif(not CHILD, reason="in the child process")
@pytest.mark.parametrize("d,page", [(128, 0), (64, 16)])
def test_child_weights(mp, monkeypatch, d, page):
    c = Cache(mp, "bf16", 8, 2, d, page, [1000])
    cu, cu_t = offsets([300])
    q = c.randn(300, 8, d)
    lse = R.attention(q, cu, c.kv, c.keys, c.values, c.table, 2)[1].float()
    scores = torch.zeros(1, 2, c.ps * c.cols, device=DEV)
    call = lambda: mp.mp_cache_weights(c.cfg, q, lse, cu_t, c.kv_len, 300, 1000, c.keys, c.table, scores, c.status)
    call()
    want = scores.clone()
    monkeypatch.setenv("MP_FAULT_INJECT", "weights_wait")
    scores.zero_()
    _, s = timed(call)
    assert c.status.item() == mp.MP_STATUS_WAIT_TIMEOUT and LIMIT <= s < 6 * LIMIT
    monkeypatch.delenv("MP_FAULT_INJECT")
    c.status.zero_()
    for _ in range(3):
        scores.zero_()
        _, s = timed(call)
        assert c.status.item() == 0 and s < LIMIT / 4
        assert torch.equal(scores, want)
    assert ((scores.double().sum(-1) - 1200.0).abs() <= 2.0 ** -10 * 1200.0).all()  # one per query head and token


@pytest.mark.skipif(CHILD, reason="the parent process")
def test_waits_that_run_out_end_the_call_and_leave_nothing_behind():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__._builder().build(check=True)
    r = subprocess.run([sys.executable, "-m", "pytest", __file__, "-m", "gpu", "-q", "-x", "-p", "no:cacheprovider", "-k", "child"], cwd=ROOT,
                       env=dict(os.environ, MP_BOUNDS_CHECK="1"), capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "4 passed" in r.stdout, (r.stdout[-3000:], r.stderr[-2000:])
