"""Waits that run out in the attention over shared prefixes: one CTA of the large tiles stops half way
(MP_FAULT_INJECT=prefix_wait, in the bounds-checking build only), the bounded waits for it expire, the call
ends with MP_STATUS_WAIT_TIMEOUT, and the next call is right. The cases run in a child process with that
build."""
import os
import subprocess
import sys

import pytest
import torch

from test_gpu_cache import offsets
from test_gpu_cache_waits import CHILD, LIMIT, ROOT, mp, timed  # noqa: F401
from test_gpu_share import Shared, attend_prefix, check_prefix

pytestmark = pytest.mark.gpu


@pytest.mark.skipif(not CHILD, reason="in the child process")
@pytest.mark.parametrize("hq,hk,d,page,q_lens,prefix", [
    (8, 2, 128, 64, [600, 500], 12000),       # chunks: groups and sequences on large tiles
    (8, 2, 64, 16, [600, 500], 12000),
    (32, 8, 128, 64, [1] * 20, 60000),        # slices, the halves of a tile on alternate steps, own slots beside
    (32, 8, 64, 0, [1] * 20, 60000),
    (16, 2, 128, 0, [1] * 40, 60000),         # slices of several tiles
    (16, 2, 64, 16, [1] * 40, 60000),
])
def test_child_prefix(mp, monkeypatch, hq, hk, d, page, q_lens, prefix):  # noqa: F811
    c = Shared(mp, "bf16", hq, hk, d, page, [m + 300 for m in q_lens], [len(q_lens)], [prefix])
    cu, cu_t = offsets(q_lens)
    q = c.randn(cu[-1], hq, d, by=1.5)
    attend_prefix(mp, c, q, cu, cu_t, max(q_lens))
    monkeypatch.setenv("MP_FAULT_INJECT", "prefix_wait")
    _, s = timed(lambda: attend_prefix(mp, c, q, cu, cu_t, max(q_lens)))
    assert c.status.item() == mp.MP_STATUS_WAIT_TIMEOUT and LIMIT <= s < 6 * LIMIT
    monkeypatch.delenv("MP_FAULT_INJECT")
    c.status.zero_()
    for _ in range(3):
        (out, lse), s = timed(lambda: attend_prefix(mp, c, q, cu, cu_t, max(q_lens)))
        assert c.status.item() == 0 and s < LIMIT / 4
        check_prefix(c, "bf16", q, cu, out, lse)


@pytest.mark.skipif(CHILD, reason="the parent process")
def test_waits_of_the_prefix_attention_run_out():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__._builder().build(check=True)
    r = subprocess.run([sys.executable, "-m", "pytest", __file__, "-m", "gpu", "-q", "-x", "-p", "no:cacheprovider", "-k", "child"], cwd=ROOT,
                       env=dict(os.environ, MP_BOUNDS_CHECK="1"), capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "6 passed" in r.stdout, (r.stdout[-3000:], r.stderr[-2000:])
