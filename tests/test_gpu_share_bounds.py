"""The bounds-checking build over planning, attention over shared prefixes and rotation: every index that comes from
lengths, tables and numbers of pieces is tested against its buffer, and a failure sets MP_STATUS_BAD_INDEX, which the
cases' own checks of the status would show. In that build a warp of the few-row kernel can be made to wait for bytes that
never come (MP_FAULT_INJECT=prefix_few_wait): the call ends with MP_STATUS_WAIT_TIMEOUT and the next one is right. The
cases run in child processes."""
import os
import subprocess
import sys

import pytest
import torch

from test_gpu_cache import offsets
from test_gpu_cache_waits import CHILD, LIMIT, ROOT, mp, timed  # noqa: F401
from test_gpu_share import Shared, attend_prefix, check_prefix

pytestmark = pytest.mark.gpu

SHARE = "plan or rotate or test_prefix_attention or serving"
SKIP = "32_bits or first or two_streams or many_slots or most_sequences"


@pytest.mark.skipif(not CHILD, reason="in the child process")
@pytest.mark.parametrize("hq,hk,d,page,seqs,own,prefix", [
    (8, 2, 128, 16, 3, 900, 2000),        # all rows few
    (8, 2, 64, 0, 3, 900, 2000),
    (32, 8, 128, 64, 20, 600, 60000),     # own slots beside prefixes in slices
    (32, 8, 64, 16, 20, 600, 60000),
])
def test_child_few_rows(mp, monkeypatch, hq, hk, d, page, seqs, own, prefix):  # noqa: F811
    c = Shared(mp, "bf16", hq, hk, d, page, [own] * seqs, [seqs], [prefix])
    cu, cu_t = offsets([1] * seqs)
    q = c.randn(seqs, hq, d, by=1.5)
    attend_prefix(mp, c, q, cu, cu_t, 1)
    monkeypatch.setenv("MP_FAULT_INJECT", "prefix_few_wait")
    _, s = timed(lambda: attend_prefix(mp, c, q, cu, cu_t, 1))
    assert c.status.item() == mp.MP_STATUS_WAIT_TIMEOUT and LIMIT <= s < 6 * LIMIT
    monkeypatch.delenv("MP_FAULT_INJECT")
    c.status.zero_()
    for _ in range(3):
        (out, lse), s = timed(lambda: attend_prefix(mp, c, q, cu, cu_t, 1))
        assert c.status.item() == 0 and s < LIMIT / 4
        check_prefix(c, "bf16", q, cu, out, lse)


def child(path, select):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__._builder().build(check=True)
    r = subprocess.run([sys.executable, "-m", "pytest", path, "-m", "gpu", "-q", "-x", "-p", "no:cacheprovider", "-k", select], cwd=ROOT,
                       env=dict(os.environ, MP_BOUNDS_CHECK="1"), capture_output=True, text=True, timeout=900)
    assert r.returncode == 0 and " passed" in r.stdout, (r.stdout[-3000:], r.stderr[-2000:])
    return r.stdout


@pytest.mark.skipif(CHILD, reason="the parent process")
def test_waits_of_few_rows_run_out():
    assert "4 passed" in child(__file__, "child_few_rows")


@pytest.mark.skipif(CHILD, reason="the parent process")
def test_plan_prefixes_and_rotation_on_the_bounds_checking_build():
    child(os.path.join(ROOT, "tests", "test_gpu_share.py"), f"({SHARE}) and not ({SKIP})")
