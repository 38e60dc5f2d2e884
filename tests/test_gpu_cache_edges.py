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
from test_gpu_cache import DEV, DT, HALF, Cache, attend, make_scores, offsets, pool_rows

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
