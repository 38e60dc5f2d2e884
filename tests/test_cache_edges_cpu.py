"""Edges of the cache operators that need no GPU: index arithmetic on the host, refusals that
come after every other check, workspace sizes, the binding's build."""
import ctypes
import os
import shutil
import subprocess
import sys

import pytest

from test_cache_cpu import FAKE, ROOT, attend, cfg_of, evict


@pytest.fixture(scope="module")
def mp():
    import __graft_entry__
    __graft_entry__.build()
    import lsh_sampled_sparse_centered_gb300 as m
    return m


def test_rows_keep_their_slots_whatever_is_cut(mp, tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("no nvcc")
    exe = str(tmp_path / "cache_slots_host")
    subprocess.run([nvcc, "-std=c++17", "-O1", "-gencode", "arch=compute_103a,code=sm_103a", "-I", os.path.join(ROOT, "include"), "-I",
                    os.path.join(os.path.dirname(mp.__file__), "csrc"), os.path.join(ROOT, "tests", "cache_slots_host.cu"), "-o", exe],
                   check=True)
    out = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert out.returncode == 0 and out.stdout.strip() == "ok", out.stdout


# ---- eviction: buffers that are read and written ----

MB = 1 << 20
APART = dict(keys=16 * MB, values=64 * MB, table=112 * MB, kv=113 * MB, scores=114 * MB, dkeys=128 * MB, dvalues=192 * MB, dtable=240 * MB,
             dscores=241 * MB, dlen=242 * MB, kept=243 * MB, ws=244 * MB)


def evict_at(mp, cfg, dst, **kw):
    return evict(mp, cfg, dst, **{**APART, **kw})


def test_evict_refuses_to_overwrite_what_it_reads(mp):
    """scores are read while dst_scores are written, in no order; the same for the others."""
    c = cfg_of(mp)  # scores: 2 sequences x 2 heads x 512 slots of 4 bytes, kept: 2 x 2 x 100
    for bad in (dict(dscores=APART["scores"]), dict(dscores=APART["scores"] + 8188), dict(dscores=APART["scores"] - 8188),
                dict(kept=APART["scores"] + 4), dict(kept=None, ws=APART["scores"] + 4096), dict(dlen=APART["scores"] + 4),
                dict(dlen=APART["kv"] + 4), dict(dlen=APART["kv"] - 4), dict(dscores=APART["kv"]), dict(kept=APART["table"]),
                dict(dscores=APART["dtable"])):
        assert evict_at(mp, c, c, **bad) == mp.MP_ERR_INVALID_ARG, bad
    # a dense cache into itself: the pages that it reads are the ones that it writes
    d = cfg_of(mp, page_size=512, n_pages=2, max_pages=1)
    dense = dict(table=None, dtable=None)
    size = 2 * 2 * 512 * 128 * 2
    for bad in (dict(dkeys=APART["keys"]), dict(dvalues=APART["values"]), dict(dkeys=APART["values"]), dict(dkeys=APART["keys"] + size - 16),
                dict(dvalues=APART["keys"] - size + 16)):
        assert evict_at(mp, d, d, **dense, **bad) == mp.MP_ERR_INVALID_ARG, bad
    # and what is allowed passes every check up to the launch (an injected error stands before the
    # overlaps, the device's refusal behind them)
    import torch
    if torch.cuda.is_available():
        return
    for good in (dict(), dict(dlen=APART["kv"]), dict(dscores=APART["scores"] + 8192), dict(kept=None), dict(dscores=None),
                 dict(dkeys=APART["keys"], dvalues=APART["values"])):  # free pages of the same pool
        assert evict_at(mp, c, c, **good) == mp.MP_ERR_CUDA, good
    for good in (dict(), dict(dkeys=APART["keys"] + size), dict(dlen=APART["kv"])):
        assert evict_at(mp, d, d, **dense, **good) == mp.MP_ERR_CUDA, good
