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
