"""Host side of the attention over shared prefixes: index arithmetic over numbers that no kernel wrote, arguments of the
older calls."""
import os
import shutil
import subprocess

import pytest

from test_cache_cpu import ROOT

CSRC = os.path.join(ROOT, "lsh_sampled_sparse_centered_gb300", "csrc")


def run_host(name, tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("no nvcc")
    exe = str(tmp_path / name)
    subprocess.run([nvcc, "-std=c++17", "-O1", "-gencode", "arch=compute_103a,code=sm_103a", "-I", os.path.join(ROOT, "include"), "-I", CSRC,
                    os.path.join(ROOT, "tests", name + ".cu"), "-o", exe], check=True)
    return subprocess.run([exe], capture_output=True, text=True, timeout=300)


def test_the_join_stays_inside_the_sums_whatever_its_numbers_are(tmp_path):
    """A wait that ran out leaves numbers of pieces unwritten; the join runs behind it."""
    r = run_host("row_sums_host", tmp_path)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout


def test_the_older_calls_take_no_arguments_of_the_prefixes(tmp_path):
    r = run_host("call_sizes_host", tmp_path)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout
