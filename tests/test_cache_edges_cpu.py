"""Edges of the cache operators that need no GPU: index arithmetic on the host, refusals that
come after every other check, workspace sizes, the binding's build."""
import ctypes
import os
import shutil
import subprocess

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


# ---- workspaces of the attention ----

def needed(mp, c, total, max_q, max_kv, size):
    """What a call with a workspace of `size` bytes is answered, short of a launch."""
    return attend(mp, c, table=FAKE if c.max_pages > 1 else None, total=total, max_q=max_q, max_kv=max_kv, wsn=size)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_workspace_for_the_largest_limits_serves_all_smaller_ones(mp, monkeypatch, dtype):
    import random
    monkeypatch.setenv("MP_FAULT_INJECT", "chunk")  # answered after the workspace has been looked at
    rng = random.Random(7)
    log = lambda lo, hi: min(hi, max(lo, round(lo * (hi / lo) ** rng.random())))
    dips = 0
    for _ in range(400):
        hk, group = rng.choice((1, 2, 4, 8, 40)), rng.choice((1, 3, 4, 8, 12, 16, 100, 300))
        ps = 16 * log(1, 4096)
        c = cfg_of(mp, batch=log(1, 64), kv_heads=hk, q_heads=hk * group, head_dim=rng.choice((64, 128)), page_size=ps, n_pages=64, max_pages=8,
                   dtype=dtype)
        max_kv, max_q, total = log(1, 8 * ps), log(1, 3000), log(1, 5000)
        size = mp.mp_chunk_workspace_bytes(c, total, max_q, max_kv)
        for _ in range(30):
            t, q, n = log(1, total), log(1, max_q), log(1, max_kv)
            own = mp.mp_chunk_workspace_bytes(c, t, q, n)
            assert own <= size
            assert needed(mp, c, t, q, n, size) == mp.MP_ERR_INJECTED, (t, q, n)
            dips += size > 0 and needed(mp, c, total, max_q, max_kv, 0) == mp.MP_ERR_INJECTED and needed(mp, c, t, q, n, 0) == mp.MP_ERR_SCRATCH
        for t, q, n in ((total, 1, max_kv), (total, max_q, max(1, max_kv // 8)), (min(total, 3), 1, min(max_kv, 300)), (total, 1, 1)):
            assert needed(mp, c, t, q, n, size) == mp.MP_ERR_INJECTED, (t, q, n)
    assert dips  # calls that need a workspace below a call that needs none


def test_a_workspace_that_is_too_small_or_astray_is_refused(mp, monkeypatch):
    c = cfg_of(mp, page_size=4096)  # 5000 slots in 40 slices of a token each of 8 heads, for 2 tokens
    need = 40 * 2 * 8 * 128 * 4 + 40 * 2 * 8 * 8
    monkeypatch.setenv("MP_FAULT_INJECT", "chunk")
    call = lambda **kw: attend(mp, c, total=2, max_q=1, max_kv=5000, **kw)
    assert call(wsn=need) == mp.MP_ERR_INJECTED
    assert call(wsn=need - 1) == mp.MP_ERR_SCRATCH
    assert call(ws=None) == mp.MP_ERR_INVALID_ARG
    assert call(ws=FAKE + 16) == mp.MP_ERR_INVALID_ARG
    # rows of no sequence need no place, however many there are
    assert attend(mp, c, total=2000, max_q=1, max_kv=5000, wsn=need) == mp.MP_ERR_INJECTED
    # fp32 and the large tiles, by the size that the library names
    for kw, limits in ((dict(dtype="f32"), (6, 4, 512)), (dict(), (60, 40, 512))):
        d = cfg_of(mp, **kw)
        size = mp.mp_chunk_workspace_bytes(d, *limits)
        ask = lambda **k: attend(mp, d, total=limits[0], max_q=limits[1], max_kv=limits[2], **k)
        assert size > 0 and ask(wsn=size) == mp.MP_ERR_INJECTED
        assert ask(wsn=0) == mp.MP_ERR_SCRATCH and ask(ws=None) == mp.MP_ERR_INVALID_ARG and ask(ws=FAKE + 128) == mp.MP_ERR_INVALID_ARG


# ---- the binding's build ----

def test_the_python_calls_are_of_one_interpreter_and_pytorch(mp, monkeypatch):
    """The extension uses PyTorch's inline C++: one of another version must not be loaded."""
    import torch
    import __graft_entry__
    b = __graft_entry__._builder()
    root, version = b.installed_torch()
    assert version == str(torch.__version__) and os.path.samefile(root, os.path.dirname(torch.__file__))
    assert os.path.exists(b.calls_path(version)) and mp._cache_calls() is not None
    monkeypatch.setattr(torch, "__version__", "1.0.0+other")
    with pytest.raises(ImportError, match="1.0.0"):
        mp._cache_calls()
    monkeypatch.undo()
    import sysconfig
    real = sysconfig.get_config_var
    monkeypatch.setattr(sysconfig, "get_config_var", lambda n: "cpython-99-none" if n == "SOABI" else real(n))
    with pytest.raises(ImportError, match="cpython-99-none"):
        mp._cache_calls()


def test_the_library_builds_without_pytorch(mp, monkeypatch, capfd):
    """A user of the C library alone needs no PyTorch."""
    import importlib.util
    import __graft_entry__
    b = __graft_entry__._builder()
    real = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else real(name, *a))
    assert b.build() == mp.LIB_PATH
    assert "without the Python calls" in capfd.readouterr().err


def test_a_change_of_the_build_or_the_header_rebuilds_the_python_calls(mp, monkeypatch, tmp_path):
    import __graft_entry__
    b = __graft_entry__._builder()
    out = b.calls_path(b.installed_torch()[1])
    ran = []
    monkeypatch.setattr(b.subprocess, "run", lambda cmd, **kw: ran.append(cmd) or subprocess.CompletedProcess(cmd, 1, "", "stopped"))
    b.build_calls(b._nvcc())
    assert not ran
    real = os.path.getmtime
    for changed in ("build.py", "magicpig.h", "mp_binding.cpp"):
        monkeypatch.setattr(os.path, "getmtime", lambda p: real(out) + 1 if os.path.basename(p) == changed else real(p))
        with pytest.raises(RuntimeError, match="stopped"):
            b.build_calls(b._nvcc())
    assert len(ran) == 3


def test_a_c_caller_of_the_cache_operators(mp, tmp_path):
    """The header's structures, codes and sizes are those of the binding, compiled as C99 without a warning."""
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    libdir, exe = os.path.dirname(mp.LIB_PATH), str(tmp_path / "cache_abi_from_c")
    subprocess.run([cc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"),
                    os.path.join(ROOT, "tests", "cache_abi_from_c.c"), "-L", libdir, "-lmagicpig", "-Wl,-rpath," + libdir, "-o", exe], check=True)
    env = {k: v for k, v in os.environ.items() if k != "MP_FAULT_INJECT"}
    out = subprocess.run([exe], check=True, capture_output=True, text=True, env=env).stdout
    got = dict(line.split(" ", 1) for line in out.strip().splitlines())
    c = cfg_of(mp, page_size=4096)
    want = dict(sizeof_cache_config=ctypes.sizeof(mp.mp_cache_config), offset_dtype=mp.mp_cache_config.dtype.offset,
                sizeof_rotary=ctypes.sizeof(mp.mp_rotary), offset_eps=mp.mp_rotary.eps.offset, check_ok=mp.MP_OK,
                check_null=mp.MP_ERR_INVALID_ARG, chunk_bytes_rc=mp.MP_OK, chunk_bytes=mp.mp_chunk_workspace_bytes(c, 2, 1, 5000),
                evict_bytes_rc=mp.MP_OK, evict_bytes=mp.mp_evict_workspace_bytes(c, 5000, 100), append_rotary=mp.MP_ERR_INVALID_ARG,
                append_empty=mp.MP_OK, attention_scratch=mp.MP_ERR_SCRATCH, weights_capacity=mp.MP_ERR_CAPACITY,
                evict_budget=mp.MP_ERR_INVALID_ARG, bits=f"{mp.MP_STATUS_BAD_PAGE} {mp.MP_STATUS_BAD_LENGTH}")
    assert got == {k: str(v) for k, v in want.items()}
