"""Host side of the planning of a step, the attention over shared prefixes and the rotation of cached keys:
refusals before any launch, workspace sizes, and the index arithmetic of groups run on the host."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

from test_cache_cpu import FAKE, ROOT, cfg_of

MB = 1 << 20
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def mp():
    import __graft_entry__
    __graft_entry__.build()
    import lsh_sampled_sparse_centered_gb300 as m
    return m


# ---- planning ----

PLAN = dict(change=1 * MB, base=2 * MB, kv=3 * MB, n_free=4 * MB, max_rows=100, table=5 * MB, free=6 * MB, new_len=7 * MB, new_free=8 * MB,
            cu=9 * MB, positions=10 * MB, slots=11 * MB, seq=12 * MB, status=13 * MB)


def plan(mp, cfg, **kw):
    a = {**PLAN, **kw}
    return mp.call_raw("mp_cache_plan", cfg, *(a[k] for k in PLAN), None)


@pytest.mark.parametrize("change", [
    dict(change=None), dict(kv=None), dict(n_free=None), dict(free=None), dict(new_len=None), dict(new_free=None), dict(cu=None), dict(max_rows=-1),
    dict(table=None), dict(change=MB + 2), dict(positions=MB * 10 + 1), dict(status=MB * 13 + 2),
    # what is written overlaps what is read, or what else is written; the two that may be updated in place only as a whole
    dict(new_len=PLAN["change"]), dict(new_len=PLAN["kv"] + 4), dict(cu=PLAN["kv"]), dict(positions=PLAN["base"]), dict(new_free=PLAN["n_free"] - 4, n_free=4 * MB + 4, kv=4 * MB - 4),
    dict(slots=PLAN["positions"]), dict(seq=PLAN["slots"] + 396), dict(cu=PLAN["new_len"] - 8), dict(free=PLAN["table"]), dict(table=PLAN["kv"] - 60),
    dict(status=PLAN["cu"] + 8)])
def test_plan_refusals(mp, change):
    assert plan(mp, cfg_of(mp), **change) == mp.MP_ERR_INVALID_ARG


def test_plan_limits(mp, monkeypatch):
    assert plan(mp, cfg_of(mp, batch=mp.MP_PLAN_SEQUENCES + 1)) == mp.MP_ERR_UNSUPPORTED
    assert plan(mp, cfg_of(mp), max_rows=(1 << 30) + 1) == mp.MP_ERR_UNSUPPORTED
    assert plan(mp, cfg_of(mp, page_size=24)) == mp.MP_ERR_UNSUPPORTED
    assert plan(mp, cfg_of(mp, batch=0)) == mp.MP_ERR_INVALID_ARG
    dense = cfg_of(mp, page_size=100, n_pages=2, max_pages=1)
    assert plan(mp, cfg_of(mp), table=None) == mp.MP_ERR_INVALID_ARG        # more than one page without a table
    monkeypatch.setenv("MP_FAULT_INJECT", "plan")
    for c, kw in ((dense, dict(table=None, n_free=None, free=None, new_free=None)), (cfg_of(mp), dict(base=None, positions=None, slots=None, seq=None)),
                  (cfg_of(mp), dict(new_len=PLAN["kv"], new_free=PLAN["n_free"])), (cfg_of(mp, batch=mp.MP_PLAN_SEQUENCES), {})):
        assert plan(mp, c, **kw) == mp.MP_ERR_INJECTED, kw


# ---- prefixes ----

PREFIX = dict(q=FAKE, cu=FAKE, kv=FAKE, total=6, max_q=4, max_kv=512, keys=FAKE, values=FAKE, table=FAKE, cu_group=FAKE, lens=FAKE, max_group=6,
              max_prefix=512, pkeys=FAKE, pvalues=FAKE, ptable=FAKE, out=FAKE, lse=FAKE, ws=FAKE, wsn=1 << 40, status=FAKE)


def prefix(mp, cfg, pre, **kw):
    a = {**PREFIX, **kw}
    return mp.call_raw("mp_prefix_attention", cfg, pre, *(a[k] for k in PREFIX), None)


@pytest.mark.parametrize("change", [
    dict(q=None), dict(cu=None), dict(kv=None), dict(keys=None), dict(values=None), dict(cu_group=None), dict(lens=None), dict(pkeys=None),
    dict(pvalues=None), dict(out=None), dict(total=-1), dict(max_q=0), dict(max_kv=0), dict(max_group=0), dict(max_prefix=0), dict(table=None),
    dict(ptable=None), dict(q=FAKE + 8), dict(pkeys=FAKE + 4), dict(out=FAKE + 2), dict(lse=FAKE + 2), dict(cu_group=FAKE + 1), dict(lens=FAKE + 3),
    dict(ptable=FAKE + 2), dict(ws=None), dict(ws=FAKE + 128)])
def test_prefix_refusals(mp, change):
    assert prefix(mp, cfg_of(mp), cfg_of(mp), **change) == mp.MP_ERR_INVALID_ARG


def test_prefix_limits(mp, monkeypatch):
    c = cfg_of(mp)
    for other in (dict(kv_heads=1), dict(q_heads=4), dict(head_dim=64), dict(dtype="f32"), dict(batch=0)):
        assert prefix(mp, c, cfg_of(mp, **other)) == mp.MP_ERR_INVALID_ARG, other
    assert prefix(mp, c, c, max_kv=513) == prefix(mp, c, c, max_prefix=513) == mp.MP_ERR_CAPACITY
    assert prefix(mp, c, c, max_q=1 << 30) == prefix(mp, c, c, max_group=1 << 30) == mp.MP_ERR_UNSUPPORTED
    assert prefix(mp, c, cfg_of(mp, page_size=72)) == mp.MP_ERR_UNSUPPORTED
    assert prefix(mp, c, c, total=0) == prefix(mp, c, c, total=0, q=None, out=None, ws=None) == mp.MP_OK
    assert mp.mp_prefix_workspace_bytes(c, c, 0, 4, 512, 6, 512) == 0
    monkeypatch.setenv("MP_FAULT_INJECT", "prefix")
    for kw in ({}, dict(dtype="f32"), dict(head_dim=64), dict(q_heads=64)):
        d = cfg_of(mp, **kw)
        assert prefix(mp, d, d, wsn=mp.mp_prefix_workspace_bytes(d, d, 6, 4, 512, 6, 512)) == mp.MP_ERR_INJECTED
        assert prefix(mp, d, d, wsn=0) == mp.MP_ERR_SCRATCH
    e = cfg_of(mp, batch=9, page_size=16, n_pages=900, max_pages=40)  # another number of groups, other pages
    assert prefix(mp, c, e) == mp.MP_ERR_INJECTED


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_prefix_workspace_for_the_largest_limits_serves_all_smaller_ones(mp, monkeypatch, dtype):
    import random
    monkeypatch.setenv("MP_FAULT_INJECT", "prefix")  # answered after the workspace has been looked at
    rng = random.Random(11)
    log = lambda lo, hi: min(hi, max(lo, round(lo * (hi / lo) ** rng.random())))
    for _ in range(300):
        hk, group = rng.choice((1, 2, 4, 8, 40)), rng.choice((1, 3, 4, 8, 12, 16, 100, 300))
        heads = dict(kv_heads=hk, q_heads=hk * group, head_dim=rng.choice((64, 128)), dtype=dtype, n_pages=64, max_pages=8)
        c, p = cfg_of(mp, batch=log(1, 200), page_size=16 * log(1, 200), **heads), cfg_of(mp, batch=log(1, 20), page_size=16 * log(1, 4096), **heads)
        limits = (log(1, 3000), log(1, 3000), log(1, 8 * c.page_size), log(1, 3000), log(1, 8 * p.page_size))
        size = mp.mp_prefix_workspace_bytes(c, p, *limits)
        for i in range(30):
            t, m, n, g, l = (log(1, x) for x in limits) if i else limits
            assert mp.mp_prefix_workspace_bytes(c, p, t, m, n, g, l) <= size
            assert prefix(mp, c, p, total=t, max_q=m, max_kv=n, max_group=g, max_prefix=l, wsn=size) == mp.MP_ERR_INJECTED, (t, m, n, g, l)


# ---- rotation ----

ROTATE = dict(rot=dict(rot_dim=128), keys=FAKE, table=FAKE, kv=FAKE, max_kv=512, f0=FAKE, f1=FAKE, p0=FAKE, p1=FAKE, heads=2, cols=512, scale=1.0,
              status=FAKE)


def rotate(mp, cfg, **kw):
    a = {**ROTATE, **kw}
    rot = mp.make_rotary(**a["rot"]) if isinstance(a["rot"], dict) else a["rot"]
    return mp.call_raw("mp_cache_rotate", cfg, rot, *(a[k] for k in list(ROTATE)[1:]), None)


@pytest.mark.parametrize("change", [
    dict(rot=None), dict(rot=dict(rot_dim=-2)), dict(rot=dict(rot_dim=130)), dict(rot=dict(rot_dim=7)), dict(keys=None), dict(kv=None), dict(f0=None),
    dict(max_kv=0), dict(heads=3), dict(heads=0), dict(cols=511), dict(scale=NAN), dict(scale=INF), dict(scale=-INF), dict(keys=FAKE + 8),
    dict(f0=FAKE + 4), dict(f1=FAKE + 4), dict(p0=FAKE + 2), dict(p1=FAKE + 1), dict(table=None), dict(kv=FAKE + 2), dict(status=FAKE + 3)])
def test_rotate_refusals(mp, change):
    assert rotate(mp, cfg_of(mp), **change) == mp.MP_ERR_INVALID_ARG


def test_rotate_limits(mp, monkeypatch):
    c = cfg_of(mp)
    assert rotate(mp, c, rot=dict(rot_dim=24)) == mp.MP_ERR_UNSUPPORTED  # halves that split a vector
    assert rotate(mp, cfg_of(mp, page_size=24)) == mp.MP_ERR_UNSUPPORTED
    assert rotate(mp, c, max_kv=513) == mp.MP_ERR_CAPACITY
    assert rotate(mp, c, rot=dict(rot_dim=0), f0=None) == mp.MP_OK
    monkeypatch.setenv("MP_FAULT_INJECT", "rotate")
    for kw in (dict(p0=None, p1=None, heads=77, cols=-1), dict(heads=1), dict(f1=None), dict(rot=dict(rot_dim=24, interleaved=True)), dict(scale=-0.5)):
        assert rotate(mp, c, **kw) == mp.MP_ERR_INJECTED, kw


def test_fault_injection_on_the_host(mp, monkeypatch):
    c = cfg_of(mp)
    for what, call in (("plan", lambda: plan(mp, c)), ("prefix", lambda: prefix(mp, c, c)), ("rotate", lambda: rotate(mp, c))):
        for value in (what, "all"):
            monkeypatch.setenv("MP_FAULT_INJECT", value)
            assert call() == mp.MP_ERR_INJECTED, (what, value)


def test_binding_refuses_host_tensors_and_other_values(mp):
    host, ints = torch.zeros(4, 8, 128, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)
    c = cfg_of(mp)
    with pytest.raises(ValueError):
        mp.mp_cache_plan(c, ints, None, ints, ints, 4, ints, ints, ints, ints, ints)
    with pytest.raises(ValueError):
        mp.mp_prefix_attention(c, c, host, ints, ints, 1, 1, host, host, None, ints, ints, 1, 1, host, host, None, host)
    with pytest.raises(ValueError):
        mp.mp_cache_rotate(c, mp.make_rotary(rot_dim=64), host, None, ints, 1, None)


def test_group_arithmetic_on_the_host(mp, tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("no nvcc")
    exe = str(tmp_path / "group_index_host")
    subprocess.run([nvcc, "-std=c++17", "-O1", "-gencode", "arch=compute_103a,code=sm_103a", "-I", os.path.join(ROOT, "include"), "-I",
                    os.path.join(os.path.dirname(mp.__file__), "csrc"), os.path.join(ROOT, "tests", "group_index_host.cu"), "-o", exe],
                   check=True)
    out = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert out.returncode == 0 and out.stdout.strip() == "ok", out.stdout


def test_a_c_caller(mp, tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    libdir, exe = os.path.dirname(mp.LIB_PATH), str(tmp_path / "share_abi_from_c")
    subprocess.run([cc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"),
                    os.path.join(ROOT, "tests", "share_abi_from_c.c"), "-L", libdir, "-lmagicpig", "-Wl,-rpath," + libdir, "-o", exe], check=True)
    env = {k: v for k, v in os.environ.items() if k != "MP_FAULT_INJECT"}
    got = dict(line.split(" ", 1) for line in subprocess.run([exe], check=True, capture_output=True, text=True, env=env).stdout.strip().splitlines())
    c = cfg_of(mp, page_size=4096)
    want = dict(plan_overlap=mp.MP_ERR_INVALID_ARG, plan_sequences=mp.MP_PLAN_SEQUENCES, prefix_bytes_rc=mp.MP_OK,
                prefix_bytes=mp.mp_prefix_workspace_bytes(c, c, 2, 1, 5000, 2, 9000), prefix_scratch=mp.MP_ERR_SCRATCH,
                rotate_capacity=mp.MP_ERR_CAPACITY, rotate_nothing=mp.MP_OK, bit=mp.MP_STATUS_NO_ROOM)
    assert got == {k: str(v) for k, v in want.items()}
