"""The cache operators' host side: refusals before any launch, workspace sizes, and the
index arithmetic of the kernels run on the host over bad lengths and page numbers."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20  # never dereferenced: validation fails first
NAN = float("nan")


@pytest.fixture(scope="module")
def mp():
    import __graft_entry__
    __graft_entry__.build()
    import lsh_sampled_sparse_centered_gb300 as m
    return m


def cfg_of(mp, **kw):
    base = dict(batch=2, kv_heads=2, q_heads=8, head_dim=128, page_size=64, n_pages=20, max_pages=8, dtype="bf16")
    base.update(kw)
    return mp.make_cache_config(**base)


def test_config_validation(mp):
    assert mp.mp_cache_config_check(cfg_of(mp)) == mp.MP_OK
    for bad in (dict(batch=0), dict(kv_heads=0), dict(q_heads=7), dict(page_size=0), dict(n_pages=0), dict(max_pages=0),
                dict(dtype=5)):
        assert mp.mp_cache_config_check(cfg_of(mp, **bad)) == mp.MP_ERR_INVALID_ARG, bad
    for bad in (dict(head_dim=96), dict(batch=70000), dict(page_size=1 << 20, max_pages=1 << 11),
                dict(page_size=1 << 16, n_pages=1 << 15)):
        assert mp.mp_cache_config_check(cfg_of(mp, **bad)) == mp.MP_ERR_UNSUPPORTED, bad
    c = cfg_of(mp)
    c.reserved[3] = 1
    assert mp.mp_cache_config_check(c) == mp.MP_ERR_INVALID_ARG
    assert mp.call_raw("mp_cache_config_check", None) == mp.MP_ERR_INVALID_ARG


APPEND = dict(rot=dict(rot_dim=128), q=FAKE, qs=8 * 128, k=FAKE, ks=256, v=FAKE, vs=256, qn=FAKE, kn=FAKE, f=FAKE, pos=FAKE, cu=FAKE,
              kv=FAKE, total=5, keys=FAKE, values=FAKE, table=FAKE, out=FAKE, status=FAKE)


def append(mp, cfg, **kw):
    a = dict(APPEND)
    a.update(kw)
    rot = mp.make_rotary(**a["rot"]) if isinstance(a["rot"], dict) else a["rot"]
    return mp.call_raw("mp_cache_append", cfg, rot, a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["qn"], a["kn"], a["f"], a["pos"],
                       a["cu"], a["kv"], a["total"], a["keys"], a["values"], a["table"], a["out"], a["status"], None)


@pytest.mark.parametrize("change", [
    dict(rot=None), dict(rot=dict(rot_dim=-2)), dict(rot=dict(rot_dim=130)), dict(rot=dict(rot_dim=7)), dict(rot=dict(rot_dim=128, eps=-1.0)),
    dict(rot=dict(rot_dim=128, eps=NAN)), dict(q=None), dict(k=None), dict(v=None), dict(f=None), dict(cu=None), dict(kv=None), dict(keys=None),
    dict(values=None), dict(out=None), dict(total=-1), dict(qs=8 * 128 - 8), dict(ks=248), dict(vs=0), dict(qs=8 * 128 + 4), dict(q=FAKE + 2),
    dict(keys=FAKE + 8), dict(f=FAKE + 4), dict(cu=FAKE + 2), dict(status=FAKE + 1), dict(table=None)])
def test_append_refusals(mp, change):
    assert append(mp, cfg_of(mp), **change) == mp.MP_ERR_INVALID_ARG


def test_append_unsupported_and_empty(mp):
    assert append(mp, cfg_of(mp), rot=dict(rot_dim=24)) == mp.MP_ERR_UNSUPPORTED       # halves that split a vector
    assert append(mp, cfg_of(mp, page_size=24)) == mp.MP_ERR_UNSUPPORTED
    assert append(mp, cfg_of(mp), total=0) == mp.MP_OK
    assert append(mp, cfg_of(mp), total=0, q=None, k=None, v=None, out=None) == mp.MP_OK
    assert append(mp, cfg_of(mp, batch=2, n_pages=1, max_pages=1), table=None) == mp.MP_ERR_INVALID_ARG
    assert append(mp, cfg_of(mp), rot=dict(rot_dim=0), f=None, total=0) == mp.MP_OK


def attend(mp, cfg, **kw):
    a = dict(q=FAKE, cu=FAKE, kv=FAKE, total=6, max_q=4, max_kv=512, keys=FAKE, values=FAKE, table=FAKE, out=FAKE, lse=FAKE, ws=FAKE,
             wsn=1 << 30, status=FAKE)
    a.update(kw)
    return mp.call_raw("mp_chunk_attention", cfg, a["q"], a["cu"], a["kv"], a["total"], a["max_q"], a["max_kv"], a["keys"], a["values"],
                       a["table"], a["out"], a["lse"], a["ws"], a["wsn"], a["status"], None)


@pytest.mark.parametrize("change", [
    dict(q=None), dict(cu=None), dict(kv=None), dict(keys=None), dict(values=None), dict(out=None), dict(total=-1), dict(max_q=0), dict(max_kv=0),
    dict(table=None), dict(q=FAKE + 8), dict(keys=FAKE + 4), dict(out=FAKE + 2), dict(lse=FAKE + 2), dict(kv=FAKE + 1)])
def test_attention_refusals(mp, change):
    assert attend(mp, cfg_of(mp), **change) == mp.MP_ERR_INVALID_ARG


def test_attention_limits_and_workspace(mp):
    c = cfg_of(mp)
    assert attend(mp, c, max_kv=513) == mp.MP_ERR_CAPACITY
    assert attend(mp, c, max_q=1 << 30) == mp.MP_ERR_UNSUPPORTED
    assert attend(mp, c, total=1 << 29) == mp.MP_ERR_UNSUPPORTED
    assert attend(mp, cfg_of(mp, page_size=40)) == mp.MP_ERR_UNSUPPORTED
    assert attend(mp, c, total=0) == mp.MP_OK
    need = mp.mp_chunk_workspace_bytes(c, 2, 1, 512)
    if need:
        assert attend(mp, c, total=2, max_q=1, wsn=need - 1) == mp.MP_ERR_SCRATCH
        assert attend(mp, c, total=2, max_q=1, ws=None) == mp.MP_ERR_INVALID_ARG
        assert attend(mp, c, total=2, max_q=1, ws=FAKE + 16) == mp.MP_ERR_INVALID_ARG
    with pytest.raises(mp.MagicPigError) as e:
        mp.mp_chunk_workspace_bytes(c, 2, 1, 513)
    assert e.value.code == mp.MP_ERR_CAPACITY
    # one token over a long cache is split over the SMs; a long chunk over the same cache need not be
    big = cfg_of(mp, batch=1, page_size=65536, n_pages=1, max_pages=1)
    assert mp.mp_chunk_workspace_bytes(big, 1, 1, 65536) > 0
    assert mp.mp_chunk_workspace_bytes(big, 0, 1, 65536) == 0


def weights(mp, cfg, **kw):
    a = dict(q=FAKE, lse=FAKE, cu=FAKE, kv=FAKE, total=6, max_q=4, max_kv=512, keys=FAKE, table=FAKE, scores=FAKE, status=FAKE)
    a.update(kw)
    return mp.call_raw("mp_cache_weights", cfg, a["q"], a["lse"], a["cu"], a["kv"], a["total"], a["max_q"], a["max_kv"], a["keys"],
                       a["table"], a["scores"], a["status"], None)


@pytest.mark.parametrize("change", [
    dict(q=None), dict(lse=None), dict(cu=None), dict(kv=None), dict(keys=None), dict(scores=None), dict(total=-1), dict(max_q=0), dict(max_kv=0),
    dict(table=None), dict(q=FAKE + 8), dict(keys=FAKE + 4), dict(scores=FAKE + 2), dict(lse=FAKE + 2)])
def test_weights_refusals(mp, change):
    assert weights(mp, cfg_of(mp), **change) == mp.MP_ERR_INVALID_ARG
    assert weights(mp, cfg_of(mp), max_kv=513) == mp.MP_ERR_CAPACITY
    assert weights(mp, cfg_of(mp), total=0) == mp.MP_OK


def evict(mp, cfg, dst, **kw):
    a = dict(keys=FAKE, values=FAKE, table=FAKE, kv=FAKE, max_kv=512, scores=FAKE, sink=4, window=16, budget=100, dkeys=FAKE, dvalues=FAKE,
             dtable=FAKE, dscores=FAKE, dlen=FAKE, kept=FAKE, ws=FAKE, wsn=1 << 30, status=FAKE)
    a.update(kw)
    return mp.call_raw("mp_cache_evict", cfg, dst, a["keys"], a["values"], a["table"], a["kv"], a["max_kv"], a["scores"], a["sink"],
                       a["window"], a["budget"], a["dkeys"], a["dvalues"], a["dtable"], a["dscores"], a["dlen"], a["kept"], a["ws"], a["wsn"],
                       a["status"], None)


@pytest.mark.parametrize("change", [
    dict(keys=None), dict(values=None), dict(kv=None), dict(scores=None), dict(dkeys=None), dict(dvalues=None), dict(dlen=None), dict(ws=None),
    dict(budget=0), dict(sink=-1), dict(window=-1), dict(sink=90, window=11), dict(sink=2**31 - 1, window=2**31 - 1), dict(max_kv=0),
    dict(table=None), dict(dtable=None), dict(ws=FAKE + 16), dict(dkeys=FAKE + 8), dict(scores=FAKE + 2), dict(kept=FAKE + 2)])
def test_evict_refusals(mp, change):
    assert evict(mp, cfg_of(mp), cfg_of(mp), **change) == mp.MP_ERR_INVALID_ARG


def test_evict_limits(mp):
    c = cfg_of(mp)
    assert evict(mp, c, cfg_of(mp, max_pages=1)) == mp.MP_ERR_CAPACITY           # 100 slots into one page of 64
    assert evict(mp, c, c, max_kv=513) == mp.MP_ERR_CAPACITY
    assert evict(mp, c, c, wsn=mp.mp_evict_workspace_bytes(c, 512, 100) - 1) == mp.MP_ERR_SCRATCH
    for other in (dict(batch=3), dict(kv_heads=1), dict(q_heads=4), dict(head_dim=64), dict(dtype="f32")):
        assert evict(mp, c, cfg_of(mp, **other)) == mp.MP_ERR_INVALID_ARG, other


def test_fault_injection_on_the_host(mp, monkeypatch):
    c = cfg_of(mp)
    for what, call in (("append", lambda: append(mp, c)), ("chunk", lambda: attend(mp, c)), ("weights", lambda: weights(mp, c)),
                       ("evict", lambda: evict(mp, c, c))):
        for value in (what, "all"):
            monkeypatch.setenv("MP_FAULT_INJECT", value)
            assert call() == mp.MP_ERR_INJECTED, (what, value)


def test_binding_refuses_host_tensors_and_other_values(mp):
    host = torch.zeros(4, 8, 128, dtype=torch.bfloat16)
    c = cfg_of(mp)
    with pytest.raises(ValueError):
        mp.mp_chunk_attention(c, host, None, None, 1, 1, host, host, None, host)
    with pytest.raises(ValueError):
        mp.mp_cache_append(c, mp.make_rotary(rot_dim=64), host, host, host, None, None, None, None, None, None, host, host, None, host)
    with pytest.raises(ValueError):
        mp.mp_cache_weights(c, 12345, None, None, None, 1, 1, host, None, host)
    with pytest.raises(KeyError):
        cfg_of(mp, dtype="fp16")


def test_index_arithmetic_on_the_host(mp, tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("no nvcc")
    exe = str(tmp_path / "cache_index_host")
    subprocess.run([nvcc, "-std=c++17", "-O1", "-gencode", "arch=compute_103a,code=sm_103a", "-I", os.path.join(ROOT, "include"), "-I",
                    os.path.join(os.path.dirname(mp.__file__), "csrc"), os.path.join(ROOT, "tests", "cache_index_host.cu"), "-o", exe],
                   check=True)
    out = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert out.returncode == 0 and out.stdout.strip() == "ok", out.stdout
