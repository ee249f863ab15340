"""What the hybrid's entry points refuse: every check runs on the host before
the first HIP call, so the pointers here are never dereferenced and no GPU is
needed.  Then the compiler's resource report of the kernels."""
import csv
import ctypes
import glob
import os
import re

import pytest
import torch

import mamba_selective_scan_04_amd as m
from mamba_selective_scan_04_amd import hybrid

NULL, DTYPE, SHAPE, ALIGN, WORKSPACE, ALIAS = -1, -3, -2, -4, -5, -7
GAP = 1 << 32
FAKE = {n: (i + 1) * GAP for i, n in enumerate(
    "q k v g beta lens h_init o h_final h_chunks ws dout dh_final dq dk dv dg dbeta dh_init kc ks vc vs table ctx".split())}
P = ctypes.c_void_p


def ptr(over, *names):
    return [P(over.get(n, FAKE[n])) for n in names]


def delta(batch=2, hk=2, hv=4, dk=64, dv=64, dtype=1):
    return m.DeltaShape(batch, hk, hv, dk, dv, dtype)


def scan(s=None, T=100, ws_bytes=1 << 31, **over):
    s = delta() if s is None else s
    a = ptr(over, "q", "k", "v", "g", "beta")
    b = ptr(over, "lens", "h_init", "o", "h_final", "h_chunks", "ws")
    return m.load().bdssm_delta_scan(ctypes.byref(s) if s else None, T, *a, 1.0, *b, ws_bytes, None)


def scan_bwd(s=None, T=100, ws_bytes=1 << 31, **over):
    s = delta() if s is None else s
    a = ptr(over, "q", "k", "v", "g", "beta")
    b = ptr(over, "lens", "h_chunks", "dout", "dh_final", "dq", "dk", "dv", "dg", "dbeta", "dh_init", "ws")
    return m.load().bdssm_delta_scan_bwd(ctypes.byref(s), T, *a, 1.0, *b, ws_bytes, None)


def step(s=None, T=4, **over):
    s = delta() if s is None else s
    a = ptr(over, "h_init", "q", "k", "v", "g", "beta")
    return m.load().bdssm_delta_step(ctypes.byref(s), T, *a, 1.0, *ptr(over, "lens", "o", "h_final"), None)


def kv(batch=2, hq=4, hkv=2, d=64, page=16, n_pages=9, max_pages=4, dtype=1, code=0):
    return m.KvShape(batch, hq, hkv, d, page, n_pages, max_pages, dtype, code)


def commit(s=None, T=32, **over):
    s = kv() if s is None else s
    return m.load().bdssm_kv_commit(ctypes.byref(s), T, *ptr(over, "k", "v", "table", "ctx", "lens", "kc", "ks", "vc", "vs"), None)


def attn(s=None, L=4, Lq=4, ws_bytes=1 << 31, **over):
    s = kv() if s is None else s
    a = ptr(over, "q", "k", "v", "kc", "ks", "vc", "vs", "table", "ctx", "lens")
    return m.load().bdssm_kv_attn_step(ctypes.byref(s), L, Lq, *a, 0, 1.0, *ptr(over, "o", "ws"), ws_bytes, None)


BAD_DELTA = [(dict(dtype=2), DTYPE), (dict(batch=-1), SHAPE), (dict(batch=65536), SHAPE), (dict(hk=0), SHAPE), (dict(hv=0), SHAPE),
             (dict(hv=5), SHAPE), (dict(hk=4, hv=2), SHAPE), (dict(dk=32), SHAPE), (dict(dv=96), SHAPE), (dict(dk=256), SHAPE),
             (dict(batch=65535, hk=1, hv=65535), SHAPE)]


@pytest.mark.parametrize("bad,rc", BAD_DELTA)
def test_delta_shapes(bad, rc):
    s = delta(**bad)
    assert scan(s) == scan_bwd(s) == step(s) == rc
    for bwd in (0, 1):
        assert m.load().bdssm_delta_workspace_bytes(ctypes.byref(s), 100, bwd) == ctypes.c_size_t(-1).value
    with pytest.raises(ValueError):
        m.delta_workspace_bytes(s, 100)


@pytest.mark.parametrize("T", [-1, 1 << 29, 1 << 40, (1 << 63) - 1])
def test_delta_lengths(T):
    assert scan(T=T) == scan_bwd(T=T) == step(T=T) == SHAPE


def test_delta_null():
    assert m.load().bdssm_delta_scan(None, 1, *[None] * 5, 1.0, *[None] * 6, 0, None) == NULL
    for n in ("k", "v", "g", "beta", "q"):
        assert scan(**{n: None}) == NULL, n
        assert step(**{n: None}) == NULL, n
    for n in ("q", "k", "v", "g", "beta", "h_chunks", "dout", "dq", "dk", "dv", "dg", "dbeta"):
        assert scan_bwd(**{n: None}) == NULL, n


@pytest.mark.parametrize("call,names", [
    (scan, "q k v g beta lens h_init o h_final h_chunks ws"),
    (scan_bwd, "q k v g beta lens h_chunks dout dh_final dq dk dv dg dbeta dh_init ws"),
    (step, "h_init q k v g beta lens o h_final"),
    (commit, "k v table ctx lens kc ks vc vs"),
    (attn, "q k v kc ks vc vs table ctx lens o ws")])
def test_alignment(call, names):
    for n in names.split():
        assert call(**{n: FAKE[n] + 8}) == ALIGN, n


@pytest.mark.parametrize("call,ins,outs", [
    (scan, "q k v g beta lens h_init", "o h_final h_chunks"),
    (scan_bwd, "q k v g beta lens h_chunks dout dh_final", "dq dk dv dg dbeta dh_init"),
    (step, "q k v g beta lens", "o h_final"),
    (commit, "k v table ctx lens", "kc ks vc vs"),
    (attn, "q k v kc ks vc vs table ctx lens", "o")])
def test_overlaps(call, ins, outs):
    """An output on an input or on another output, whole or by its last bytes; h_final on h_init is in place."""
    outs = outs.split()
    for o in outs:
        for n in ins.split() + [x for x in outs if x != o]:
            if (n, o) == ("h_init", "h_final"):
                continue
            assert call(**{o: FAKE[n]}) == ALIAS, (n, o)
            if n not in ("lens", "ctx"):
                assert call(**{o: FAKE[n] + 16}) == ALIAS, (n, o)
    if call is scan:
        assert scan(h_final=FAKE["h_init"] + 16) == ALIAS
        assert scan(ws=FAKE["k"]) == ALIAS
    if call is scan_bwd:
        assert scan_bwd(ws=FAKE["h_chunks"]) == ALIAS


def test_workspaces():
    for bwd, call in ((0, scan), (1, scan_bwd)):
        n = m.delta_workspace_bytes(delta(), 100, bool(bwd))
        assert n > 0
        assert call(ws_bytes=n - 1) == WORKSPACE and call(ws=None) == WORKSPACE
    s = kv(max_pages=4000)
    n = m.load().bdssm_kv_workspace_bytes(ctypes.byref(s), 4)
    assert n > 0
    assert attn(s, ws_bytes=n - 1) == WORKSPACE and attn(s, ws=None) == WORKSPACE


def test_nothing_to_do():
    """Empty calls return without a launch (or a look at their pointers)."""
    none = dict.fromkeys(FAKE, None)
    assert scan(delta(batch=0), **none) == scan_bwd(delta(batch=0), **none) == step(delta(batch=0), **none) == 0
    assert scan(o=None, h_final=None, h_chunks=None) == 0 and step(o=None, h_final=None) == 0
    assert commit(kv(batch=0), **none) == commit(T=15, **none) == commit(kv(n_pages=0), **none) == commit(kv(max_pages=0), **none) == 0
    assert attn(kv(batch=0), **none) == attn(Lq=0, **none) == 0


BAD_KV = [(dict(dtype=2), DTYPE), (dict(code=2), DTYPE), (dict(code=-1), DTYPE), (dict(batch=-1), SHAPE), (dict(batch=32768), SHAPE),
          (dict(hq=0), SHAPE), (dict(hkv=0), SHAPE), (dict(hq=5), SHAPE), (dict(hq=2, hkv=4), SHAPE), (dict(d=32), SHAPE),
          (dict(d=96), SHAPE), (dict(page=8), SHAPE), (dict(page=48), SHAPE), (dict(page=256), SHAPE), (dict(n_pages=-1), SHAPE),
          (dict(max_pages=-1), SHAPE), (dict(max_pages=1 << 28), SHAPE), (dict(n_pages=1 << 31), SHAPE),
          (dict(n_pages=(1 << 31) - 1, hkv=4096, hq=4096), SHAPE)]


@pytest.mark.parametrize("bad,rc", BAD_KV)
def test_kv_shapes(bad, rc):
    s = kv(**bad)
    assert commit(s) == attn(s) == rc
    assert m.load().bdssm_kv_workspace_bytes(ctypes.byref(s), 4) == ctypes.c_size_t(-1).value


def test_kv_lengths_and_null():
    assert commit(T=-1) == SHAPE and attn(L=-1) == attn(L=4, Lq=5) == attn(L=4, Lq=-1) == SHAPE
    assert commit(T=1 << 31) == attn(L=1 << 40, Lq=1) == SHAPE
    assert commit(kv(batch=1024), T=1 << 20) == SHAPE                  # more workgroups than a launch counts
    assert attn(kv(batch=4096, hkv=4096, hq=4096), L=4, Lq=4) == SHAPE
    for n in ("k", "v", "table", "ctx", "kc", "ks", "vc", "vs"):
        assert commit(**{n: None}) == NULL, n
        assert attn(**{n: None}) == NULL, n
    assert attn(q=None) == attn(o=None) == NULL
    assert m.load().bdssm_kv_commit(None, 1, *[None] * 10) == NULL
    assert m.load().bdssm_kv_workspace_bytes(None, 1) == ctypes.c_size_t(-1).value


def test_python_checks():
    z = torch.zeros
    k, v, g = z(1, 4, 1, 64), z(1, 4, 1, 64), z(1, 4, 1)
    for call in (lambda: m.delta_scan(k, k, v, g, g), lambda: m.delta_step(None, k, k, v, g, g),
                 lambda: m.delta_scan_bwd(k, k, v, g, g, k, v)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(ValueError):
        m.delta_scan(k, k[0], v, g, g)
    with pytest.raises(ValueError):
        m.delta_scan(k, None, v, g, g)
    with pytest.raises(ValueError, match="q is needed"):
        m.delta_scan_bwd(None, k, v, g, g, k, v)
    with pytest.raises(TypeError):
        m.kv_cache(1, 1, 64, code=torch.float16, device="cpu")
    c = m.kv_cache(3, 2, 64, 16, torch.int8, device="cpu")
    assert c.k.shape == (3, 2, 16, 64) and c.v.shape == (3, 2, 64, 16) and c.k_scale.shape == c.v_scale.shape == (3, 2)
    assert m.kv_cache(3, 2, 64, device="cpu").k.dtype == torch.float8_e4m3fn
    table, n = z(1, 2, dtype=torch.int32), z(1, dtype=torch.int32)
    x = z(1, 16, 2, 64)
    with pytest.raises(ValueError, match="GPU"):
        m.kv_commit(c, x, x, table, n)
    with pytest.raises(ValueError, match="KvCache"):
        m.kv_commit(tuple(c), x, x, table, n)
    with pytest.raises(TypeError):
        m.kv_commit(c._replace(k=c.k.float()), x, x, table, n)
    with pytest.raises(ValueError, match="page_table"):
        m.kv_commit(c, x, x, n, n)
    with pytest.raises(ValueError):
        m.kv_attn_step(c, x[0], x, x, table, n)


def test_other_devices_are_refused(monkeypatch):
    class On:
        def __init__(self, i):
            self.i = i

        def get_device(self):
            return self.i

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 40 + i)
    assert hybrid._stream(0, On(0), None, On(0)) == 40
    with pytest.raises(ValueError, match="current device"):
        hybrid._stream(1, On(1))
    with pytest.raises(ValueError, match="all tensors"):
        hybrid._stream(0, On(0), On(1))


HERE = os.path.dirname(os.path.abspath(__file__))
ROWS = []
for path in glob.glob(os.path.join(os.path.dirname(HERE), "mamba_selective_scan_04_amd", "_build", "launch_*.resources.tsv")):
    with open(path) as f:
        ROWS += list(csv.DictReader(f, delimiter="\t"))


@pytest.mark.skipif(not ROWS, reason="no resource report (run the build first)")
@pytest.mark.parametrize("kernel,count", [("delta_prep_kernelIt", 4), ("delta_chain_kernelIt", 8), ("delta_adjoint_kernelIt", 6),
                                          ("delta_grad_kernelIt", 8), ("delta_step_kernelI[tf]", 4), ("delta_block_kernel", 2), ("delta_join_kernel", 4),
                                          ("kv_commit_kernelI[tf]", 40), ("kv_attn_kernelI[tf]", 14), ("kv_join_kernel", 4)])
def test_kernels_do_not_spill(kernel, count):
    got = [r for r in ROWS if re.search(kernel, r["kernel"])]
    assert len(got) == count, [r["kernel"] for r in got]
    assert all(int(r["vgpr_spill"] or 0) == 0 for r in got), [(r["kernel"], r["vgpr_spill"]) for r in got]
