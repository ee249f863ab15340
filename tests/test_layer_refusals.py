"""What the entry points around the scans and of the cache's upkeep refuse: every
check runs on the host before the first HIP call, so the pointers here are never
dereferenced and no GPU is needed."""
import ctypes

import pytest
import torch

import mamba_selective_scan_04_amd as m

NULL, SHAPE, DTYPE, ALIGN, WORKSPACE, ALIAS = -1, -2, -3, -4, -5, -7
GAP = 1 << 36
NAMES = ("u w bias lens starts c_init y c_final dy dc_final du dw dbias dc_init ws x res h rstd codes scales dh dx dres "
         "q lse kc ks vc vs k v o table ctx mass out table_out ctx_out mass_out").split()
FAKE = {n: (i + 1) * GAP for i, n in enumerate(NAMES)}
NONE = dict.fromkeys(NAMES)
P = ctypes.c_void_p


def ptr(over, *names):
    return [P(over.get(n, FAKE[n])) for n in names]


def conv(batch=2, ch=64, width=4, ld=None, batch_ld=None, dtype=1, T=10):
    ld = ch if ld is None else ld
    return m.ConvShape(batch, ch, width, ld, T * ld if batch_ld is None else batch_ld, dtype)


def scan(s=None, T=10, **over):
    s = conv() if s is None else s
    return m.load().bdssm_conv_scan(ctypes.byref(s), T, *ptr(over, "u", "w", "bias"), 1, *ptr(over, "lens", "starts", "c_init", "y", "c_final"),
                                    None)


def step(s=None, T=10, **over):
    s = conv() if s is None else s
    return m.load().bdssm_conv_step(ctypes.byref(s), T, *ptr(over, "c_init", "u", "w", "bias"), 1, *ptr(over, "lens", "y", "c_final"), None)


def scan_bwd(s=None, T=10, ld=64, batch_ld=640, ws_bytes=1 << 31, **over):
    s = conv() if s is None else s
    return m.load().bdssm_conv_scan_bwd(ctypes.byref(s), T, *ptr(over, "u", "w", "bias"), 1,
                                        *ptr(over, "lens", "starts", "c_init", "dy", "dc_final", "du"), ld, batch_ld,
                                        *ptr(over, "dw", "dbias", "dc_init", "ws"), ws_bytes, None)


def norm(rows=5, ch=256, dtype=1, res_dtype=0):
    return m.NormShape(rows, ch, dtype, res_dtype)


def rms(s=None, eps=1e-5, **over):
    s = norm() if s is None else s
    return m.load().bdssm_rms_norm(ctypes.byref(s), *ptr(over, "x", "res", "w"), eps, *ptr(over, "y", "h", "rstd"), None)


def rms_codes(s=None, eps=1e-5, code=0, group=0, **over):
    s = norm() if s is None else s
    return m.load().bdssm_rms_norm_codes(ctypes.byref(s), *ptr(over, "x", "res", "w"), eps, code, group, *ptr(over, "codes", "scales", "h"), None)


def rms_bwd(s=None, ws_bytes=1 << 31, **over):
    s = norm() if s is None else s
    return m.load().bdssm_rms_norm_bwd(ctypes.byref(s), *ptr(over, "h", "w", "rstd", "dy", "dh", "dx", "dres", "dw", "ws"), ws_bytes, None)


def kv(batch=2, hq=4, hkv=2, d=64, page=16, n_pages=9, max_pages=4, dtype=1, code=0):
    return m.KvShape(batch, hq, hkv, d, page, n_pages, max_pages, dtype, code)


def attn(s=None, L=4, Lq=4, ws_bytes=1 << 31, **over):
    s = kv() if s is None else s
    a = ptr(over, "q", "k", "v", "kc", "ks", "vc", "vs", "table", "ctx", "lens")
    return m.load().bdssm_kv_attn_step_ex(ctypes.byref(s), L, Lq, *a, 0, 1.0, *ptr(over, "o", "lse", "ws"), ws_bytes, None)


def weights(s=None, Lq=4, **over):
    s = kv() if s is None else s
    return m.load().bdssm_kv_attn_weights(ctypes.byref(s), Lq, *ptr(over, "q", "lse", "kc", "ks", "table", "ctx", "lens"), 1.0,
                                          *ptr(over, "mass", "out"), None)


def evict(batch=2, pages=100, page=16, budget=50, sink=2, recent=3, **over):
    return m.load().bdssm_kv_evict(batch, pages, page, budget, sink, recent,
                                   *ptr(over, "table", "ctx", "mass", "table_out", "ctx_out", "mass_out"), None)


BAD_CONV = [(dict(dtype=2), DTYPE), (dict(dtype=-1), DTYPE), (dict(width=1), SHAPE), (dict(width=5), SHAPE), (dict(ch=0), SHAPE),
            (dict(ch=1 << 31), SHAPE), (dict(batch=-1), SHAPE), (dict(ld=63), SHAPE), (dict(ld=-64), SHAPE), (dict(batch_ld=639), SHAPE),
            (dict(batch_ld=-640), SHAPE), (dict(ld=1 << 41), SHAPE), (dict(batch_ld=1 << 41), SHAPE), (dict(batch=1 << 40, ch=1 << 20), SHAPE)]


@pytest.mark.parametrize("bad,rc", BAD_CONV)
def test_conv_shapes(bad, rc):
    s = conv(**bad)
    assert scan(s) == step(s) == scan_bwd(s) == rc
    assert m.load().bdssm_conv_workspace_bytes(ctypes.byref(s), 10) == ctypes.c_size_t(-1).value


def test_conv_strides():
    """A row or a token alone has no stride; the gradient's are checked as the input's."""
    lib = m.load()
    ok = lambda s, T: lib.bdssm_conv_workspace_bytes(ctypes.byref(s), T) != ctypes.c_size_t(-1).value  # noqa: E731
    assert ok(conv(batch=1, batch_ld=0), 10) and ok(conv(ld=0, batch_ld=64), 1) and ok(conv(batch=0, ld=0, batch_ld=0), 10)
    assert not ok(conv(ld=0, batch_ld=63), 1)
    assert scan_bwd(ld=63) == scan_bwd(batch_ld=639) == scan_bwd(ld=-1) == SHAPE


@pytest.mark.parametrize("width", [2, 3, 4])
def test_conv_gradients_widest(width):
    """The sum of the gradients' parts: 1,024 threads for 64 of (width + 1) * channels
    columns, and a grid's threads are counted in 32 bits."""
    most = 64 * ((1 << 22) - 1) // (width + 1)
    room = lambda ch: m.load().bdssm_conv_workspace_bytes(ctypes.byref(conv(batch=1, ch=ch, width=width, T=1)), 1)  # noqa: E731
    assert room(most) == (width + 1) * most * 4
    assert room(most + 1) == ctypes.c_size_t(-1).value
    s = conv(batch=1, ch=most + 1, width=width, T=1)
    assert scan_bwd(s, 1, ld=most + 1, batch_ld=most + 1) == SHAPE
    assert scan(s, 1, y=None, c_final=None) == 0   # forward there is no such sum


@pytest.mark.parametrize("T", [-1, 1 << 30, 1 << 40, (1 << 63) - 1])
def test_conv_lengths(T):
    s = conv(batch=1)
    assert scan(s, T=T) == step(s, T=T) == scan_bwd(s, T=T) == SHAPE


BAD_NORM = [(dict(dtype=2), DTYPE), (dict(res_dtype=2), DTYPE), (dict(dtype=0, res_dtype=1), DTYPE), (dict(rows=-1), SHAPE), (dict(ch=0), SHAPE),
            (dict(ch=32769), SHAPE), (dict(rows=1 << 40), SHAPE)]


@pytest.mark.parametrize("bad,rc", BAD_NORM)
def test_norm_shapes(bad, rc):
    s = norm(**bad)
    assert rms(s) == rms_codes(s) == rms_bwd(s) == rc
    assert m.load().bdssm_norm_workspace_bytes(ctypes.byref(s)) == ctypes.c_size_t(-1).value


def test_norm_arguments():
    for eps in (-1e-5, float("nan"), float("inf")):
        assert rms(eps=eps) == rms_codes(eps=eps) == SHAPE
    assert rms_codes(code=2) == rms_codes(code=-1) == DTYPE
    assert rms_codes(group=64) == rms_codes(group=-128) == rms_codes(norm(ch=200), group=128) == SHAPE
    # without a residual h is x: there is no output for it, nor another type
    assert rms(norm(res_dtype=1), res=None) == rms(h=None) == NULL
    assert rms(res=None, h=None) == SHAPE


BAD_KV = [(dict(dtype=2), DTYPE), (dict(code=2), DTYPE), (dict(batch=-1), SHAPE), (dict(batch=32768), SHAPE), (dict(hq=5), SHAPE),
          (dict(d=32), SHAPE), (dict(page=8), SHAPE), (dict(n_pages=-1), SHAPE), (dict(max_pages=1 << 28), SHAPE)]


@pytest.mark.parametrize("bad,rc", BAD_KV)
def test_kv_shapes(bad, rc):
    assert weights(kv(**bad)) == attn(kv(**bad)) == rc


def test_kv_lengths():
    assert weights(Lq=-1) == weights(Lq=1 << 31) == SHAPE
    assert weights(kv(batch=1, hq=32767, hkv=1), Lq=1 << 20) == SHAPE      # more query rows than are counted
    assert attn(L=4, Lq=5) == SHAPE


@pytest.mark.parametrize("bad", [dict(batch=-1), dict(batch=32768), dict(pages=-1), dict(pages=(1 << 18) + 1), dict(page=8), dict(page=48),
                                 dict(budget=-1), dict(sink=-1), dict(recent=-1), dict(sink=51), dict(sink=25, recent=26),
                                 dict(sink=1 << 62, recent=1 << 62, budget=1 << 62)])
def test_evict_arguments(bad):
    assert evict(**bad) == SHAPE


def test_null():
    for n in ("u", "w"):
        assert scan(**{n: None}) == step(**{n: None}) == NULL, n
    for n in ("u", "w", "dy", "du", "dw"):
        assert scan_bwd(**{n: None}) == NULL, n
    for n in ("x", "w", "y"):
        assert rms(**{n: None}) == NULL, n
    for n in ("x", "w", "codes", "scales"):
        assert rms_codes(**{n: None}) == NULL, n
    for n in ("h", "w", "rstd", "dy", "dx", "dw"):
        assert rms_bwd(**{n: None}) == NULL, n
    for n in ("q", "lse", "kc", "ks", "table", "ctx", "out"):
        assert weights(**{n: None}) == NULL, n
    for n in ("table", "ctx", "mass", "table_out", "ctx_out", "mass_out"):
        assert evict(**{n: None}) == NULL, n
    lib = m.load()
    assert lib.bdssm_conv_scan(None, 1, *[None] * 3, 1, *[None] * 6) == NULL
    assert lib.bdssm_conv_step(None, 1, *[None] * 4, 1, *[None] * 4) == NULL
    assert lib.bdssm_conv_scan_bwd(None, 1, *[None] * 3, 1, *[None] * 6, 1, 1, *[None] * 4, 0, None) == NULL
    assert lib.bdssm_rms_norm(None, None, None, None, 0.0, *[None] * 4) == NULL
    assert lib.bdssm_rms_norm_codes(None, None, None, None, 0.0, 0, 0, *[None] * 4) == NULL
    assert lib.bdssm_rms_norm_bwd(*[None] * 10, 0, None) == NULL
    assert lib.bdssm_kv_attn_weights(None, 1, *[None] * 7, 1.0, None, None, None) == NULL
    assert lib.bdssm_conv_workspace_bytes(None, 1) == lib.bdssm_norm_workspace_bytes(None) == ctypes.c_size_t(-1).value


@pytest.mark.parametrize("call,names", [
    (scan, "w bias lens starts c_init y c_final"), (step, "c_init w bias lens y c_final"),
    (scan_bwd, "w bias lens starts c_init dy dc_final dw dbias dc_init ws"), (rms, "x res w y h rstd"),
    (rms_codes, "x res w codes scales h"), (rms_bwd, "h w rstd dy dh dx dres dw ws"),
    (weights, "q lse kc ks table ctx lens mass out"), (attn, "lse"), (evict, "table ctx mass table_out ctx_out mass_out")])
def test_alignment(call, names):
    for n in names.split():
        assert call(**{n: FAKE[n] + 8}) == ALIGN, n


def test_alignment_of_slices():
    """u and du may start at any value, not inside one."""
    for dtype, bad in ((1, (1, 3)), (0, (1, 2, 6))):
        for off in bad:
            s = conv(dtype=dtype)
            assert scan(s, u=FAKE["u"] + off) == step(s, u=FAKE["u"] + off) == scan_bwd(s, u=FAKE["u"] + off) == ALIGN
            assert scan_bwd(s, du=FAKE["du"] + off) == ALIGN


@pytest.mark.parametrize("call,ins,outs", [
    (scan, "u w bias lens starts c_init", "y c_final"), (step, "u w bias lens c_init", "y c_final"),
    (scan_bwd, "u w bias lens starts c_init dy dc_final", "du dw dbias dc_init ws"), (rms, "x res w", "y h rstd"),
    (rms_codes, "x res w", "codes scales h"), (rms_bwd, "h w rstd dy dh", "dx dres dw ws"),
    (weights, "q lse kc ks table ctx lens", "out"), (attn, "q k v kc ks vc vs table ctx lens", "o lse"),
    (evict, "table ctx mass", "table_out ctx_out mass_out")])
def test_overlaps(call, ins, outs):
    """An output on an input or on another output; what may be in place is so only as a whole."""
    may = {("c_init", "c_final"), ("res", "h"), ("mass", "out")} if call is not scan_bwd else set()
    outs = outs.split()
    for o in outs:
        for n in ins.split() + [x for x in outs if x != o]:
            if (n, o) not in may:
                assert call(**{o: FAKE[n]}) == ALIAS, (n, o)
    for n, o in may:
        if n in ins.split() and o in outs:
            assert call(**{o: FAKE[n] + 16}) == ALIAS, (n, o)


def test_overlaps_of_slices():
    """What lies between the slices' rows counts as theirs."""
    s = conv(ld=200, batch_ld=2000)
    last = 2 * ((2 - 1) * 2000 + 9 * 200 + 64)                   # bytes
    assert scan(s, y=FAKE["u"] + last - 16) == ALIAS
    assert scan_bwd(s, du=FAKE["u"] + last - 2) == ALIAS


def test_workspaces():
    lib = m.load()
    n = lib.bdssm_conv_workspace_bytes(ctypes.byref(conv()), 10)
    assert 0 < n < 1 << 31
    assert scan_bwd(ws_bytes=n - 1) == scan_bwd(ws=None) == WORKSPACE
    n = lib.bdssm_norm_workspace_bytes(ctypes.byref(norm()))
    assert n > 0
    assert rms_bwd(ws_bytes=n - 1) == rms_bwd(ws=None) == WORKSPACE


def test_nothing_to_do():
    """Empty calls return without a launch (or a look at their pointers)."""
    assert scan(conv(batch=0), **NONE) == step(conv(batch=0), **NONE) == 0
    assert scan(y=None, c_final=None) == step(y=None, c_final=None) == 0
    assert rms(norm(rows=0), **NONE) == SHAPE and rms(norm(rows=0, res_dtype=1), **NONE) == 0
    assert rms_codes(norm(rows=0, res_dtype=1), **NONE) == 0
    assert weights(kv(batch=0), **NONE) == weights(kv(max_pages=0), **NONE) == evict(batch=0, **NONE) == 0


def test_python_checks():
    z = torch.zeros
    u, w, x = z(1, 4, 8), z(8, 4), z(3, 8)
    state = z(1, 3, 8)
    for call in (lambda: m.conv_scan(u, w), lambda: m.conv_step(state, u, w), lambda: m.conv_scan_bwd(u, w, u),
                 lambda: m.rms_norm(x, z(8)), lambda: m.rms_norm_codes(x, z(8)), lambda: m.rms_norm_bwd(x, z(8), z(3), x)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(ValueError, match="batch, T, channels"):
        m.conv_scan(u[0], w)
    with pytest.raises(ValueError, match="batch, T, channels"):
        m.conv_step(state, None, w)
    with pytest.raises(ValueError, match="group"):
        m.rms_norm_codes(x, z(8), group=64)
    with pytest.raises(TypeError):
        m.rms_norm_codes(x, z(8), code=torch.float16)
    with pytest.raises(ValueError):
        m.rms_norm_bwd(None, z(8), z(3), x)
    table, n = z(1, 2, dtype=torch.int32), z(1, dtype=torch.int32)
    c = m.kv_cache(3, 2, 64, 16, torch.int8, device="cpu")
    q = z(1, 4, 2, 64)
    with pytest.raises(ValueError, match="GPU"):
        m.kv_attn_weights(c, q, z(1, 4, 2), table, n)
    with pytest.raises(ValueError, match="lse"):
        m.kv_attn_weights(c, q, None, table, n)
    with pytest.raises(ValueError, match="KvCache"):
        m.kv_attn_weights(tuple(c), q, z(1, 4, 2), table, n)
    with pytest.raises(TypeError):
        m.kv_attn_weights(c._replace(k=c.k.float()), q, z(1, 4, 2), table, n)
    with pytest.raises(ValueError, match="GPU"):
        m.kv_evict(table, n, z(1, 2), 16, 1)
    with pytest.raises(ValueError, match="needed"):
        m.kv_evict(table, n, None, 16, 1)
    with pytest.raises(ValueError, match="page_table"):
        m.kv_evict(n, n, z(1, 2), 16, 1)


def test_strides_of_slices():
    """What the binding takes for a slice, and what it refuses (host tensors: no stride is read on a GPU)."""
    from mamba_selective_scan_04_amd.layer import _strides
    p = torch.zeros(3, 5, 40)
    assert _strides(p[..., 8:24], "u") == (40, 200) and _strides(p[:, 1:4, :16], "u") == (40, 200) and _strides(p[::2], "u") == (40, 400)
    assert _strides(p[:, :1, 3:7], "u") == (4, 200) and _strides(p[:1, :, :4], "u") == (40, 200)
    assert _strides(torch.zeros(0, 5, 4), "u") == (4, 20) and _strides(torch.zeros(2, 0, 4), "u")[0] == 4
    for bad in (p.transpose(1, 2), p[..., ::2], p[:, :1].expand(3, 5, 40), p[:1].expand(3, 5, 40), p.flip(0).as_strided((3, 5, 40), (100, 40, 1))):
        with pytest.raises(ValueError):
            _strides(bad, "u")
