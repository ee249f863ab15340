"""ctypes binding of the hybrid layer's other operators (include/bdssm.h), in
the manner of bdssm.py: argument marshalling only.

The gated delta rule:
  delta_scan(q, k, v, g, beta, scale=None, h_init=None, lens=None, want_o=True, want_chunks=False)
  delta_scan_bwd(q, k, v, g, beta, h_chunks, do, scale=None, lens=None, dh_final=None, want_dh_init=False)
  delta_step(h_cache, q, k, v, g, beta, scale=None, lens=None, h_out=None, want_o=True)
Shapes: q, k [batch, T, heads_k, d_k]; v, o [batch, T, heads_v, d_v]; g (log
decay), beta [batch, T, heads_v] fp32; states [batch, heads_v, d_k, d_v] fp32;
lens [batch] int32 or None.  q, k, v, o share fp32 or bf16.  scale None:
d_k ** -0.5.  ws (delta_scan, delta_scan_bwd, kv_attn_step): the caller's own
workspace, a contiguous tensor of the library's *_workspace_bytes.

Attention over the paged 8-bit cache:
  kv_cache(n_pages, heads_kv, head_dim, page_len, code) -> KvCache
  kv_commit(cache, k, v, page_table, ctx_lens, lens=None)
  kv_attn_step(cache, q, k, v, page_table, ctx_lens, lens=None, causal=False, scale=None)
Shapes: k, v [batch, L, heads_kv, head_dim]; q, o [batch, Lq, heads_q,
head_dim]; page_table [batch, max_pages], ctx_lens, lens [batch] int32.

All tensors contiguous and on the current CUDA (HIP) device; work
is enqueued on torch's current stream and nothing synchronises.
"""
import collections
import ctypes

import torch

from .bdssm import _check, _dtype_code, _raise, _workspace, load

DELTA_CHUNK = 64        # BDSSM_DELTA_CHUNK


def _room(ws, name, *args):
    """The workspace to use and its bytes: the caller's, or a new one of what the
    library asks for (a shape it does not take asks for none: the call says so)."""
    if ws is None:
        n = getattr(load(), name)(*args[:-1])
        ws = _workspace(n if n != ctypes.c_size_t(-1).value else 0, args[-1])
        return ws, 0 if ws is None else ws.numel()
    _check(ws, "ws")   # contiguous: its elements are as many bytes as it has
    return ws, ws.numel() * ws.element_size()


def _p(t):
    # an int: ctypes takes it for a pointer argument, and makes no object of it
    return None if t is None else t.data_ptr()


def _stream(dev, *tensors):
    """The current stream of device `dev`, which must be the current device and
    that of every tensor: the library launches on the current device, and a
    pointer of another one would fault there."""
    if dev != torch._C._cuda_getDevice():
        raise ValueError("the tensors must be on the current device (cuda:%d), got cuda:%d"
                         % (torch._C._cuda_getDevice(), dev))
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError("all tensors must be on cuda:%d (got cuda:%d)" % (dev, t.get_device()))
    # the raw handle: making a torch.cuda.Stream of it costs 3 us a call
    return torch._C._cuda_getCurrentRawStream(dev)


class DeltaShape(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("heads_k", ctypes.c_int64), ("heads_v", ctypes.c_int64),
                ("d_k", ctypes.c_int64), ("d_v", ctypes.c_int64), ("dtype", ctypes.c_int32)]


def _delta(q, k, v, g, beta, lens, scale):
    """Checks of the delta rule's operands -> (shape, T, device, scale)."""
    if not isinstance(k, torch.Tensor) or k.dim() != 4 or not isinstance(v, torch.Tensor) or v.dim() != 4:
        raise ValueError("k must be [batch, T, heads_k, d_k] and v [batch, T, heads_v, d_v]")
    _check(k, "k")
    code = _dtype_code(k)
    batch, T, hk, dk = k.shape
    hv, dv = v.shape[2:]
    _check(v, "v", k.dtype, (batch, T, hv, dv))
    _check(q, "q", k.dtype, (batch, T, hk, dk))
    _check(g, "g", torch.float32, (batch, T, hv))
    _check(beta, "beta", torch.float32, (batch, T, hv))
    _check(lens, "lens", torch.int32, (batch,))
    return DeltaShape(batch, hk, hv, dk, dv, code), T, k.device, float(dk ** -0.5 if scale is None else scale)


def delta_workspace_bytes(s, T, bwd=False):
    """Workspace bytes of delta_scan (or of its backward) for a DeltaShape."""
    n = load().bdssm_delta_workspace_bytes(ctypes.byref(s), T, 1 if bwd else 0)
    if n == ctypes.c_size_t(-1).value:
        raise ValueError("invalid shape for workspace query")
    return n


def _state(s):
    return (s.batch, s.heads_v, s.d_k, s.d_v)


def _chunk_states(s, T):
    return (s.batch, -(-T // DELTA_CHUNK), s.heads_v, s.d_v, s.d_k)


def delta_scan(q, k, v, g, beta, scale=None, h_init=None, lens=None, want_o=True, want_chunks=False, o=None,
               h_final=None, h_chunks=None, ws=None):
    """The gated delta rule over whole rows -> (o or None, h_final, h_chunks or
    None).  h_chunks [batch, ceil(T / 64), heads_v, d_v, d_k]: the (transposed)
    states before every 64th token, for delta_scan_bwd.
    Tokens at and behind lens[b] are padding.  q may be None with want_o=False."""
    want_o = want_o or o is not None
    s, T, dev, scale = _delta(q, k, v, g, beta, lens, scale)
    if want_o and q is None:
        raise ValueError("q is needed for o")
    _check(h_init, "h_init", torch.float32, _state(s))
    if want_o and o is None:
        o = torch.empty_like(v)
    _check(o, "o", k.dtype, tuple(v.shape))
    if h_final is None:
        h_final = torch.empty(_state(s), dtype=torch.float32, device=dev)
    _check(h_final, "h_final", torch.float32, _state(s))
    if want_chunks and h_chunks is None:
        h_chunks = torch.empty(_chunk_states(s, T), dtype=torch.float32, device=dev)
    _check(h_chunks, "h_chunks", torch.float32, _chunk_states(s, T))
    stream = _stream(k.get_device(), q, v, g, beta, lens, h_init, o, h_final, h_chunks, ws)
    ws, room = _room(ws, "bdssm_delta_workspace_bytes", ctypes.byref(s), T, 0, dev)
    rc = load().bdssm_delta_scan(ctypes.byref(s), T, _p(q), _p(k), _p(v), _p(g), _p(beta), scale, _p(lens),
                                 _p(h_init), _p(o), _p(h_final), _p(h_chunks), _p(ws),
                                 room, stream)
    _raise("bdssm_delta_scan", rc)
    return o, h_final, h_chunks


def delta_scan_bwd(q, k, v, g, beta, h_chunks, do, scale=None, lens=None, dh_final=None, want_dh_init=False, ws=None):
    """Gradients of delta_scan given do (and dJ/dh_final) -> dict with dq, dk, dv
    (stream dtype), dg, dbeta (fp32) and dh_init (fp32 or None).  h_chunks: what
    delta_scan(..., want_chunks=True) returned for the same inputs."""
    if q is None:
        raise ValueError("q is needed for the gradients")
    s, T, dev, scale = _delta(q, k, v, g, beta, lens, scale)
    if h_chunks is None or do is None:
        raise ValueError("h_chunks and do are needed for the gradients")
    _check(h_chunks, "h_chunks", torch.float32, _chunk_states(s, T))
    _check(do, "do", k.dtype, tuple(v.shape))
    _check(dh_final, "dh_final", torch.float32, _state(s))
    stream = _stream(k.get_device(), q, v, g, beta, lens, h_chunks, do, dh_final, ws)
    dq, dk, dv, dg, dbeta = (torch.empty_like(x) for x in (q, k, v, g, beta))
    dh = torch.empty(_state(s), dtype=torch.float32, device=dev) if want_dh_init else None
    ws, room = _room(ws, "bdssm_delta_workspace_bytes", ctypes.byref(s), T, 1, dev)
    rc = load().bdssm_delta_scan_bwd(ctypes.byref(s), T, _p(q), _p(k), _p(v), _p(g), _p(beta), scale, _p(lens),
                                     _p(h_chunks), _p(do), _p(dh_final), _p(dq), _p(dk), _p(dv), _p(dg), _p(dbeta),
                                     _p(dh), _p(ws), room, stream)
    _raise("bdssm_delta_scan_bwd", rc)
    return {"dq": dq, "dk": dk, "dv": dv, "dg": dg, "dbeta": dbeta, "dh_init": dh}


def delta_step(h_cache, q, k, v, g, beta, scale=None, lens=None, h_out=None, want_o=True, o=None):
    """The gated delta rule token by token on the active tokens -> o or None.
    h_cache None: zero state.  h_out None: the cache is read only (a denoising
    step); h_out=h_cache: the state advances in place (a commit)."""
    want_o = want_o or o is not None
    s, T, dev, scale = _delta(q, k, v, g, beta, lens, scale)
    if want_o and q is None:
        raise ValueError("q is needed for o")
    _check(h_cache, "h_cache", torch.float32, _state(s))
    _check(h_out, "h_out", torch.float32, _state(s))
    if want_o and o is None:
        o = torch.empty_like(v)
    _check(o, "o", k.dtype, tuple(v.shape))
    stream = _stream(k.get_device(), h_cache, q, v, g, beta, lens, o, h_out)
    rc = load().bdssm_delta_step(ctypes.byref(s), T, _p(h_cache), _p(q), _p(k), _p(v), _p(g), _p(beta), scale,
                                 _p(lens), _p(o), _p(h_out), stream)
    _raise("bdssm_delta_step", rc)
    return o


CODES = {torch.float8_e4m3fn: 0, torch.int8: 1}     # bdssm_code

# the cache's tensors: codes of keys [n_pages, heads_kv, page_len, head_dim] and
# values [n_pages, heads_kv, head_dim, page_len] (float8_e4m3fn or int8), their
# scales [n_pages, heads_kv] fp32
KvCache = collections.namedtuple("KvCache", "k k_scale v v_scale")


class KvShape(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("heads_q", ctypes.c_int64), ("heads_kv", ctypes.c_int64),
                ("head_dim", ctypes.c_int64), ("page_len", ctypes.c_int64), ("n_pages", ctypes.c_int64),
                ("max_pages", ctypes.c_int64), ("dtype", ctypes.c_int32), ("code", ctypes.c_int32)]


def kv_cache(n_pages, heads_kv, head_dim, page_len=16, code=torch.float8_e4m3fn, device="cuda"):
    """An empty cache (codes and scales zero)."""
    if code not in CODES:
        raise TypeError("code must be torch.float8_e4m3fn or torch.int8")
    z = lambda *s: torch.zeros(*s, dtype=torch.int8, device=device).view(code)  # noqa: E731
    sc = lambda: torch.zeros(n_pages, heads_kv, dtype=torch.float32, device=device)  # noqa: E731
    return KvCache(z(n_pages, heads_kv, page_len, head_dim), sc(), z(n_pages, heads_kv, head_dim, page_len), sc())


def _kv(cache, k, v, page_table, ctx_lens, lens, heads_q):
    """Checks of the cache's operands -> (shape, L)."""
    if not isinstance(k, torch.Tensor) or k.dim() != 4:
        raise ValueError("k must be [batch, L, heads_kv, head_dim]")
    if not isinstance(cache, KvCache) or not isinstance(cache.k, torch.Tensor) or cache.k.dim() != 4:
        raise ValueError("cache must be a KvCache with k [n_pages, heads_kv, page_len, head_dim]")
    if cache.k.dtype not in CODES:
        raise TypeError("the cache's codes must be float8_e4m3fn or int8, got %s" % cache.k.dtype)
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
        raise ValueError("page_table must be [batch, max_pages]")
    batch, L, hkv, d = k.shape
    n_pages, page = cache.k.shape[0], cache.k.shape[2]
    _check(k, "k")
    _check(v, "v", k.dtype, k.shape)
    _check(cache.k, "cache.k", cache.k.dtype, (n_pages, hkv, page, d))
    _check(cache.v, "cache.v", cache.k.dtype, (n_pages, hkv, d, page))
    _check(cache.k_scale, "cache.k_scale", torch.float32, (n_pages, hkv))
    _check(cache.v_scale, "cache.v_scale", torch.float32, (n_pages, hkv))
    _check(page_table, "page_table", torch.int32, (batch, page_table.shape[1]))
    _check(ctx_lens, "ctx_lens", torch.int32, (batch,))
    _check(lens, "lens", torch.int32, (batch,))
    return KvShape(batch, heads_q or hkv, hkv, d, page, n_pages, page_table.shape[1], _dtype_code(k), CODES[cache.k.dtype]), L


def kv_commit(cache, k, v, page_table, ctx_lens, lens=None):
    """The rows' whole blocks of k, v into the pages behind ctx_lens, in place.
    Tokens behind a row's last whole block are not cached."""
    s, L = _kv(cache, k, v, page_table, ctx_lens, lens, 0)
    stream = _stream(k.get_device(), v, page_table, ctx_lens, lens, *cache)
    rc = load().bdssm_kv_commit(ctypes.byref(s), L, _p(k), _p(v), _p(page_table), _p(ctx_lens), _p(lens), _p(cache.k),
                                _p(cache.k_scale), _p(cache.v), _p(cache.v_scale), stream)
    _raise("bdssm_kv_commit", rc)


def kv_attn_step(cache, q, k, v, page_table, ctx_lens, lens=None, causal=False, scale=None, o=None, ws=None):
    """Attention of the active tokens' queries over the cache and the active keys
    and values -> o.  Lq <= L queries a row: those of its last active tokens.
    causal: among the active tokens; scale None: head_dim ** -0.5."""
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise ValueError("q must be [batch, Lq, heads_q, head_dim]")
    s, L = _kv(cache, k, v, page_table, ctx_lens, lens, q.shape[2])
    Lq = q.shape[1]
    _check(q, "q", k.dtype, (s.batch, Lq, s.heads_q, s.head_dim))
    if o is None:
        o = torch.empty_like(q)
    _check(o, "o", k.dtype, tuple(q.shape))
    stream = _stream(k.get_device(), q, v, page_table, ctx_lens, lens, o, ws, *cache)
    ws, room = _room(ws, "bdssm_kv_workspace_bytes", ctypes.byref(s), Lq, k.device)
    rc = load().bdssm_kv_attn_step(ctypes.byref(s), L, Lq, _p(q), _p(k), _p(v), _p(cache.k), _p(cache.k_scale),
                                   _p(cache.v), _p(cache.v_scale), _p(page_table), _p(ctx_lens), _p(lens),
                                   1 if causal else 0, float(s.head_dim ** -0.5 if scale is None else scale), _p(o),
                                   _p(ws), room, stream)
    _raise("bdssm_kv_attn_step", rc)
    return o
