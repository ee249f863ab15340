"""ctypes binding of the operators around the scans (include/bdssm.h), in the
manner of hybrid.py: argument marshalling only.

The short causal convolution:
  conv_scan(u, w, bias=None, silu=True, lens=None, starts=None, c_init=None, want_y=True) -> (y, c_final)
  conv_step(c_cache, u, w, bias=None, silu=True, lens=None, c_out=None, want_y=True) -> y
  conv_scan_bwd(u, w, dy, bias=None, silu=True, lens=None, starts=None, c_init=None, dc_final=None, want_dc_init=False)
Shapes: u, y [batch, T, channels] fp32 or bf16; w [channels, width], bias
[channels] fp32; states [batch, width - 1, channels] of u's type; lens [batch]
int32; starts [batch, T] bool.  u (and du, if passed in) may be a slice of the
channels or tokens of a wider tensor.

Root-mean-square norm with the residual's addition:
  rms_norm(x, w, res=None, eps=1e-5, want_rstd=False) -> (y, h, rstd)
  rms_norm_codes(x, w, res=None, eps=1e-5, code=torch.float8_e4m3fn, group=0) -> (codes, scales, h)
  rms_norm_bwd(h, w, rstd, dy, dh=None) -> dict
Shapes: x, y [..., channels] fp32 or bf16; res, h the same, of x's type or fp32;
w [channels], rstd [...] fp32; scales [...] or [..., channels / group] fp32.

All other tensors contiguous, everything on the current CUDA (HIP) device; work
is enqueued on torch's current stream and nothing synchronises.
"""
import ctypes

import torch

from .bdssm import _check, _dtype_code, _raise, load
from .hybrid import CODES, _p, _room, _stream


class ConvShape(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("channels", ctypes.c_int64), ("width", ctypes.c_int64),
                ("u_stride", ctypes.c_int64), ("u_batch_stride", ctypes.c_int64), ("dtype", ctypes.c_int32)]


class NormShape(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("channels", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("res_dtype", ctypes.c_int32)]


def _strides(u, name):
    """(token stride, row stride) of a slice of a [batch, T, wider] tensor.  What a
    dimension of one has for a stride says nothing."""
    batch, T, ch = u.shape
    sb, st, sc = u.stride()
    if ch > 1 and sc != 1:
        raise ValueError("%s: neighbouring channels must lie next to each other" % name)
    st = st if T > 1 else ch
    sb = sb if batch > 1 else T * st
    if st < ch or (batch > 1 and T > 0 and sb < (T - 1) * st + ch):
        raise ValueError("%s: tokens and rows must not overlap" % name)
    return st, sb


def _conv(u, w, bias, lens, starts):
    """Checks of the convolution's operands -> (shape, T)."""
    if not isinstance(u, torch.Tensor) or u.dim() != 3:
        raise ValueError("u must be [batch, T, channels]")
    if not u.is_cuda:
        raise ValueError("u must be on the GPU (got %s)" % u.device)
    if not isinstance(w, torch.Tensor) or w.dim() != 2:
        raise ValueError("w must be [channels, width]")
    batch, T, ch = u.shape
    _check(w, "w", torch.float32, (ch, w.shape[1]))
    _check(bias, "bias", torch.float32, (ch,))
    _check(lens, "lens", torch.int32, (batch,))
    _check(starts, "starts", torch.bool, (batch, T))
    return ConvShape(batch, ch, w.shape[1], *_strides(u, "u"), _dtype_code(u)), T


def _conv_state(s):
    return (s.batch, s.width - 1, s.channels)


def conv_scan(u, w, bias=None, silu=True, lens=None, starts=None, c_init=None, want_y=True, y=None, c_final=None):
    """The short causal convolution over whole rows -> (y or None, c_final: the
    last width - 1 inputs).  Tokens at and behind lens[b] are padding; where
    starts[b, t] is set a document begins, in front of which no tap reaches."""
    s, T = _conv(u, w, bias, lens, starts)
    _check(c_init, "c_init", u.dtype, _conv_state(s))
    if y is not None:
        _check(y, "y", u.dtype, u.shape)
    elif want_y:
        y = torch.empty_like(u, memory_format=torch.contiguous_format)
    if c_final is not None:
        _check(c_final, "c_final", u.dtype, _conv_state(s))
    else:
        c_final = u.new_empty(_conv_state(s))
    stream = _stream(u.get_device(), w, bias, lens, starts, c_init, y, c_final)
    rc = load().bdssm_conv_scan(ctypes.byref(s), T, _p(u), _p(w), _p(bias), 1 if silu else 0, _p(lens), _p(starts),
                                _p(c_init), _p(y), _p(c_final), stream)
    _raise("bdssm_conv_scan", rc)
    return y, c_final


def conv_step(c_cache, u, w, bias=None, silu=True, lens=None, c_out=None, want_y=True, y=None):
    """The short causal convolution of the active tokens -> y or None.  c_cache
    None: zero state.  c_out None: the cache is read only (a denoising step);
    c_out=c_cache: the state advances in place (a commit)."""
    s, T = _conv(u, w, bias, lens, None)
    _check(c_cache, "c_cache", u.dtype, _conv_state(s))
    _check(c_out, "c_out", u.dtype, _conv_state(s))
    if y is not None:
        _check(y, "y", u.dtype, u.shape)
    elif want_y:
        y = torch.empty_like(u, memory_format=torch.contiguous_format)
    stream = _stream(u.get_device(), c_cache, w, bias, lens, y, c_out)
    rc = load().bdssm_conv_step(ctypes.byref(s), T, _p(c_cache), _p(u), _p(w), _p(bias), 1 if silu else 0, _p(lens),
                                _p(y), _p(c_out), stream)
    _raise("bdssm_conv_step", rc)
    return y


def conv_scan_bwd(u, w, dy, bias=None, silu=True, lens=None, starts=None, c_init=None, dc_final=None,
                  want_dc_init=False, du=None, ws=None):
    """Gradients of conv_scan given dy (and dJ/dc_final) -> dict with du, dc_init
    (or None; u's type), dw and dbias (or None; fp32).  du may be a slice of a
    wider gradient."""
    s, T = _conv(u, w, bias, lens, starts)
    _check(c_init, "c_init", u.dtype, _conv_state(s))
    if dy is None:
        raise ValueError("dy is needed for the gradients")
    _check(dy, "dy", u.dtype, u.shape)
    _check(dc_final, "dc_final", u.dtype, _conv_state(s))
    if du is None:
        du = torch.empty_like(u, memory_format=torch.contiguous_format)
    if not isinstance(du, torch.Tensor) or du.dtype is not u.dtype or du.shape != u.shape or not du.is_cuda:
        raise ValueError("du must be on the GPU with u's shape and type")
    ld = _strides(du, "du")
    dw = torch.empty_like(w)
    dbias = None if bias is None else torch.empty_like(bias)
    dc = u.new_empty(_conv_state(s)) if want_dc_init else None
    stream = _stream(u.get_device(), w, bias, lens, starts, c_init, dy, dc_final, du, ws)
    ws, room = _room(ws, "bdssm_conv_workspace_bytes", ctypes.byref(s), T, u.device)
    rc = load().bdssm_conv_scan_bwd(ctypes.byref(s), T, _p(u), _p(w), _p(bias), 1 if silu else 0, _p(lens), _p(starts),
                                    _p(c_init), _p(dy), _p(dc_final), _p(du), *ld, _p(dw), _p(dbias), _p(dc), _p(ws), room,
                                    stream)
    _raise("bdssm_conv_scan_bwd", rc)
    return {"du": du, "dw": dw, "dbias": dbias, "dc_init": dc}


def _norm(x, w, res):
    """Checks of the norm's operands -> shape."""
    if not isinstance(x, torch.Tensor) or x.dim() < 1:
        raise ValueError("x must be [..., channels]")
    _check(x, "x")
    code, ch = _dtype_code(x), x.shape[-1]
    if res is not None and (not isinstance(res, torch.Tensor) or res.dtype is not x.dtype and res.dtype is not torch.float32):
        raise TypeError("res must have x's type or float32")
    _check(res, "res", None, x.shape)
    _check(w, "w", torch.float32, (ch,))
    return NormShape(x.numel() // ch if ch else 0, ch, code, code if res is None else _dtype_code(res))


def _norm_h(x, res, h):
    if res is None:
        if h is not None:
            raise ValueError("h is x without a residual")
        return None
    if h is None:
        return torch.empty_like(res)
    _check(h, "h", res.dtype, x.shape)
    return h


def rms_norm(x, w, res=None, eps=1e-5, want_rstd=False, y=None, h=None):
    """Root-mean-square norm of x + res -> (y, h, rstd or None): h is the sum, of
    res's type (without res: x itself; h=res: in place), rstd what rms_norm_bwd
    needs."""
    s = _norm(x, w, res)
    out = _norm_h(x, res, h)
    if y is None:
        y = torch.empty_like(x)
    else:
        _check(y, "y", x.dtype, x.shape)
    rstd = w.new_empty(x.shape[:-1]) if want_rstd else None
    stream = _stream(x.get_device(), w, res, y, out)
    rc = load().bdssm_rms_norm(ctypes.byref(s), _p(x), _p(res), _p(w), eps, _p(y), _p(out), _p(rstd), stream)
    _raise("bdssm_rms_norm", rc)
    return y, x if res is None else out, rstd


def rms_norm_codes(x, w, res=None, eps=1e-5, code=torch.float8_e4m3fn, group=0, h=None):
    """The norm in 8 bits -> (codes, scales, h): value = code * scale, one scale
    a row (group 0: scales [...]) or each 128 channels (scales [..., channels / 128])."""
    if code not in CODES:
        raise TypeError("code must be torch.float8_e4m3fn or torch.int8")
    if group not in (0, 128):
        raise ValueError("group must be 0 (a row) or 128, got %r" % (group,))
    s = _norm(x, w, res)
    out = _norm_h(x, res, h)
    codes = torch.empty_like(x, dtype=code)
    scales = w.new_empty(x.shape[:-1] + (x.shape[-1] // group,) if group else x.shape[:-1])
    stream = _stream(x.get_device(), w, res, out)
    rc = load().bdssm_rms_norm_codes(ctypes.byref(s), _p(x), _p(res), _p(w), eps, CODES[code], group, _p(codes),
                                     _p(scales), _p(out), stream)
    _raise("bdssm_rms_norm_codes", rc)
    return codes, scales, x if res is None else out


def rms_norm_bwd(h, w, rstd, dy, dh=None, ws=None):
    """Gradients of rms_norm given dy (and dh: what reaches h from elsewhere) ->
    dict with dx (dy's type), dres (h's type; dx itself where that is dy's) and
    dw (fp32).  h, rstd: what rms_norm returned."""
    if not isinstance(dy, torch.Tensor) or dy.dim() < 1 or not isinstance(h, torch.Tensor):
        raise ValueError("h and dy must be [..., channels]")
    s = _norm(dy, w, h)
    _check(rstd, "rstd", torch.float32, dy.shape[:-1])
    if rstd is None:
        raise ValueError("rstd is needed for the gradients")
    _check(dh, "dh", h.dtype, dy.shape)
    dx, dw = torch.empty_like(dy), torch.empty_like(w)
    dres = dx if h.dtype is dy.dtype else torch.empty_like(h)
    stream = _stream(dy.get_device(), h, w, rstd, dh, ws)
    ws, room = _room(ws, "bdssm_norm_workspace_bytes", ctypes.byref(s), dy.device)
    rc = load().bdssm_rms_norm_bwd(ctypes.byref(s), _p(h), _p(w), _p(rstd), _p(dy), _p(dh), _p(dx),
                                   None if dres is dx else _p(dres), _p(dw), _p(ws), room, stream)
    _raise("bdssm_rms_norm_bwd", rc)
    return {"dx": dx, "dres": dres, "dw": dw}
