"""Binding of the 8-bit integer layers declared in include/tg_int8.h.

    tg_quantize_i8(x, q, scale)
    tg_linear_i8(x, W, Y, scale_x, scale_w, bias=None, act="none", residual=None, workspace=None)
    tg_linear_i8_workspace_bytes(M, N, K)

Outputs are tensors of the caller's.  ``workspace`` is ``tg_ops_workspace``'s.
Wrong shapes, types or devices raise ValueError before anything is launched,
what the library itself refuses raises TGError.
"""
from __future__ import annotations

import ctypes

import torch

from . import _CDTYPE, TGError, _stream, load
from .ops import _2d, _NONE, _OWN, _act, _current_stream, _device, _mat, _vec, _ws

EXPORTS = ("tg_quantize_i8", "tg_linear_i8", "tg_linear_i8_workspace_bytes")

_fns = None
_I8 = (torch.int8,)
_FLOATS = tuple(_CDTYPE)


def _lib():
    """The library with the argument types of these entry points set."""
    global _fns
    if _fns is None:
        lib = load()
        i64, vp, ci = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
        mat, ws = [vp, i64], [vp, i64, vp]
        lib.tg_quantize_i8.argtypes = [ci, i64, i64, *mat, *mat, vp, vp]
        lib.tg_linear_i8.argtypes = [i64, i64, i64, *mat, *mat, vp, vp, vp, ci, *mat, *mat, ci, *ws]
        lib.tg_quantize_i8.restype = lib.tg_linear_i8.restype = ci
        lib.tg_linear_i8_workspace_bytes.argtypes = [i64, i64, i64]
        lib.tg_linear_i8_workspace_bytes.restype = i64
        _fns = lib
    return _fns


def tg_quantize_i8(x, q, scale, stream=None) -> None:
    """q = round(x / scale) as int8 with scale[m] = max |x[m]| / 127: tokens of activations, or channels of a weight."""
    M, K = _2d(x, "x")
    dev = _device(x, "x")
    px, ldx = _mat(x, "x", M, K, _FLOATS, dev)
    pq, ldq = _mat(q, "q", M, K, _I8, dev)
    ps = _vec(scale, "scale", M, dev)
    code = (_fns or _lib()).tg_quantize_i8(_CDTYPE[x.dtype], M, K, px, ldx, pq, ldq, ps,
                                           _current_stream(dev) if stream is None else _stream(stream))
    if code:
        raise TGError("tg_quantize_i8", code)


def tg_linear_i8_workspace_bytes(M: int, N: int, K: int) -> int:
    """Workspace bytes tg_linear_i8 can use for this problem (0: it never splits)."""
    n = int(_lib().tg_linear_i8_workspace_bytes(int(M), int(N), int(K)))
    if n < 0:
        raise ValueError("invalid sizes")
    return n


def tg_linear_i8(x, W, Y, scale_x, scale_w, bias=None, act: str = "none", residual=None, workspace=None, stream=None) -> None:
    """Y = act(scale_x[m] scale_w[n] (x . W^T) + bias) + residual, x and W int8 (W stored N x K), the sums exact."""
    M, K = _2d(x, "x")
    N = _2d(W, "W")[0]
    a = _act(act)
    dev = _device(x, "x")
    px, ldx = _mat(x, "x", M, K, _I8, dev)
    pw, ldw = _mat(W, "W", N, K, _I8, dev)
    py, ldy = _mat(Y, "Y", M, N, _FLOATS, dev)
    yt = Y.dtype
    pr, ldr = _NONE if residual is None else _mat(residual, "residual", M, N, _OWN[yt], dev)
    sx, sw = _vec(scale_x, "scale_x", M, dev), _vec(scale_w, "scale_w", N, dev)
    pb = None if bias is None else _vec(bias, "bias", N, dev)
    ps, ns = _ws(workspace, dev)
    code = (_fns or _lib()).tg_linear_i8(M, N, K, px, ldx, pw, ldw, sx, sw, pb, a, pr, ldr, py, ldy, _CDTYPE[yt], ps, ns,
                                         _current_stream(dev) if stream is None else _stream(stream))
    if code:
        raise TGError("tg_linear_i8", code)
