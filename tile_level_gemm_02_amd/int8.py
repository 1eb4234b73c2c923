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

from . import TGError, _stream, load
from . import ops as _ops
from .ops import _act, _current_stream, _device

EXPORTS = ("tg_quantize_i8", "tg_linear_i8", "tg_linear_i8_workspace_bytes")

_fns = None
_quantize_address = _linear_address = 0  # in the loaded library


def _lib():
    """The library with the argument types of these entry points set."""
    global _fns, _quantize_address, _linear_address
    if _fns is None:
        lib = load()
        i64, vp, ci = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
        mat, ws = [vp, i64], [vp, i64, vp]
        lib.tg_quantize_i8.argtypes = [ci, i64, i64, *mat, *mat, vp, vp]
        lib.tg_linear_i8.argtypes = [i64, i64, i64, *mat, *mat, vp, vp, vp, ci, *mat, *mat, ci, *ws]
        lib.tg_quantize_i8.restype = lib.tg_linear_i8.restype = ci
        lib.tg_linear_i8_workspace_bytes.argtypes = [i64, i64, i64]
        lib.tg_linear_i8_workspace_bytes.restype = i64
        _quantize_address = ctypes.cast(lib.tg_quantize_i8, ctypes.c_void_p).value
        _linear_address = ctypes.cast(lib.tg_linear_i8, ctypes.c_void_p).value
        _fns = lib
    return _fns


def _bind():
    """The native helper, which reads the tensors of these calls."""
    if _fns is None:
        _lib()
    if _ops._bind is None:
        _ops._load_bind()
    return _ops._bind


def tg_quantize_i8(x, q, scale, stream=None) -> None:
    """q = round(x / scale) as int8 with scale[m] = max |x[m]| / 127: tokens of activations, or channels of a weight."""
    dev = _device(x, "x")
    code = _bind().quantize_i8(_quantize_address, x, q, scale, dev, _current_stream(dev) if stream is None else _stream(stream))
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
    a = _act(act)
    dev = _device(x, "x")
    code = _bind().linear_i8(_linear_address, x, W, Y, scale_x, scale_w, bias, a, residual, workspace, dev,
                             _current_stream(dev) if stream is None else _stream(stream))
    if code:
        raise TGError("tg_linear_i8", code)
