"""Binding of the training operators declared in include/tg_train.h.

    tg_linear_xent(x, W, targets, loss=None, lse=None, total=None, scale=1.0, ignore_index=-100, z_loss=0.0, ...)
    tg_linear_xent_backward(x, W, targets, lse, dx=None, dw=None, dloss=None, total=None, grad_scale=1.0, scale=1.0, ...)
    tg_adamw(params, grads, exp_avg, exp_avg_sq, step, lr, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, masters=None, ...)
    tg_linear_xent_workspace_bytes(dtype, M, V, D), tg_linear_xent_backward_workspace_bytes(dtype, M, V, D, piece=0)

Outputs are tensors of the caller's; None leaves an optional one out.  A
``workspace`` is an int32 tensor that is zero before its first use, as
``tg_ops_workspace`` makes one; the loss needs its query's bytes.  Wrong
shapes, types or devices raise ValueError before anything is launched, what
the library itself refuses raises TGError.
"""
from __future__ import annotations

import ctypes

import torch

from . import _CDTYPE, TGError, _stream, load
from . import ops as _ops
from .ops import _2d, _NONE, _OWN, _OWN_OR_F32, _current_stream, _device, _input16, _mat, _vec, _ws

EXPORTS = ("tg_linear_xent", "tg_linear_xent_workspace_bytes", "tg_linear_xent_backward",
           "tg_linear_xent_backward_workspace_bytes", "tg_adamw")

_fns = None
_adamw_address = 0  # of tg_adamw in the loaded library


def _lib():
    """The library with the argument types of these entry points set."""
    global _fns, _adamw_address
    if _fns is None:
        lib = load()
        i64, vp, f32, f64, ci = ctypes.c_int64, ctypes.c_void_p, ctypes.c_float, ctypes.c_double, ctypes.c_int
        mat, ws = [vp, i64], [vp, i64, vp]
        lib.tg_linear_xent.argtypes = [ci, i64, i64, i64, *mat, *mat, f32, vp, i64, f32, vp, vp, vp, *ws]
        lib.tg_linear_xent_backward.argtypes = [ci, i64, i64, i64, *mat, *mat, f32, vp, i64, f32, vp, vp, f32, vp, *mat, *mat, ci, *ws]
        lib.tg_adamw.argtypes = [i64, vp, i64, f64, f64, f64, f64, f64, vp, f32, vp, vp, vp]
        lib.tg_linear_xent.restype = lib.tg_linear_xent_backward.restype = lib.tg_adamw.restype = ci
        lib.tg_linear_xent_workspace_bytes.argtypes = [ci, i64, i64, i64]
        lib.tg_linear_xent_backward_workspace_bytes.argtypes = [ci, i64, i64, i64, i64]
        lib.tg_linear_xent_workspace_bytes.restype = lib.tg_linear_xent_backward_workspace_bytes.restype = i64
        _adamw_address = ctypes.cast(lib.tg_adamw, ctypes.c_void_p).value
        _fns = lib
    return _fns


# -------------------------------------------------------------------- loss


def _query(name: str, dtype, *sizes: int) -> int:
    n = int(getattr(_lib(), name)(_input16_type(dtype), *(int(s) for s in sizes)))
    if n < 0:
        raise ValueError("invalid sizes")
    return n


def _input16_type(dtype) -> int:
    if dtype not in _ops._16BIT:
        raise ValueError(f"the vocabulary loss takes float16 or bfloat16 inputs, got {dtype}")
    return _ops._IN[dtype]


def tg_linear_xent_workspace_bytes(dtype, M: int, V: int, D: int) -> int:
    """Workspace bytes that tg_linear_xent needs for this problem."""
    return _query("tg_linear_xent_workspace_bytes", dtype, M, V, D)


def tg_linear_xent_backward_workspace_bytes(dtype, M: int, V: int, D: int, piece: int = 0) -> int:
    """Workspace bytes of tg_linear_xent_backward with pieces of `piece` columns of the vocabulary.

    piece 0: the size past which more gives nothing; piece 1: the least that the call takes."""
    return _query("tg_linear_xent_backward_workspace_bytes", dtype, M, V, D, piece)


def _targets(t, M: int, dev: int) -> int:
    if t.dtype != torch.int64 or t.shape != (M,) or not t.is_contiguous():
        raise ValueError(f"targets must be a contiguous int64 vector of {M}")
    if t.get_device() != dev:
        raise ValueError(f"every tensor must be on the current GPU, targets is on {t.device}")
    return t.data_ptr()


def tg_linear_xent(x, W, targets, loss=None, lse=None, total=None, scale: float = 1.0, ignore_index: int = -100,
                   z_loss: float = 0.0, workspace=None, stream=None) -> None:
    """loss[m] = lse[m] - t[m][targets[m]] + z_loss lse[m]^2 with t = scale x . W^T and lse its log-sum-exp over the rows of W.

    Rows whose target is ``ignore_index`` lose 0.  ``loss`` and ``lse`` are
    float32 vectors, ``total`` (float32, 2) receives the sum of the losses and
    the number of rows that count.  Logits are never stored."""
    i = _input16(x, "tg_linear_xent")
    M, D = _2d(x, "x")
    V = _2d(W, "W")[0]
    dev = _device(x, "x")
    own = _OWN[x.dtype]
    px, ldx = _mat(x, "x", M, D, own, dev)
    pw, ldw = _mat(W, "W", V, D, own, dev)
    pt = _targets(targets, M, dev)
    pl = None if loss is None else _vec(loss, "loss", M, dev)
    pe = None if lse is None else _vec(lse, "lse", M, dev)
    pq = None if total is None else _vec(total, "total", 2, dev)
    ps, ns = _ws(workspace, dev)
    code = (_fns or _lib()).tg_linear_xent(i, M, V, D, px, ldx, pw, ldw, scale, pt, ignore_index, z_loss, pl, pe, pq, ps, ns,
                                           _current_stream(dev) if stream is None else _stream(stream))
    if code:
        raise TGError("tg_linear_xent", code)


def tg_linear_xent_backward(x, W, targets, lse, dx=None, dw=None, dloss=None, total=None, grad_scale: float = 1.0,
                            scale: float = 1.0, ignore_index: int = -100, z_loss: float = 0.0, workspace=None,
                            stream=None) -> None:
    """Gradients of sum over m of g[m] loss[m], g = grad_scale * dloss / count (dloss None: 1; total None: count 1).

    ``lse`` and ``total`` are tg_linear_xent's; each of dx (like x) and dw
    (like W, or float32) that is given is written.  The workspace's size sets
    how many pieces the vocabulary is taken in."""
    i = _input16(x, "tg_linear_xent_backward")
    M, D = _2d(x, "x")
    V = _2d(W, "W")[0]
    dev = _device(x, "x")
    t = x.dtype
    own = _OWN[t]
    px, ldx = _mat(x, "x", M, D, own, dev)
    pw, ldw = _mat(W, "W", V, D, own, dev)
    pt = _targets(targets, M, dev)
    pe = _vec(lse, "lse", M, dev)
    pd = None if dloss is None else _vec(dloss, "dloss", M, dev)
    pq = None if total is None else _vec(total, "total", 2, dev)
    pdx, lddx = _NONE if dx is None else _mat(dx, "dx", M, D, own, dev)
    pdw, lddw = _NONE if dw is None else _mat(dw, "dw", V, D, _OWN_OR_F32[t], dev)
    ps, ns = _ws(workspace, dev)
    code = (_fns or _lib()).tg_linear_xent_backward(
        i, M, V, D, px, ldx, pw, ldw, scale, pt, ignore_index, z_loss, pe, pd, grad_scale, pq, pdx, lddx, pdw, lddw,
        0 if dw is None else _CDTYPE[dw.dtype], ps, ns, _current_stream(dev) if stream is None else _stream(stream))
    if code:
        raise TGError("tg_linear_xent_backward", code)


# --------------------------------------------------------------- optimizer


def tg_adamw(params, grads, exp_avg, exp_avg_sq, step, lr, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay: float = 0.01,
             masters=None, exp_avg_scales=None, exp_avg_sq_scales=None, norm=None, max_norm: float = float("inf"),
             stream=None) -> None:
    """One AdamW step over lists of tensors, in one launch per 48 of them.

    params and grads are float32, float16 or bfloat16; masters (float32, or
    None) hold the weights where params are their rounded copies.  States are
    float32, or float8_e4m3fn with float32 scales for each block of 256
    elements: exp_avg = scale q and the root of exp_avg_sq = scale q.  ``norm``
    (float32, one element, as tg_clip_grads writes it) scales the gradients by
    min(1, max_norm / (norm + 1e-6)); a norm that is not finite leaves
    everything as it is.  ``step`` (1 for the first) and ``lr`` may be tensors
    of one int64 and one float32 on the GPU, for a captured step."""
    lists = [v if v is None or type(v) is list else list(v)
             for v in (params, grads, exp_avg, exp_avg_sq, masters, exp_avg_scales, exp_avg_sq_scales)]
    if not any(lists):
        return
    if _fns is None:
        _lib()
    if _ops._bind is None:
        _ops._load_bind()
    first = next(v[0] for v in lists if v)
    dev = _device(first, "the first tensor")
    code = _ops._bind.adamw(_adamw_address, *lists, step, lr, betas[0], betas[1], eps, weight_decay, norm, max_norm, dev,
                            _current_stream(dev) if stream is None else _stream(stream))
    if code:
        raise TGError("tg_adamw", code)
