"""Binding of the feed-forward operators declared in include/tg_ops.h.

    tg_linear(x, W, Y, bias=None, act="none", residual=None, preact=None, ...)
    tg_linear_backward(dY, x, W, dx=None, dw=None, dbias=None, preact=None, act="none", dz=None, ...)
    tg_glu(x, W, H, act="silu", gate_up=None, ...)
    tg_glu_backward(dY, Wd, x, W, gate_up, H, dgate_up, dx=None, dw_gate_up=None, dw_down=None, act="silu", ...)
    tg_clip_grads(grads, max_norm, out=None, norm=None, eps=1e-6, ...)
    tg_linear_workspace_bytes(dtype, M, N, K), tg_linear_backward_workspace_bytes, tg_glu_workspace_bytes,
    tg_glu_backward_workspace_bytes, tg_clip_grads_workspace_bytes(count), tg_ops_workspace()

Activations are "none", "relu", "gelu", "gelu_tanh" and "silu".  Outputs are
tensors of the caller's; None leaves an optional one out.  ``workspace`` is
the split workspace of ``tg_gemm_ex`` (``tg_ops_workspace()`` makes one that
serves every call).  Wrong shapes, types or devices raise ValueError before
anything is launched, what the library itself refuses raises TGError.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os

import torch

from . import _CDTYPE, _IN, TGError, _stream, load

ACTS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}

EXPORTS = ("tg_linear", "tg_linear_workspace_bytes", "tg_linear_backward", "tg_linear_backward_workspace_bytes",
           "tg_glu", "tg_glu_workspace_bytes", "tg_glu_backward", "tg_glu_backward_workspace_bytes",
           "tg_clip_grads", "tg_clip_grads_workspace_bytes")

# a workspace of this size serves every call of the library: 64 KiB of
# counters and one round of 256 x 256 fp32 partial tiles
WORKSPACE_BYTES = (64 << 20) + (64 << 10)

_fns = None
_bind = None          # the native helper _tgbind.so of tg_clip_grads
_clip_address = 0     # of tg_clip_grads in the loaded library
_BIND_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_tgbind.so")


def _load_bind():
    """The helper, loaded by the first call that needs it (tg_clip_grads, tg_adamw, the int8 layers): the other products do without."""
    global _bind, _clip_address
    if not os.path.exists(_BIND_PATH):
        raise ImportError(f"{_BIND_PATH}, which tg_clip_grads, tg_adamw and the int8 layers need, is not built; run `python -m tile_level_gemm_02_amd.build`")
    loader = importlib.machinery.ExtensionFileLoader("_tgbind", _BIND_PATH)
    module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_tgbind", loader))
    loader.exec_module(module)
    _clip_address = ctypes.cast(_lib().tg_clip_grads, ctypes.c_void_p).value
    _bind = module


def _lib():
    """The library with the argument types of these entry points set."""
    global _fns
    if _fns is None:
        lib = load()
        i64, vp, f32, ci = ctypes.c_int64, ctypes.c_void_p, ctypes.c_float, ctypes.c_int
        mat, ws = [vp, i64], [vp, i64, vp]
        args = {
            "tg_linear": [ci, i64, i64, i64, *mat, *mat, vp, ci, *mat, f32, f32, *mat, ci, *mat, *ws],
            "tg_linear_backward": [ci, i64, i64, i64, *mat, *mat, *mat, *mat, ci, *mat, *mat, *mat, ci, vp, *ws],
            "tg_glu": [ci, i64, i64, i64, *mat, *mat, ci, f32, f32, *mat, ci, *mat, *ws],
            "tg_glu_backward": [ci, i64, i64, i64, *mat, *mat, *mat, *mat, *mat, *mat, ci, *mat, *mat, *mat, *mat, ci,
                                *ws],
            "tg_clip_grads": [i64, vp, vp, vp, vp, f32, f32, vp, *ws],
        }
        for name, types in args.items():
            fn = getattr(lib, name)
            fn.argtypes, fn.restype = types, ci
        for name in ("tg_linear", "tg_linear_backward", "tg_glu", "tg_glu_backward"):
            fn = getattr(lib, name + "_workspace_bytes")
            fn.argtypes, fn.restype = [ci, i64, i64, i64], i64
        lib.tg_clip_grads_workspace_bytes.argtypes = [i64]
        lib.tg_clip_grads_workspace_bytes.restype = i64
        _fns = lib
    return _fns


# ------------------------------------------------------------- marshalling
#
# A small product's kernel runs in 5 to 10 us, so a call's marshalling is kept
# near that: each tensor attribute is read once (about 0.1 us each), and the
# current device and stream are read without torch.cuda's wrappers.


def _act(name: str) -> int:
    try:
        return ACTS[name]
    except KeyError:
        raise ValueError(f"unknown activation {name!r}: one of {', '.join(ACTS)}") from None


def _mat(t, name: str, rows: int, cols: int, dtypes, dev: int):
    """(pointer, leading dimension) of a rows x cols matrix of one of `dtypes` on GPU `dev`."""
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if t.shape != (rows, cols):
        raise ValueError(f"{name} must be {rows}x{cols}, got shape {tuple(t.shape)}")
    ld, unit = t.stride()
    if unit != 1 and cols > 1:
        raise ValueError(f"{name} must have unit stride along its last dimension")
    if t.get_device() != dev:
        raise ValueError(f"every tensor must be on the current GPU, {name} is on {t.device}")
    # one row has no second one: its stride is not looked at, an aligned one stands for it
    return t.data_ptr(), (ld if rows > 1 else cols + 15 & -16)


_NONE = (None, 0)


def _2d(t, name: str):
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be 2-D, got shape {tuple(shape)}")
    return shape


def _vec(t, name: str, n: int, dev: int):
    if t.dtype != torch.float32 or t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 vector of {n}")
    if t.get_device() != dev:
        raise ValueError(f"every tensor must be on the current GPU, {name} is on {t.device}")
    return t.data_ptr()


def _ws(workspace, dev: int):
    if workspace is None:
        return _NONE
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    if workspace.get_device() != dev:
        raise ValueError(f"every tensor must be on the current GPU, the workspace is on {workspace.device}")
    return workspace.data_ptr(), workspace.nbytes


_current_device = torch._C._cuda_getDevice
_current_stream = torch._C._cuda_getCurrentRawStream


def _device(t, name: str) -> int:
    """The index of the current GPU, which `t` has to be on."""
    dev = t.get_device()
    if dev < 0 or dev != _current_device():
        raise ValueError(f"every tensor must be on the current GPU, {name} is on {t.device}")
    return dev


def _input(x, what: str) -> int:
    try:
        return _IN[x.dtype]
    except KeyError:
        raise ValueError(f"{what} takes float16, bfloat16 or float8_e4m3fn inputs, got {x.dtype}") from None


def _input16(x, what: str) -> int:
    if x.dtype not in _16BIT:
        raise ValueError(f"{what} takes float16 or bfloat16 inputs, got {x.dtype}")
    return _IN[x.dtype]


_16BIT = (torch.float16, torch.bfloat16)
_OWN = {d: (d,) for d in (*_CDTYPE, *_IN)}
_OWN_OR_F32 = {d: (torch.float32, d) for d in _16BIT}
_OWN_OR_F32[torch.float8_e4m3fn] = tuple(_CDTYPE)


def _bytes(name: str, dtype, *sizes: int) -> int:
    if dtype not in _IN:
        raise ValueError(f"unsupported input dtype {dtype}")
    n = int(getattr(_lib(), name)(_IN[dtype], *(int(s) for s in sizes)))
    if n < 0:
        raise ValueError("invalid sizes")
    return n


# ---------------------------------------------------------------- products


def tg_linear_workspace_bytes(dtype, M: int, N: int, K: int) -> int:
    """Workspace bytes tg_linear can use for this problem (0: it never splits)."""
    return _bytes("tg_linear_workspace_bytes", dtype, M, N, K)


def tg_linear_backward_workspace_bytes(dtype, M: int, N: int, K: int) -> int:
    """Workspace bytes tg_linear_backward can use for this problem."""
    return _bytes("tg_linear_backward_workspace_bytes", dtype, M, N, K)


def tg_glu_workspace_bytes(dtype, M: int, F: int, D: int) -> int:
    """Workspace bytes tg_glu can use for this problem."""
    return _bytes("tg_glu_workspace_bytes", dtype, M, F, D)


def tg_glu_backward_workspace_bytes(dtype, M: int, F: int, D: int) -> int:
    """Workspace bytes tg_glu_backward can use for this problem."""
    return _bytes("tg_glu_backward_workspace_bytes", dtype, M, F, D)


def tg_ops_workspace(device="cuda"):
    """A zeroed workspace tensor that serves every call of the library (one per stream that calls)."""
    return torch.zeros(WORKSPACE_BYTES // 4, dtype=torch.int32, device=device)


def tg_linear(x, W, Y, bias=None, act: str = "none", residual=None, preact=None, scale_x: float = 1.0,
              scale_w: float = 1.0, workspace=None, stream=None) -> None:
    """Y = act(z) + residual, z = scale_x scale_w x . W^T + bias; z is kept in ``preact`` if given."""
    i = _input(x, "tg_linear")
    M, K = _2d(x, "x")
    N = _2d(W, "W")[0]
    a = _act(act)
    dev = _device(x, "x")
    own = _OWN[x.dtype]
    px, ldx = _mat(x, "x", M, K, own, dev)
    pw, ldw = _mat(W, "W", N, K, own, dev)
    py, ldy = _mat(Y, "Y", M, N, _OWN_OR_F32[x.dtype], dev)
    yt = Y.dtype
    pr, ldr = _NONE if residual is None else _mat(residual, "residual", M, N, _OWN[yt], dev)
    pz, ldz = _NONE if preact is None else _mat(preact, "preact", M, N, _OWN[yt], dev)
    pb = None if bias is None else _vec(bias, "bias", N, dev)
    ps, ns = _ws(workspace, dev)
    code = (_fns or _lib()).tg_linear(i, M, N, K, px, ldx, pw, ldw, pb, a, pr, ldr, scale_x, scale_w, py, ldy, _CDTYPE[yt],
                                      pz, ldz, ps, ns, _current_stream(dev) if stream is None else _stream(stream))
    if code:
        raise TGError("tg_linear", code)


def tg_linear_backward(dY, x, W, dx=None, dw=None, dbias=None, preact=None, act: str = "none", dz=None, workspace=None,
                       stream=None) -> None:
    """dz = dY * act'(preact); dx = dz . W; dw = dz^T . x; dbias = column sums of dz.

    Each output that is given is written.  With an activation ``dz`` is a
    buffer like dY (dY itself may serve); without one dz is dY, and
    ``preact`` and ``dz`` are not looked at."""
    i = _input16(dY, "tg_linear_backward")
    M, N = _2d(dY, "dY")
    K = _2d(x, "x")[1]
    a = _act(act)
    if a == 0:
        preact = dz = None
    elif preact is None or dz is None:
        raise ValueError("an activation's gradient needs preact and a dz buffer")
    dev = _device(dY, "dY")
    t = dY.dtype
    own = _OWN[t]
    pd, ldd = _mat(dY, "dY", M, N, own, dev)
    px, ldx = _mat(x, "x", M, K, own, dev)
    pw, ldw = _mat(W, "W", N, K, own, dev)
    pz, ldz = _NONE if preact is None else _mat(preact, "preact", M, N, own, dev)
    pq, ldq = _NONE if dz is None else _mat(dz, "dz", M, N, own, dev)
    pdx, lddx = _NONE if dx is None else _mat(dx, "dx", M, K, own, dev)
    pdw, lddw = _NONE if dw is None else _mat(dw, "dw", N, K, _OWN_OR_F32[t], dev)
    pb = None if dbias is None else _vec(dbias, "dbias", N, dev)
    ps, ns = _ws(workspace, dev)
    code = (_fns or _lib()).tg_linear_backward(
        i, M, N, K, pd, ldd, px, ldx, pw, ldw, pz, ldz, a, pq, ldq, pdx, lddx, pdw, lddw,
        0 if dw is None else _CDTYPE[dw.dtype], pb, ps, ns, _current_stream(dev) if stream is None else _stream(stream))
    if code:
        raise TGError("tg_linear_backward", code)


def tg_glu(x, W, H, act: str = "silu", gate_up=None, scale_x: float = 1.0, scale_w: float = 1.0, workspace=None,
           stream=None) -> None:
    """H = act(g) * u with [g | u] = scale_x scale_w x . W^T, W = [Wg; Wu] (2F x D); [g | u] is kept in ``gate_up`` if given."""
    i = _input(x, "tg_glu")
    M, D = _2d(x, "x")
    F = _2d(H, "H")[1]
    a = _act(act)
    dev = _device(x, "x")
    own = _OWN[x.dtype]
    px, ldx = _mat(x, "x", M, D, own, dev)
    pw, ldw = _mat(W, "W", 2 * F, D, own, dev)
    ph, ldh = _mat(H, "H", M, F, _16BIT if i == 2 else own, dev)
    ht = H.dtype
    pg, ldg = _NONE if gate_up is None else _mat(gate_up, "gate_up", M, 2 * F, _OWN[ht], dev)
    ps, ns = _ws(workspace, dev)
    code = (_fns or _lib()).tg_glu(i, M, F, D, px, ldx, pw, ldw, a, scale_x, scale_w, ph, ldh, _CDTYPE[ht], pg, ldg, ps, ns,
                                   _current_stream(dev) if stream is None else _stream(stream))
    if code:
        raise TGError("tg_glu", code)


def tg_glu_backward(dY, Wd, x, W, gate_up, H, dgate_up, dx=None, dw_gate_up=None, dw_down=None, act: str = "silu",
                    workspace=None, stream=None) -> None:
    """Gradients of y = H . Wd^T, H = act(g) * u, [g | u] = x . W^T.

    ``dgate_up`` (M x 2F, may be gate_up itself) receives [dg | du]; each of
    dx, dw_gate_up (2F x D) and dw_down (D x F) that is given is written.
    ``H`` may be None where dw_down is."""
    i = _input16(dY, "tg_glu_backward")
    M, D = _2d(dY, "dY")
    F = _2d(Wd, "Wd")[1]
    a = _act(act)
    if H is None and dw_down is not None:
        raise ValueError("dw_down needs H")
    if dw_gate_up is not None and dw_down is not None and dw_gate_up.dtype != dw_down.dtype:
        raise ValueError("dw_gate_up and dw_down must have one type")
    dev = _device(dY, "dY")
    t = dY.dtype
    own, out = _OWN[t], _OWN_OR_F32[t]
    pd, ldd = _mat(dY, "dY", M, D, own, dev)
    pwd, ldwd = _mat(Wd, "Wd", D, F, own, dev)
    px, ldx = _mat(x, "x", M, D, own, dev)
    pw, ldw = _mat(W, "W", 2 * F, D, own, dev)
    pg, ldg = _mat(gate_up, "gate_up", M, 2 * F, own, dev)
    ph, ldh = _NONE if H is None else _mat(H, "H", M, F, own, dev)
    pq, ldq = _mat(dgate_up, "dgate_up", M, 2 * F, own, dev)
    pdx, lddx = _NONE if dx is None else _mat(dx, "dx", M, D, own, dev)
    pdw, lddw = _NONE if dw_gate_up is None else _mat(dw_gate_up, "dw_gate_up", 2 * F, D, out, dev)
    pdd, lddd = _NONE if dw_down is None else _mat(dw_down, "dw_down", D, F, out, dev)
    ps, ns = _ws(workspace, dev)
    wt = dw_gate_up if dw_gate_up is not None else dw_down
    code = (_fns or _lib()).tg_glu_backward(
        i, M, F, D, pd, ldd, pwd, ldwd, px, ldx, pw, ldw, pg, ldg, ph, ldh, a, pq, ldq, pdx, lddx, pdw, lddw, pdd, lddd,
        0 if wt is None else _CDTYPE[wt.dtype], ps, ns, _current_stream(dev) if stream is None else _stream(stream))
    if code:
        raise TGError("tg_glu_backward", code)


# ---------------------------------------------------------------- clipping


def tg_clip_grads_workspace_bytes(count: int) -> int:
    """Workspace bytes tg_clip_grads needs for `count` tensors (it is the same for any count)."""
    n = int(_lib().tg_clip_grads_workspace_bytes(int(count)))
    if n < 0:
        raise ValueError("invalid count")
    return n


def tg_clip_grads(grads, max_norm: float, out=None, norm=None, eps: float = 1e-6, workspace=None, stream=None) -> None:
    """out[i] = grads[i] * min(1, max_norm / (norm + eps)), norm = sqrt(sum of all squares).

    ``out`` None clips in place; ``norm`` (float32, one element) receives the
    norm before clipping.  Tensors are contiguous, of float32, float16 or
    bfloat16, mixed as they come.  Nothing is copied to the host."""
    if workspace is None:
        raise ValueError("tg_clip_grads needs a workspace")
    dev = _device(workspace, "the workspace")
    ps, ns = _ws(workspace, dev)
    if _bind is None:
        _load_bind()
    code = _bind.clip_grads(_clip_address, grads if type(grads) is list else list(grads),
                            out if out is None or type(out) is list else list(out), max_norm, eps, norm, dev, ps, ns,
                            _current_stream(dev) if stream is None else _stream(stream))
    if code:
        raise TGError("tg_clip_grads", code)
