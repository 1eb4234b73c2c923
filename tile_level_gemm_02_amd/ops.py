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

import array
import ctypes

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


def _act(name: str) -> int:
    try:
        return ACTS[name]
    except KeyError:
        raise ValueError(f"unknown activation {name!r}: one of {', '.join(ACTS)}") from None


def _mat(t, name: str, rows: int, cols: int, dtypes):
    """(pointer, leading dimension) of a rows x cols matrix of one of `dtypes`."""
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if t.shape != (rows, cols):
        raise ValueError(f"{name} must be {rows}x{cols}, got shape {tuple(t.shape)}")
    s = t.stride()
    if cols > 1 and s[1] != 1:
        raise ValueError(f"{name} must have unit stride along its last dimension")
    return t.data_ptr(), (s[0] if rows > 1 else max(s[0], cols))


def _opt(t, name: str, rows: int, cols: int, dtypes):
    return (None, 0) if t is None else _mat(t, name, rows, cols, dtypes)


def _2d(t, name: str):
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D, got shape {tuple(t.shape)}")
    return t.shape


def _vec(t, name: str, n: int):
    if t is None:
        return None
    if t.dtype != torch.float32 or t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 vector of {n}")
    return t.data_ptr()


def _ws(workspace):
    if workspace is None:
        return None, 0
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _on_device(*tensors) -> None:
    """Every tensor given is on the current GPU."""
    want = torch.cuda.current_device() if torch.cuda.is_available() else -2
    for t in tensors:
        if t is not None and t.get_device() != want:
            raise ValueError(f"every tensor must be on the current GPU, got one on {t.device}")


def _call(name: str, *args) -> None:
    code = getattr(_fns, name)(*args)
    if code:
        raise TGError(name, code)


def _input(x, what: str) -> int:
    try:
        return _IN[x.dtype]
    except KeyError:
        raise ValueError(f"{what} takes float16, bfloat16 or float8_e4m3fn inputs, got {x.dtype}") from None


def _input16(x, what: str) -> int:
    if x.dtype not in (torch.float16, torch.bfloat16):
        raise ValueError(f"{what} takes float16 or bfloat16 inputs, got {x.dtype}")
    return _IN[x.dtype]


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
    _lib()
    i = _input(x, "tg_linear")
    M, K = _2d(x, "x")
    N = _2d(W, "W")[0]
    a = _act(act)
    own = (x.dtype,)
    px, ldx = _mat(x, "x", M, K, own)
    pw, ldw = _mat(W, "W", N, K, own)
    out = _CDTYPE if i == 2 else (torch.float32, x.dtype)
    py, ldy = _mat(Y, "Y", M, N, out)
    like = (Y.dtype,)
    pr, ldr = _opt(residual, "residual", M, N, like)
    pz, ldz = _opt(preact, "preact", M, N, like)
    pb = _vec(bias, "bias", N)
    _on_device(x, W, Y, bias, residual, preact, workspace)
    _call("tg_linear", i, M, N, K, px, ldx, pw, ldw, pb, a, pr, ldr, scale_x, scale_w, py, ldy, _CDTYPE[Y.dtype], pz, ldz,
          *_ws(workspace), _stream(stream))


def tg_linear_backward(dY, x, W, dx=None, dw=None, dbias=None, preact=None, act: str = "none", dz=None, workspace=None,
                       stream=None) -> None:
    """dz = dY * act'(preact); dx = dz . W; dw = dz^T . x; dbias = column sums of dz.

    Each output that is given is written.  With an activation ``dz`` is a
    buffer like dY (dY itself may serve); without one dz is dY, and
    ``preact`` and ``dz`` are not looked at."""
    _lib()
    i = _input16(dY, "tg_linear_backward")
    M, N = _2d(dY, "dY")
    K = _2d(x, "x")[1]
    a = _act(act)
    own = (dY.dtype,)
    pd, ldd = _mat(dY, "dY", M, N, own)
    px, ldx = _mat(x, "x", M, K, own)
    pw, ldw = _mat(W, "W", N, K, own)
    if a == 0:
        preact = dz = None
    elif preact is None or dz is None:
        raise ValueError("an activation's gradient needs preact and a dz buffer")
    pz, ldz = _opt(preact, "preact", M, N, own)
    pq, ldq = _opt(dz, "dz", M, N, own)
    pdx, lddx = _opt(dx, "dx", M, K, own)
    pdw, lddw = _opt(dw, "dw", N, K, (torch.float32, dY.dtype))
    pb = _vec(dbias, "dbias", N)
    _on_device(dY, x, W, preact, dz, dx, dw, dbias, workspace)
    _call("tg_linear_backward", i, M, N, K, pd, ldd, px, ldx, pw, ldw, pz, ldz, a, pq, ldq, pdx, lddx, pdw, lddw,
          0 if dw is None else _CDTYPE[dw.dtype], pb, *_ws(workspace), _stream(stream))


def tg_glu(x, W, H, act: str = "silu", gate_up=None, scale_x: float = 1.0, scale_w: float = 1.0, workspace=None,
           stream=None) -> None:
    """H = act(g) * u with [g | u] = scale_x scale_w x . W^T, W = [Wg; Wu] (2F x D); [g | u] is kept in ``gate_up`` if given."""
    _lib()
    i = _input(x, "tg_glu")
    M, D = _2d(x, "x")
    F = _2d(H, "H")[1]
    a = _act(act)
    own = (x.dtype,)
    px, ldx = _mat(x, "x", M, D, own)
    pw, ldw = _mat(W, "W", 2 * F, D, own)
    ph, ldh = _mat(H, "H", M, F, (torch.float16, torch.bfloat16) if i == 2 else own)
    pg, ldg = _opt(gate_up, "gate_up", M, 2 * F, (H.dtype,))
    _on_device(x, W, H, gate_up, workspace)
    _call("tg_glu", i, M, F, D, px, ldx, pw, ldw, a, scale_x, scale_w, ph, ldh, _CDTYPE[H.dtype], pg, ldg,
          *_ws(workspace), _stream(stream))


def tg_glu_backward(dY, Wd, x, W, gate_up, H, dgate_up, dx=None, dw_gate_up=None, dw_down=None, act: str = "silu",
                    workspace=None, stream=None) -> None:
    """Gradients of y = H . Wd^T, H = act(g) * u, [g | u] = x . W^T.

    ``dgate_up`` (M x 2F, may be gate_up itself) receives [dg | du]; each of
    dx, dw_gate_up (2F x D) and dw_down (D x F) that is given is written.
    ``H`` may be None where dw_down is."""
    _lib()
    i = _input16(dY, "tg_glu_backward")
    M, D = _2d(dY, "dY")
    F = _2d(Wd, "Wd")[1]
    a = _act(act)
    own = (dY.dtype,)
    args = []
    for t, name, rows, cols in ((dY, "dY", M, D), (Wd, "Wd", D, F), (x, "x", M, D), (W, "W", 2 * F, D),
                                (gate_up, "gate_up", M, 2 * F)):
        args += _mat(t, name, rows, cols, own)
    if H is None and dw_down is not None:
        raise ValueError("dw_down needs H")
    args += _opt(H, "H", M, F, own)
    args.append(a)
    args += _mat(dgate_up, "dgate_up", M, 2 * F, own)
    args += _opt(dx, "dx", M, D, own)
    out = (torch.float32, dY.dtype)
    args += _opt(dw_gate_up, "dw_gate_up", 2 * F, D, out)
    args += _opt(dw_down, "dw_down", D, F, out)
    given = {t.dtype for t in (dw_gate_up, dw_down) if t is not None}
    if len(given) > 1:
        raise ValueError("dw_gate_up and dw_down must have one type")
    _on_device(dY, Wd, x, W, gate_up, H, dgate_up, dx, dw_gate_up, dw_down, workspace)
    _call("tg_glu_backward", i, M, F, D, *args, _CDTYPE[given.pop()] if given else 0, *_ws(workspace), _stream(stream))


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
    _lib()
    grads = list(grads)
    count = len(grads)
    outs = grads if out is None else list(out)
    if len(outs) != count:
        raise ValueError(f"out must hold {count} tensors, got {len(outs)}")
    try:
        types = array.array("i", [_CDTYPE[g.dtype] for g in grads])
    except KeyError as e:
        raise ValueError(f"unsupported gradient dtype {e.args[0]}") from None
    sizes = array.array("q", [g.numel() for g in grads])
    pin = array.array("Q", [g.data_ptr() for g in grads])
    pout = pin
    for g in grads:
        if not g.is_contiguous():
            raise ValueError("gradients must be contiguous")
    if out is not None:
        for g, o in zip(grads, outs):
            if o.dtype != g.dtype or o.shape != g.shape or not o.is_contiguous():
                raise ValueError("each out must be a contiguous tensor like its gradient")
        pout = array.array("Q", [o.data_ptr() for o in outs])
    if norm is not None and (norm.dtype != torch.float32 or norm.numel() != 1):
        raise ValueError("norm must be a float32 tensor of one element")
    if workspace is None:
        raise ValueError("tg_clip_grads needs a workspace")
    _on_device(workspace, norm, *grads, *(outs if out is not None else ()))
    _call("tg_clip_grads", count, pin.buffer_info()[0], pout.buffer_info()[0], sizes.buffer_info()[0],
          types.buffer_info()[0], max_norm, eps, None if norm is None else norm.data_ptr(), *_ws(workspace),
          _stream(stream))
