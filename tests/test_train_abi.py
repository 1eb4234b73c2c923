"""The training operators' and the 8-bit integer layers' C ABI and binding:
every declared symbol is exported, and wrong arguments are refused before any
HIP call (CPU only: nothing here launches)."""
import ctypes
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 0x10000  # a fake aligned device address: never dereferenced on these paths
W = 1 << 20  # a fake workspace
BIG = 1 << 40


@pytest.fixture(scope="module")
def tg():
    import tile_level_gemm_02_amd as tg

    return tg


@pytest.mark.parametrize("header,module", [("tg_train.h", "train"), ("tg_int8.h", "int8")])
def test_every_declared_symbol_is_exported_and_bound(tg, header, module):
    import importlib

    m = importlib.import_module(f"tile_level_gemm_02_amd.{module}")
    src = open(os.path.join(ROOT, "include", header)).read()
    declared = set(re.findall(r"^(?:tg_status|int64_t) (tg_[a-z0-9_]+)\(", src, re.M))
    assert declared == set(m.EXPORTS)
    raw = ctypes.CDLL(tg.LIB_PATH)
    for name in declared:
        assert hasattr(raw, name) and hasattr(tg, name), name


@pytest.fixture(scope="module")
def train(tg):
    from tile_level_gemm_02_amd import train

    return train._lib()


@pytest.fixture(scope="module")
def int8(tg):
    from tile_level_gemm_02_amd import int8

    return int8._lib()


def test_loss_refusals(tg, train):
    inv, mis, nos = tg.TG_ERR_INVALID_VALUE, tg.TG_ERR_MISALIGNED, tg.TG_ERR_NOT_SUPPORTED

    def call(i=1, M=8, V=8, D=8, x=A, ldx=8, w=A, ldw=8, s=1.0, t=A, ig=-100, z=0.0, loss=A, lse=A, total=A, ws=W, nb=BIG):
        return train.tg_linear_xent(i, M, V, D, x, ldx, w, ldw, s, t, ig, z, loss, lse, total, ws, nb, None)

    need = train.tg_linear_xent_workspace_bytes(1, 8, 8, 8)
    for bad in (dict(M=-1), dict(V=-1), dict(D=-1), dict(i=3), dict(i=-1), dict(x=None), dict(w=None), dict(t=None), dict(V=0), dict(ldx=7),
                dict(ldw=7), dict(s=float("inf")), dict(z=float("nan")), dict(ws=None, nb=0), dict(nb=need - 1), dict(nb=-1),
                dict(M=0, ws=None, nb=0), dict(M=0, nb=65536)):
        assert call(**bad) == inv, bad
    for bad in (dict(x=A + 8), dict(w=A + 2), dict(ldx=12), dict(t=A + 4), dict(loss=A + 2), dict(lse=A + 1), dict(total=A + 2), dict(ws=W + 64)):
        assert call(**bad) == mis, bad
    for bad in (dict(i=2), dict(D=12, ldx=16, ldw=16), dict(M=1 << 31), dict(ldx=1 << 31), dict(ldx=1 << 23), dict(ldw=1 << 23)):
        assert call(**bad) == nos, bad
    assert call(M=0, x=None, w=None, t=None, total=None, ws=None, nb=0) == tg.TG_OK


def test_loss_gradient_refusals(tg, train):
    inv, mis, nos = tg.TG_ERR_INVALID_VALUE, tg.TG_ERR_MISALIGNED, tg.TG_ERR_NOT_SUPPORTED

    def call(i=1, M=8, V=8, D=8, x=A, ldx=8, w=A, ldw=8, s=1.0, t=A, ig=-100, z=0.0, lse=A, dl=A, gs=1.0, total=A, dx=A, lddx=8, dw=A, lddw=8,
             od=2, ws=W, nb=BIG):
        return train.tg_linear_xent_backward(i, M, V, D, x, ldx, w, ldw, s, t, ig, z, lse, dl, gs, total, dx, lddx, dw, lddw, od, ws, nb, None)

    need = train.tg_linear_xent_backward_workspace_bytes(1, 8, 8, 8, 1)
    for bad in (dict(M=-1), dict(V=-1), dict(i=5), dict(od=3), dict(od=-1), dict(x=None), dict(w=None), dict(t=None), dict(lse=None), dict(V=0),
                dict(ldx=4), dict(ldw=4), dict(lddx=4), dict(lddw=4), dict(s=float("nan")), dict(gs=float("inf")), dict(z=float("inf")),
                dict(ws=None, nb=0), dict(nb=need - 1), dict(nb=-1)):
        assert call(**bad) == inv, bad
    for bad in (dict(x=A + 8), dict(dx=A + 2), dict(dw=A + 8), dict(lddx=12), dict(t=A + 4), dict(lse=A + 2), dict(dl=A + 1), dict(total=A + 2),
                dict(ws=W + 128)):
        assert call(**bad) == mis, bad
    for bad in (dict(i=2), dict(od=1), dict(i=0, od=2), dict(D=12, ldx=16, ldw=16, lddx=16, lddw=16), dict(V=1 << 31), dict(lddw=1 << 31),
                dict(ldw=1 << 23)):
        assert call(**bad) == nos, bad
    assert call(dx=None, dw=None, ws=None, nb=0) == tg.TG_OK  # nothing asked for
    assert call(dx=None, dw=None, lse=None) == tg.TG_OK
    assert call(M=0, x=None, w=None, t=None, lse=None, dw=None) == tg.TG_OK


def test_loss_workspace_queries(tg):
    bf = torch.bfloat16
    for M, V, D in ((1, 1, 8), (7, 32000, 2048), (160, 452, 1256), (4096, 128256, 4096), (100000, 200000, 1024), (2000000, 1000, 64)):
        n = [tg.tg_linear_xent_backward_workspace_bytes(bf, M, V, D, p) for p in (1, 256, 257, 4096, 0)]
        assert 0 < n[0] == n[1] <= n[2] and n[1] <= n[4] and n[3] <= n[4], (M, V, D, n)
        assert n[4] <= (128 << 20) + (1 << 20) + M * (16 + 4 * D) + max(512 << 20, 2 * 8192 * M), (M, V, D, n)
        f = tg.tg_linear_xent_workspace_bytes(bf, M, V, D)
        assert 65536 < f <= 65536 + M * (V // 8 + 40) * (4 if M <= 32 else 1) + 4096, (M, V, D, f)
    for q in (lambda *a: tg.tg_linear_xent_workspace_bytes(*a), lambda *a: tg.tg_linear_xent_backward_workspace_bytes(*a)):
        with pytest.raises(ValueError):
            q(bf, -1, 8, 8)
        with pytest.raises(ValueError):
            q(torch.float32, 8, 8, 8)
        with pytest.raises(ValueError):
            q(torch.float8_e4m3fn, 8, 8, 8)
    with pytest.raises(ValueError):
        tg.tg_linear_xent_backward_workspace_bytes(bf, 8, 8, 8, -1)


class _T(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("p", "w", "g", "m", "v", "sm", "sv")] + [("n", ctypes.c_int64), ("pt", ctypes.c_int32), ("gt", ctypes.c_int32)]


def test_adamw_refusals(tg, train):
    inv, mis = tg.TG_ERR_INVALID_VALUE, tg.TG_ERR_MISALIGNED

    def call(count=2, step=1, lr=1e-3, b1=0.9, b2=0.99, eps=1e-8, wd=0.1, norm=A, most=1.0, sd=None, ld=None, none=False, **t):
        one = dict(p=A, w=None, g=A, m=A, v=A, sm=None, sv=None, n=4, pt=2, gt=0) | t
        ts = (_T * 2)(_T(**(one | dict(n=0))), _T(**one))
        return train.tg_adamw(count, None if none else ctypes.byref(ts), step, lr, b1, b2, eps, wd, norm, most, sd, ld, None)

    nan, inf = float("nan"), float("inf")
    for bad in (dict(count=-1), dict(none=True), dict(step=0), dict(lr=nan), dict(lr=inf), dict(b1=1.0), dict(b1=-0.1), dict(b2=1.0), dict(b2=nan),
                dict(eps=-1.0), dict(eps=inf), dict(wd=nan), dict(most=-1.0), dict(most=nan), dict(n=-1), dict(pt=3), dict(gt=-1), dict(p=None),
                dict(g=None), dict(m=None), dict(v=None), dict(sm=A), dict(sv=A), dict(w=A, pt=0)):
        assert call(**bad) == inv, bad
    for bad in (dict(norm=A + 2), dict(sd=A + 4), dict(ld=A + 2), dict(p=A + 1), dict(g=A + 2), dict(m=A + 2), dict(v=A + 1), dict(w=A + 2),
                dict(sm=A + 2, sv=A), dict(sm=A, sv=A + 1)):
        assert call(**bad) == mis, bad
    # fp32 states beside 8-bit ones
    ts = (_T * 2)(_T(A, None, A, A, A, A, A, 4, 2, 0), _T(A, None, A, A, A, None, None, 4, 2, 0))
    assert train.tg_adamw(2, ctypes.byref(ts), 1, 1e-3, 0.9, 0.99, 1e-8, 0.1, None, 1.0, None, None, None) == inv
    assert call(n=0, p=None, g=None) == tg.TG_OK and call(count=0) == tg.TG_OK and call(count=0, none=True) == tg.TG_OK


def test_int8_refusals(tg, int8):
    inv, mis, nos = tg.TG_ERR_INVALID_VALUE, tg.TG_ERR_MISALIGNED, tg.TG_ERR_NOT_SUPPORTED

    def quant(t=2, M=8, K=16, x=A, ldx=16, q=A, ldq=16, s=A):
        return int8.tg_quantize_i8(t, M, K, x, ldx, q, ldq, s, None)

    for bad in (dict(t=3), dict(t=-1), dict(M=-1), dict(K=-1), dict(x=None), dict(q=None), dict(s=None), dict(ldx=8), dict(ldq=8)):
        assert quant(**bad) == inv, bad
    for bad in (dict(x=A + 2), dict(q=A + 8), dict(s=A + 2), dict(ldx=20), dict(ldq=24)):
        assert quant(**bad) == mis, bad
    assert quant(M=1 << 31) == nos and quant(M=0, x=None, q=None, s=None) == tg.TG_OK

    def call(M=8, N=8, K=16, x=A, ldx=16, w=A, ldw=16, sx=A, sw=A, b=None, act=0, r=None, ldr=8, y=A, ldy=8, od=2, ws=None, nb=0):
        return int8.tg_linear_i8(M, N, K, x, ldx, w, ldw, sx, sw, b, act, r, ldr, y, ldy, od, ws, nb, None)

    for bad in (dict(M=-1), dict(act=5), dict(act=-1), dict(od=3), dict(od=-1), dict(x=None), dict(w=None), dict(y=None), dict(sx=None),
                dict(sw=None), dict(ldx=8), dict(ldw=8), dict(ldy=7), dict(r=A, ldr=4), dict(nb=-1), dict(nb=256),
                dict(M=256, N=512, K=8192, ldx=8192, ldw=8192, ldy=512, ws=W, nb=65536)):
        assert call(**bad) == inv, bad
    for bad in (dict(x=A + 8), dict(w=A + 4), dict(y=A + 8), dict(ldx=24), dict(ldw=17), dict(ldy=9), dict(sx=A + 2), dict(sw=A + 1), dict(b=A + 2),
                dict(r=A + 8), dict(r=A, ldr=12), dict(ws=W + 64, nb=BIG)):
        assert call(**bad) == mis, bad
    for bad in (dict(K=8), dict(K=24, ldx=32, ldw=32), dict(K=131072, ldx=131072, ldw=131072), dict(N=1 << 31), dict(ldr=1 << 31)):
        assert call(**bad) == nos, bad
    assert call(M=0, x=None, w=None, y=None, sx=None, sw=None) == tg.TG_OK and call(N=0, x=None, w=None, y=None, sw=None) == tg.TG_OK
    for M, N, K in ((1, 4096, 4096), (16, 512, 8192), (256, 8192, 8192), (300, 900, 8208), (100, 7, 9)):
        assert 0 <= tg.tg_linear_i8_workspace_bytes(M, N, K) <= (64 << 20) + (64 << 10)
    with pytest.raises(ValueError):
        tg.tg_linear_i8_workspace_bytes(1, -1, 16)


def test_binding_refuses_wrong_tensors(tg):
    """Shapes, types, strides and devices are checked before the library is called."""
    t = torch.zeros
    bf, i8 = torch.bfloat16, torch.int8
    x, w, target, lse = t(4, 16, dtype=bf), t(8, 16, dtype=bf), t(4, dtype=torch.int64), t(4)

    def no(fn, *a, **k):
        with pytest.raises(ValueError):
            fn(*a, **k)

    no(tg.tg_linear_xent, x, w, target, lse)  # not on the GPU
    no(tg.tg_linear_xent, x.float(), w.float(), target)
    no(tg.tg_linear_xent, x, w.half(), target)
    no(tg.tg_linear_xent, x, w[:, :8], target)
    no(tg.tg_linear_xent, x, w, target.int())
    no(tg.tg_linear_xent, x, w, target[:3])
    no(tg.tg_linear_xent, t(16, dtype=bf), w, target)
    no(tg.tg_linear_xent_backward, x, w, target, lse)
    no(tg.tg_linear_xent_backward, x, w, target, lse.double())
    no(tg.tg_linear_xent_backward, x.to(torch.float8_e4m3fn), w, target, lse)
    q, wq, s = t(4, 16, dtype=i8), t(8, 16, dtype=i8), t(8)
    no(tg.tg_quantize_i8, x, q, lse)
    no(tg.tg_quantize_i8, x.double(), q, lse)
    no(tg.tg_quantize_i8, t(16), q, lse)
    no(tg.tg_linear_i8, q, wq, t(4, 8), lse, s)
    no(tg.tg_linear_i8, x, wq, t(4, 8), lse, s)
    no(tg.tg_linear_i8, q, wq, t(4, 8), lse, s, act="tanh")
    no(tg.tg_linear_i8, q, t(16, dtype=i8), t(4, 8), lse, s)
    no(tg.tg_adamw, [s], [s], [s], [s], 1, 1e-3)  # not on the GPU
    tg.tg_adamw([], [], [], [], 1, 1e-3)
