"""The feed-forward operators' C ABI and binding: every declared symbol is
exported, and wrong arguments are refused before any HIP call (CPU only:
nothing here launches)."""
import ctypes
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 0x10000  # a fake aligned device address: never dereferenced on these paths
W = 1 << 20  # a fake workspace
BIG = (64 << 20) + (64 << 10)


@pytest.fixture(scope="module")
def tg():
    import tile_level_gemm_02_amd as tg

    return tg


@pytest.fixture(scope="module")
def lib(tg):
    from tile_level_gemm_02_amd import ops

    return ops._lib()


def test_every_declared_symbol_is_exported_and_bound(tg):
    from tile_level_gemm_02_amd import ops

    src = open(os.path.join(ROOT, "include", "tg_ops.h")).read()
    declared = set(re.findall(r"^(?:tg_status|int64_t) (tg_[a-z0-9_]+)\(", src, re.M))
    assert declared == set(ops.EXPORTS)
    raw = ctypes.CDLL(tg.LIB_PATH)
    for name in declared:
        assert hasattr(raw, name) and hasattr(tg, name), name


def test_linear_refusals(tg, lib):
    inv, mis, nos = tg.TG_ERR_INVALID_VALUE, tg.TG_ERR_MISALIGNED, tg.TG_ERR_NOT_SUPPORTED

    def call(i=1, M=8, N=8, K=8, x=A, ldx=8, w=A, ldw=8, b=None, act=0, r=None, ldr=8, sx=1.0, sw=1.0, y=A, ldy=8, od=2, z=None, ldz=8,
             ws=None, nb=0):
        return lib.tg_linear(i, M, N, K, x, ldx, w, ldw, b, act, r, ldr, sx, sw, y, ldy, od, z, ldz, ws, nb, None)

    for bad in (dict(M=-1), dict(i=3), dict(i=-1), dict(act=5), dict(act=-1), dict(od=3), dict(x=None), dict(w=None), dict(y=None),
                dict(ldx=7), dict(ldw=7), dict(ldy=7), dict(r=A, ldr=4), dict(z=A, ldz=4), dict(nb=-1), dict(nb=256),
                dict(i=2, ldx=16, ldw=16, sx=float("inf")), dict(i=2, ldx=16, ldw=16, sw=float("nan")),
                dict(M=256, N=8192, K=8192, ldx=8192, ldw=8192, ldy=8192, ws=W, nb=65536)):
        assert call(**bad) == inv, bad
    for bad in (dict(x=A + 8), dict(w=A + 2), dict(y=A + 4), dict(ldx=12), dict(ldy=12), dict(b=A + 2), dict(r=A + 8), dict(z=A + 8),
                dict(ldr=12, r=A), dict(ws=W + 64, nb=BIG), dict(i=2, ldx=8, ldw=16)):
        assert call(**bad) == mis, bad
    for bad in (dict(od=1), dict(i=0, od=2), dict(M=1 << 31), dict(ldx=1 << 31)):
        assert call(**bad) == nos, bad
    assert call(M=0, x=None, w=None, y=None) == tg.TG_OK and call(N=0, x=None, w=None, y=None) == tg.TG_OK


def test_linear_backward_refusals(tg, lib):
    inv, mis, nos = tg.TG_ERR_INVALID_VALUE, tg.TG_ERR_MISALIGNED, tg.TG_ERR_NOT_SUPPORTED

    def call(i=1, M=8, N=8, K=8, dy=A, lddy=8, x=A, ldx=8, w=A, ldw=8, z=A, ldz=8, act=4, dz=A, lddz=8, dx=A, lddx=8, dw=A, lddw=8, od=2,
             db=A, ws=None, nb=0):
        return lib.tg_linear_backward(i, M, N, K, dy, lddy, x, ldx, w, ldw, z, ldz, act, dz, lddz, dx, lddx, dw, lddw, od, db, ws, nb, None)

    for bad in (dict(K=-1), dict(i=7), dict(act=9), dict(od=-1), dict(dy=None), dict(x=None), dict(w=None), dict(z=None), dict(dz=None),
                dict(lddy=4), dict(ldz=4), dict(lddz=4), dict(lddx=4), dict(lddw=4), dict(nb=5),
                dict(M=4096, N=256, K=256, lddy=256, ldx=256, ldw=256, ldz=256, lddz=256, lddx=256, lddw=256, ws=W, nb=65536)):
        assert call(**bad) == inv, bad
    for bad in (dict(dy=A + 2), dict(dz=A + 2), dict(db=A + 2), dict(lddx=12), dict(dw=A + 8), dict(ws=W + 8, nb=BIG)):
        assert call(**bad) == mis, bad
    for bad in (dict(i=2), dict(od=1), dict(N=1 << 31), dict(lddz=1 << 31)):
        assert call(**bad) == nos, bad
    none = dict(act=0, z=None, dz=None, dx=None, dw=None, db=None)
    assert call(**none) == tg.TG_OK  # nothing asked for
    assert call(**none, x=None, w=None) == tg.TG_OK


def test_glu_refusals(tg, lib):
    inv, mis, nos = tg.TG_ERR_INVALID_VALUE, tg.TG_ERR_MISALIGNED, tg.TG_ERR_NOT_SUPPORTED

    def call(i=1, M=8, F=8, D=8, x=A, ldx=8, w=A, ldw=8, act=4, s=1.0, h=A, ldh=8, od=2, gu=A, ldgu=16, ws=None, nb=0):
        return lib.tg_glu(i, M, F, D, x, ldx, w, ldw, act, s, 1.0, h, ldh, od, gu, ldgu, ws, nb, None)

    for bad in (dict(F=-1), dict(i=3), dict(act=5), dict(od=3), dict(x=None), dict(w=None), dict(h=None), dict(ldh=4), dict(ldgu=8),
                dict(i=2, ldx=16, ldw=16, s=float("nan")), dict(nb=1)):
        assert call(**bad) == inv, bad
    for bad in (dict(h=A + 2), dict(gu=A + 2), dict(ldgu=20), dict(ws=W + 128, nb=BIG)):
        assert call(**bad) == mis, bad
    for bad in (dict(od=0), dict(od=1), dict(i=2, ldx=16, ldw=16, od=0), dict(F=1 << 30), dict(D=1 << 31)):
        assert call(**bad) == nos, bad
    assert call(M=0, x=None, w=None, h=None, gu=None) == tg.TG_OK and call(F=0, x=None, w=None, h=None, gu=None) == tg.TG_OK


def test_glu_backward_refusals(tg, lib):
    inv, mis, nos = tg.TG_ERR_INVALID_VALUE, tg.TG_ERR_MISALIGNED, tg.TG_ERR_NOT_SUPPORTED

    def call(i=1, M=8, F=8, D=8, dy=A, wd=A, x=A, w=A, gu=A, ldgu=16, h=A, act=4, dgu=A, lddgu=16, dx=A, lddx=8, dw=A, lddw=8, dwd=A,
             lddwd=8, od=2, ws=None, nb=0):
        return lib.tg_glu_backward(i, M, F, D, dy, 8, wd, 8, x, 8, w, 8, gu, ldgu, h, 8, act, dgu, lddgu, dx, lddx, dw, lddw, dwd, lddwd,
                                   od, ws, nb, None)

    for bad in (dict(M=-1), dict(act=5), dict(i=4), dict(od=5), dict(dy=None), dict(wd=None), dict(x=None), dict(w=None), dict(gu=None),
                dict(h=None), dict(dgu=None), dict(ldgu=8), dict(lddgu=8), dict(lddx=4), dict(lddw=4), dict(lddwd=4), dict(nb=7)):
        assert call(**bad) == inv, bad
    for bad in (dict(dgu=A + 2), dict(dwd=A + 2), dict(lddgu=20), dict(ws=W + 1, nb=BIG)):
        assert call(**bad) == mis, bad
    for bad in (dict(i=2), dict(od=1), dict(F=1 << 30)):
        assert call(**bad) == nos, bad


def test_clip_refusals(tg, lib):
    inv, mis = tg.TG_ERR_INVALID_VALUE, tg.TG_ERR_MISALIGNED
    need = lib.tg_clip_grads_workspace_bytes(1)
    assert 65536 < need <= BIG and lib.tg_clip_grads_workspace_bytes(-1) == -1

    def call(count=2, g=(A, A), o=(A, A), n=(4, 4), t=(0, 1), mx=1.0, eps=1e-6, norm=A, ws=W, nb=BIG):
        p = lambda v: (ctypes.c_uint64 * len(v))(*v) if v is not None else None  # noqa: E731
        return lib.tg_clip_grads(count, p(g), p(o), (ctypes.c_int64 * len(n))(*n), (ctypes.c_int32 * len(t))(*t), mx, eps, norm, ws, nb, None)

    for bad in (dict(count=-1), dict(mx=-1.0), dict(mx=float("nan")), dict(eps=-1.0), dict(eps=float("inf")), dict(g=None), dict(o=None),
                dict(g=(0, A)), dict(o=(A, 0)), dict(n=(-1, 4)), dict(t=(0, 3)), dict(t=(-1, 0)), dict(ws=None, nb=0), dict(nb=need - 1),
                dict(nb=-1)):
        assert call(**bad) == inv, bad
    for bad in (dict(g=(A + 2, A)), dict(o=(A, A + 1)), dict(norm=A + 2), dict(ws=W + 8)):
        assert call(**bad) == mis, bad
    assert call(count=0, norm=None) == tg.TG_OK


def test_workspace_queries(tg):
    bf = torch.bfloat16
    for M, N, K in ((1, 4096, 4096), (16, 512, 8192), (256, 8192, 8192), (777, 2056, 1032), (8192, 4096, 10240), (100, 7, 9)):
        for n in (tg.tg_linear_workspace_bytes(bf, M, N, K), tg.tg_linear_backward_workspace_bytes(bf, M, N, K),
                  tg.tg_glu_workspace_bytes(bf, M, N, K), tg.tg_glu_backward_workspace_bytes(bf, M, N, K)):
            assert 0 <= n <= BIG, (M, N, K, n)
    for q in (tg.tg_linear_workspace_bytes, tg.tg_glu_workspace_bytes, tg.tg_linear_backward_workspace_bytes,
              tg.tg_glu_backward_workspace_bytes):
        with pytest.raises(ValueError):
            q(bf, -1, 8, 8)
        with pytest.raises(ValueError):
            q(torch.float32, 8, 8, 8)
    with pytest.raises(ValueError):
        tg.tg_linear_backward_workspace_bytes(torch.float8_e4m3fn, 8, 8, 8)


def test_binding_refuses_wrong_tensors(tg):
    """Shapes, types, strides and devices are checked before the library is called."""
    t = torch.zeros
    bf, f16, f8 = torch.bfloat16, torch.float16, torch.float8_e4m3fn
    x, w, y = t(4, 16, dtype=bf), t(8, 16, dtype=bf), t(4, 8, dtype=bf)

    def no(fn, *a, **k):
        with pytest.raises(ValueError):
            fn(*a, **k)

    no(tg.tg_linear, x, w, y)  # not on the GPU
    no(tg.tg_linear, x.float(), w.float(), y)
    no(tg.tg_linear, x, w.to(f16), y)
    no(tg.tg_linear, x, w, y.to(f16))
    no(tg.tg_linear, x, w[:, :8], y)
    no(tg.tg_linear, x, w, t(4, 9, dtype=bf))
    no(tg.tg_linear, x, w, t(8, 4, dtype=bf).t())
    no(tg.tg_linear, x, w, y, act="tanh")
    no(tg.tg_linear, x, w, y, bias=t(8, dtype=bf))
    no(tg.tg_linear, x, w, y, bias=t(7))
    no(tg.tg_linear, x, w, y, residual=t(4, 8))
    no(tg.tg_linear, x, w, y, preact=t(4, 7, dtype=bf))
    no(tg.tg_linear, t(16, dtype=bf), w, y)
    no(tg.tg_linear, x, t((), dtype=bf), y)
    no(tg.tg_linear_backward, y, x, w, preact=y, act="silu")
    no(tg.tg_linear_backward, y.to(f8), x, w)
    no(tg.tg_linear_backward, y, x, w, dw=t(8, 16, dtype=f16))
    no(tg.tg_linear_backward, y, x, w, dx=t(4, 8, dtype=bf))
    no(tg.tg_linear_backward, y, x, w, dbias=t(8, dtype=bf))
    no(tg.tg_glu, x, w, t(4, 4))
    no(tg.tg_glu, x, w, t(4, 5, dtype=bf))
    no(tg.tg_glu, x, w, t(4, 4, dtype=bf), gate_up=t(4, 4, dtype=bf))
    no(tg.tg_glu, x.to(f8), w.to(f8), t(4, 4))
    d = (t(4, 16, dtype=bf), t(16, 4, dtype=bf), x, w, y)  # dY, Wd, x, W, gate_up
    no(tg.tg_glu_backward, *d, None, y, dw_down=t(16, 4, dtype=bf))
    no(tg.tg_glu_backward, *d, t(4, 4, dtype=bf), y, dw_down=t(16, 4, dtype=bf), dw_gate_up=t(8, 16))
    no(tg.tg_glu_backward, *d, t(4, 4, dtype=bf), t(4, 7, dtype=bf))
    g = t(5)
    no(tg.tg_clip_grads, [g], 1.0, workspace=None)
    no(tg.tg_clip_grads, [g], 1.0, workspace=t(8))  # not on the GPU
    no(tg.tg_clip_grads, [g.double()], 1.0, workspace=t(8))
    no(tg.tg_clip_grads, [t(4, 4).t()[:, :2]], 1.0, workspace=t(8))
    no(tg.tg_clip_grads, [g], 1.0, out=[], workspace=t(8))
    no(tg.tg_clip_grads, [g], 1.0, out=[t(6)], workspace=t(8))
    no(tg.tg_clip_grads, [g], 1.0, norm=t(2), workspace=t(8))
