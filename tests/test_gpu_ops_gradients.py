"""The backward operators against central differences of the 64-bit
definitions, along directions in which the derivative does not cancel.

Along the signs of the gradient itself the directional derivative is
sum |gradient|, and the errors of the gradient's values count at most at their
full size.  In fp16 the kernel rounds dz (or [dg | du]) by half a step, 2^-11 of
the value or 2^-25, and so a 16-bit gradient; slopes and activations are off by
the bounds of _ops_ref.py, an fp32 sum of n products by 2 n u of their absolute
sum.  Every case also asserts that the bound is a small part of the
derivative: a gradient of zeros, or one with a wrong scale or a lost term,
cannot pass."""
import pytest
import torch

from _ops_ref import U, act, act_bound, slope_bound
from test_gpu_ops import rand, tg, ws  # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu

T = torch.float16
HALF, TINY = 2.0 ** -11, 2.0 ** -25
STEP = 1e-5
SMOOTH = ("none", "gelu", "gelu_tanh", "silu")


def check(what, got, loss, size, off):
    """`loss(d)`: the 64-bit loss with the parameter moved by d; `size`: the absolute sum of each gradient value's
    products; `off`: the bound of its error before it is stored."""
    g = got.double()
    v = torch.sign(g)
    v = torch.where(v == 0, torch.ones_like(v), v)
    want = float(loss(STEP * v) - loss(-STEP * v)) / (2 * STEP)
    stored = HALF * (size + off) + TINY if got.dtype == T else U * (size + off)
    tol = float((off + stored).sum()) + 1e-6 * abs(want)
    assert tol < 0.05 * abs(want), f"{what}: a bound of {tol:.3g} on {want:.3g} shows nothing"
    d = abs(float((g * v).sum()) - want)
    assert d <= tol, f"{what}: off by {d:.3g}, bound {tol:.3g}, derivative {want:.3g}"


def mm(a, b):
    return a @ b.contiguous()


def summed(a, b, ea):
    """Absolute sums of a . b and the bound of its fp32 sum where a is off by ea."""
    size = mm(a.abs(), b.abs())
    return size, mm(ea, b.abs()) * (1 + 2 * a.shape[1] * U) + 2 * a.shape[1] * U * size


@pytest.mark.parametrize("name", SMOOTH)
@pytest.mark.parametrize("M,N,K", [(40, 48, 56), (300, 136, 72), (33, 264, 33)])
@pytest.mark.parametrize("wide", [False, True])
def test_linear_gradients(tg, ws, name, M, N, K, wide):
    c, x, w = rand(M, N, T, 1), rand(M, K, T, 2), rand(N, K, T, 3, K ** -0.5)
    z = rand(M, N, T, 4)  # (the loss is taken around this pre-activation, as the kernel is given it)
    dz, dx, db = rand(M, N, T, 5), rand(M, K, T, 6), torch.empty(N, device="cuda")
    dw = rand(N, K, torch.float32 if wide else T, 7)
    tg.tg_linear_backward(c, x, w, dx=dx, dw=dw, dbias=db, preact=z, act=name, dz=dz, workspace=ws)
    c64, x64, w64 = c.double(), x.double(), w.double()
    z64 = z.double() if name != "none" else torch.zeros_like(c64)
    d = c64 * act(name, z64)[1]
    exact = torch.zeros_like(d) if name == "none" else c64.abs() * slope_bound(name) + U * d.abs()
    ez = exact if name == "none" else exact + HALF * (d.abs() + exact) + TINY

    def loss(move):
        return (c64 * act(name, z64 + move)[0]).sum()

    check("dx", dx, lambda p: loss(mm(p, w64.t())), *summed(d, w64, ez))
    check("dw", dw, lambda p: loss(mm(x64, p.t())), *summed(d.t().contiguous(), x64, ez.t().contiguous()))
    check("dbias", db, loss, d.abs().sum(0), exact.sum(0) + 2 * M * U * d.abs().sum(0))


@pytest.mark.parametrize("name", SMOOTH)
@pytest.mark.parametrize("M,F,D", [(40, 24, 40), (130, 72, 136), (33, 40, 33)])
@pytest.mark.parametrize("wide", [False, True])
def test_glu_gradients(tg, ws, name, M, F, D, wide):
    c, x, wd, w = rand(M, D, T, 1), rand(M, D, T, 2), rand(D, F, T, 3, F ** -0.5), rand(2 * F, D, T, 4, D ** -0.5)
    gu = rand(M, 2 * F, T, 5)
    g64, u64 = gu[:, :F].double(), gu[:, F:].double()
    h = rand(M, F, T, 6)
    h.copy_(act(name, g64)[0] * u64)
    o = torch.float32 if wide else T
    dgu, dx, dw, dwd = rand(M, 2 * F, T, 7), rand(M, D, T, 8), rand(2 * F, D, o, 9), rand(D, F, o, 10)
    tg.tg_glu_backward(c, wd, x, w, gu, h, dgu, dx=dx, dw_gate_up=dw, dw_down=dwd, act=name, workspace=ws)
    c64, x64, wd64, w64, h64 = c.double(), x.double(), wd.double(), w.double(), h.double()
    dh, (v, slope) = mm(c64, wd64), act(name, g64)
    eh = 2 * D * U * mm(c64.abs(), wd64.abs())
    es, ev = slope_bound(name), act_bound(name, g64, v, torch.zeros_like(g64))
    d = torch.cat([dh * u64 * slope, dh * v], 1)
    ed = torch.cat([(eh * slope.abs() + (dh.abs() + eh) * es) * u64.abs(), eh * v.abs() + (dh.abs() + eh) * ev], 1) + 3 * U * d.abs()
    ed = ed + HALF * (d.abs() + ed) + TINY

    def loss(move):
        return (dh * act(name, g64 + move[:, :F])[0] * (u64 + move[:, F:])).sum()

    check("dx", dx, lambda p: loss(mm(p, w64.t())), *summed(d, w64, ed))
    check("dw_gate_up", dw, lambda p: loss(mm(x64, p.t())), *summed(d.t().contiguous(), x64, ed.t().contiguous()))
    ct = c64.t().contiguous()
    check("dw_down", dwd, lambda p: (c64 * mm(h64, p.t())).sum(), *summed(ct, h64, torch.zeros_like(ct)))
