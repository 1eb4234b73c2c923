"""The feed-forward operators' definitions in 64 bits, and the error bounds
their fp32 kernels are held to.  TEST INFRASTRUCTURE ONLY.

Bounds (u = 2^-24, half a step of fp32; h = finfo(t).eps / 2, half a step of
the output type relative to the value):

  product    |z - z*| <= 2 K u S + 4 u |z|, S = |x| |W|^T: any order of K fp32
             additions, then scale and bias (oracle/check.py); fp8 adds
             7 2^-13 S for its matrix instruction's inner sums
  activation slopes are at most 1.13 (gelu_tanh, gelu 1.129, silu 1.1), so an
             error of z grows by at most that.  Evaluation: the exponent's
             argument t carries 4 roundings, so the logistic function is off
             by 4 u |t| (1 - s) and 6 u more, relative; |x| |t| s (1 - s) < 0.6,
             which gives under 8 u (1 + |y|).  gelu: 1.5e-7 / 2 |x| besides.
  slope      as above with up to three such products: 32 u, and 2e-7 for gelu
  rounding   h |y|, and half the smallest subnormal step
"""
import math

import torch

U = 2.0 ** -24
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def act(name, v):
    """(value, slope) in 64 bits."""
    if name == "none":
        return v, torch.ones_like(v)
    if name == "relu":
        return v.clamp(min=0), (v > 0).double()
    if name == "silu":
        s = torch.sigmoid(v)
        return v * s, s * (1 + v * (1 - s))
    if name == "gelu":
        c = 0.5 * torch.special.erfc(-v / math.sqrt(2.0))
        return v * c, c + v * torch.exp(-0.5 * v * v) / math.sqrt(2.0 * math.pi)
    k = math.sqrt(2.0 / math.pi)
    t = torch.tanh(k * (v + 0.044715 * v ** 3))
    return 0.5 * v * (1 + t), 0.5 * (1 + t) + 0.5 * v * (1 - t * t) * k * (1 + 3 * 0.044715 * v * v)


def rounding(y, dtype):
    """Half a step of dtype at y (of a value slightly off y)."""
    tiny = {torch.float32: 2.0 ** -150, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}[dtype]
    return torch.finfo(dtype).eps / 2 * y.abs() * (1 + 2.0 ** -7) + tiny


def product(x, w, alpha=1.0, inner=0.0):
    """x . w^T in 64 bits and the bound of its fp32 sum."""
    x, w = x.double(), w.double()
    z, S = x @ w.t().contiguous() * alpha, x.abs() @ w.abs().t().contiguous() * abs(alpha)
    return z, (2 * x.shape[1] * U + inner) * S + 4 * U * z.abs()


def act_bound(name, z, y, dz):
    """Bound of act(z) computed in fp32 where z is off by dz."""
    if name in ("none", "relu"):
        return dz
    return 1.13 * dz + 8 * U * (1 + y.abs()) + (0.75e-7 * z.abs() if name == "gelu" else 0.0)


def slope_bound(name):
    return 0.0 if name in ("none", "relu") else 32 * U + (2e-7 if name == "gelu" else 0.0)


def within(got, want, tol, what):
    got = got.double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    if got.numel() == 0:
        return
    assert bool(torch.isfinite(got).all()), f"{what}: not finite"
    r = (got - want).abs() / tol.clamp(min=1e-300)
    r = torch.where(got == want, torch.zeros_like(r), r)
    i = int(r.argmax())
    assert float(r.flatten()[i]) <= 1.0, f"{what}: {float(r.flatten()[i]):.3g} of its bound at flat index {i}"
