"""The training operators' definitions in 64 bits, and the error bounds their
fp32 kernels are held to.  TEST INFRASTRUCTURE ONLY.

Bounds (u = 2^-24, half a step of fp32; h = finfo(t).eps / 2):

  logits   t = scale x.W^T is off by dt = 2 D u S + 4 u |t|, S = |scale| |x| |W|^T
           (any order of D fp32 additions, then the scale)
  lse      e^(t - lse) is computed as exp2 of an argument whose products and
           differences carry 4 roundings of numbers up to |t| + |lse|, and the
           instruction is off by a unit in the last place: off by
           dp = dt + 4 u (|t| + |lse|) + 4 u relative.  A sum of positive numbers is off
           by u for each addition on a value's way (at most ADDS) besides; the
           logarithm turns relative errors into absolute ones, and is off by 2 u of
           itself.  Since lse is a mean of the t weighted by p, it moves by at most the
           largest dt of its row.
  loss     lse's and the target's errors, and 4 u of every term
  dt       p a - b: p's relative error dp + 3 u (lse itself is an input here), 2 u of each
           part, then h of itself (rounded to 16 bits; fp16: relative to 2^12 of the
           largest row's factor, so the smallest step is 2^-24 / 2^11 of that)
  products 2 K u S (K terms) + those errors of dt carried through, and h of the result
"""
import torch

U = 2.0 ** -24
# additions on a value's way into a row's sum: up to 16 in a lane and 2 between lanes, then the join: 8 in a batch, a batch
# for every 8 x 16 slots, 20 between lanes; each join multiplies by an exponential off by 4 u as well
def adds(V):
    return 18 + 2 * (8 + V / (16 * 8 * 16) + 20)


def half(dtype):
    return torch.finfo(dtype).eps / 2


def logits(x, w, scale):
    x, w = x.double(), w.double()
    t = scale * (x @ w.t().contiguous())
    S = abs(scale) * (x.abs() @ w.abs().t().contiguous())
    return t, 2 * x.shape[1] * U * S + 4 * U * t.abs()


def xent(x, w, target, scale, ignore, z):
    """(loss, lse, bounds of both) in 64 bits."""
    t, dt = logits(x, w, scale)
    lse = torch.logsumexp(t, 1)
    ref = lse[:, None].abs()
    de = (dt + 4 * U * (t.abs() + ref)).amax(1) + 4 * U + 2 * adds(t.shape[1]) * U + 2 * U * lse.abs()
    counts = target != ignore
    pick = target.clamp(0, t.shape[1] - 1)[:, None]
    tt, dtt = t.gather(1, pick)[:, 0], dt.gather(1, pick)[:, 0]
    loss = torch.where(counts, lse - tt + z * lse * lse, 0.0)
    dl = de + dtt + 4 * U * (lse.abs() + tt.abs()) + abs(z) * (2 * lse.abs() * de + 4 * U * lse * lse)
    return loss, lse, torch.where(counts, dl, 0.0), de


def xent_grad(x, w, target, scale, ignore, z, lse, g, dtype):
    """(dx, dw, bounds of both before their own rounding) in 64 bits; g: each row's factor."""
    t, dt = logits(x, w, scale)
    M, V = t.shape
    lse = lse.double()
    counts = (target != ignore).double()
    p = torch.exp(t - lse[:, None])
    a, b = counts * g * (1 + 2 * z * lse), counts * g
    d = p * a[:, None]
    hot = torch.zeros_like(d).scatter_(1, target.clamp(0, V - 1)[:, None], b[:, None])
    rel = dt + 4 * U * (t.abs() + lse.abs()[:, None]) + 7 * U
    err = p * a.abs()[:, None] * rel + 2 * U * (d.abs() + hot.abs())
    d = d - hot
    err = err + half(dtype) * (1 + 2.0 ** -7) * d.abs()
    if dtype == torch.float16:
        err = err + 2.0 ** -36 * float(torch.maximum(a.abs(), b.abs()).max()) * counts[:, None]
    x, w = x.double(), w.double()
    s = abs(scale)
    dx, dw = scale * (d @ w), scale * (d.t().contiguous() @ x)
    # (4 u: scale, count and the factor they make)
    bx = s * (err @ w.abs()) + (2 * V * U + 4 * U) * s * (d.abs() @ w.abs())
    bw = s * (err.t().contiguous() @ x.abs()) + (2 * M * U + 4 * U) * s * (d.abs().t().contiguous() @ x.abs())
    return dx, dw, bx, bw


def tiny(dtype):
    """Half the smallest subnormal step."""
    return {torch.float32: 2.0 ** -150, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}[dtype]


def rounded(y, dtype):
    return half(dtype) * y.abs() * (1 + 2.0 ** -7) + tiny(dtype)


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


# ------------------------------------------------------------------- AdamW
E4M3_MAX, E4M3_STEP, TINY, BLOCK = 448.0, 2.0 ** -9, 2.0 ** -100, 256


def held(q, scale, n):
    """Values that 8-bit states stand for, in 64 bits."""
    pad = -n % BLOCK
    v = torch.nn.functional.pad(q.double().flatten(), (0, pad)).view(-1, BLOCK)
    return (v * scale.double()[:, None]).flatten()[:n]


def adamw(w, g, m, v, step, lr, b1, b2, eps, wd, norm=None, max_norm=float("inf")):
    """One step in 64 bits."""
    w, g, m, v = (t.double() for t in (w, g, m, v))
    if norm is not None:
        g = g * min(1.0, max_norm / (norm + 1e-6))
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    up = lr / (1 - b1 ** step) * m / ((v / (1 - b2 ** step)).sqrt() + eps)
    return w * (1 - lr * wd) - up, m, v, up
