"""The feed-forward operators as a user calls them, with their plain forms.

Operators (formulas; act is none, relu, gelu, gelu_tanh or silu):

  linear      y = act(a * x.W^T + bias) + residual, W stored N x K; optionally z = a * x.W^T + bias kept for training
  linear_bwd  dz = dy * act'(z);  dx = dz.W;  dW = dz^T.x;  dbias = sum over rows of dz
  glu         g = a * x.Wg^T, u = a * x.Wu^T, h = act(g) * u; W = [Wg; Wu] stored 2F x D; optionally [g | u] kept for training
  glu_bwd     dh = dy.Wd;  dg = dh * u * act'(g);  du = dh * act(g);  dx = [dg | du].W;  dW = [dg | du]^T.x;  dWd = dy^T.h
  clip        norm = sqrt(sum over all tensors of g^2);  out = g * min(1, max_norm / (norm + 1e-6))

`listed()` are the measured cases, `draw()` gives more of the same ranges.
"""
from __future__ import annotations

import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "fp8": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "f16": 2, "f32": 4, "fp8": 1}
SCRATCH = (64 << 20) + (64 << 10)  # bytes of split workspace that every plan of the library fits in
EPS = 1e-6


def listed():
    return [
        # one token through an attention output projection: a weight read once, latency counts
        dict(name="linear_decode_1", op="linear", m=1, n=4096, k=4096, dtype="bf16", out="bf16", act="none", bias=False, residual=True, keep=False),
        # first layer of a plain feed-forward block in training, ragged token count, pre-activation kept
        dict(name="linear_gelu_ragged", op="linear", m=1003, n=4104, k=2056, dtype="f16", out="f16", act="gelu", bias=True, residual=False, keep=True),
        # down projection of a long prompt, added to the residual stream
        dict(name="linear_down_8192", op="linear", m=8192, n=4096, k=10240, dtype="bf16", out="bf16", act="none", bias=False, residual=True, keep=False),
        # gradients of a small layer with an activation, odd token count
        dict(name="linear_bwd_ragged", op="linear_bwd", m=777, n=2056, k=1032, dtype="f16", out="f16", act="gelu", bias=True),
        # gradients of a square projection, weight gradient in 32 bits for the optimizer
        dict(name="linear_bwd_4096", op="linear_bwd", m=4096, n=4096, k=4096, dtype="bf16", out="f32", act="none", bias=True),
        # a decode batch of 16 tokens through the gated pair
        dict(name="glu_decode_16", op="glu", m=16, f=8192, d=4096, dtype="bf16", out="bf16", act="silu", keep=False),
        # a prompt in 8-bit serving
        dict(name="glu_prefill_fp8", op="glu", m=2047, f=8192, d=8192, dtype="fp8", out="bf16", act="silu", keep=False),
        # training forward of the gated pair, both projections kept
        dict(name="glu_train_4096", op="glu", m=4096, f=10240, d=4096, dtype="bf16", out="bf16", act="silu", keep=True),
        # gradients of a small gated block, odd token count
        dict(name="glu_bwd_ragged", op="glu_bwd", m=509, f=2728, d=1024, dtype="f16", out="f16", act="gelu_tanh"),
        # gradients of a large gated block
        dict(name="glu_bwd_8192", op="glu_bwd", m=8192, f=10240, d=4096, dtype="bf16", out="bf16", act="silu"),
        # a few small tensors (norm weights, biases, an adapter): latency counts
        dict(name="clip_small", op="clip", count=9, total=60001, dtype="f32", max_norm=1.0),
        # all gradients of a shard: matrices and vectors, 16-bit and 32-bit ones
        dict(name="clip_large", op="clip", count=56, total=400_000_003, dtype="mixed", max_norm=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _wide(rng, lo, hi):
    """A width: a multiple of 8, as aligned rows of 16-bit values have it."""
    return max(8, _log(rng, lo, hi) // 8 * 8)


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_bwd", "glu", "glu", "glu_bwd", "clip"])
    act = rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"])
    if op == "linear":
        dtype = rng.choice(["bf16", "f16", "fp8"])  # 8-bit layers hand 16-bit activations on
        return dict(op=op, m=_log(rng, 1, 8192), n=_wide(rng, 512, 8192) + rng.choice([0, 0, 1, 5]), k=_wide(rng, 512, 8192) // 16 * 16, dtype=dtype,
                    out=rng.choice(["bf16", "f16"]) if dtype == "fp8" else rng.choice([dtype, "f32"]), act=act, bias=rng.random() < 0.5,
                    residual=rng.random() < 0.5, keep=rng.random() < 0.3)
    if op == "linear_bwd":
        dtype = rng.choice(["bf16", "f16"])
        return dict(op=op, m=_log(rng, 64, 8192), n=_wide(rng, 512, 8192), k=_wide(rng, 512, 8192), dtype=dtype,
                    out=rng.choice([dtype, "f32"]) if act == "none" else dtype, act=act, bias=rng.random() < 0.5)
    act = rng.choice(["silu", "gelu", "gelu_tanh", "relu"])
    if op == "glu":
        dtype = rng.choice(["bf16", "f16", "fp8"])
        return dict(op=op, m=_log(rng, 1, 4096), f=_wide(rng, 512, 10240), d=_wide(rng, 512, 8192) // 16 * 16, dtype=dtype,
                    out="bf16" if dtype == "fp8" else dtype, act=act, keep=rng.random() < 0.4)
    if op == "glu_bwd":
        dtype = rng.choice(["bf16", "f16"])
        return dict(op=op, m=_log(rng, 64, 8192), f=_wide(rng, 512, 10240), d=_wide(rng, 256, 4096), dtype=dtype, out=dtype, act=act)
    return dict(op="clip", count=rng.randint(1, 60), total=_log(rng, 1000, 190_000_000), dtype=rng.choice(["f32", "bf16", "f16", "mixed"]),
                max_norm=rng.choice([0.5, 1.0, 1e9]))


def _sizes(case):
    """Numbers of values of the tensors: one in four a matrix, which hold nearly all of them, and the rest short vectors."""
    count, total = int(case["count"]), int(case["total"])
    small = [min(1 + 613 * i % 4099, total // (2 * count) + 1) for i in range(count)]
    matrices = [i for i in range(count) if i % 4 == 0]
    left = max(0, total - sum(small[i] for i in range(count) if i % 4))
    for j, i in enumerate(matrices):
        small[i] = max(1, left * (j + 1) // sum(range(1, len(matrices) + 1)))
    return small


def _types(case):
    return [("f32" if i % 4 else "bf16") if case["dtype"] == "mixed" else case["dtype"] for i in range(int(case["count"]))]


def _ld(n):
    """Leading dimension of a matrix of n columns: rows that start on 16 bytes, whatever the type."""
    return -(-n // 16) * 16


def _make(case, seed):
    """The inputs, from the seed alone."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))

    def normal(shape, std=1.0, dtype="f32"):
        t = torch.empty(shape[0], _ld(shape[1]), device="cuda")[:, :shape[1]] if len(shape) == 2 else torch.empty(shape, device="cuda")
        t.normal_(0.0, std, generator=gen)
        if dtype == "f32":
            return t
        o = torch.empty(t.shape[0], _ld(shape[1]), device="cuda", dtype=DT[dtype])[:, :shape[1]] if len(shape) == 2 else torch.empty(shape, device="cuda", dtype=DT[dtype])
        return o.copy_(t)

    def eight(shape, std):
        """8-bit values and the step that they count in: the largest value on the type's largest."""
        t = torch.empty(shape, device="cuda").normal_(0.0, std, generator=gen)
        step = 5.5 * std / 448.0
        return (t / step).clamp_(-448, 448).to(torch.float8_e4m3fn), step

    op, s = case["op"], {}
    if op == "clip":
        s["grads"] = [torch.empty(n, device="cuda").normal_(0.0, 10.0 ** (i % 3 - 1), generator=gen).to(DT[t])
                      for i, (n, t) in enumerate(zip(_sizes(case), _types(case)))]
        return s
    t = case["dtype"]
    s["scale_x"] = s["scale_w"] = 1.0
    if op in ("linear", "linear_bwd"):
        m, n, k = case["m"], case["n"], case["k"]
        if t == "fp8":
            s["x"], s["scale_x"] = eight((m, k), 1.0)
            s["w"], s["scale_w"] = eight((n, k), k ** -0.5)
        else:
            s["x"], s["w"] = normal((m, k), 1.0, t), normal((n, k), k ** -0.5, t)
        if op == "linear":
            s["bias"] = normal((n,), 0.5) if case["bias"] else None
            s["residual"] = normal((m, n), 1.0, case["out"]) if case["residual"] else None
        else:
            s["dy"], s["z"] = normal((m, n), 1.0, t), normal((m, n), 1.0, t)
        return s
    m, f, d = case["m"], case["f"], case["d"]
    if t == "fp8":
        s["x"], s["scale_x"] = eight((m, d), 1.0)
        s["w"], s["scale_w"] = eight((2 * f, d), d ** -0.5)
    else:
        s["x"], s["w"] = normal((m, d), 1.0, t), normal((2 * f, d), d ** -0.5, t)
    if op == "glu_bwd":
        s["dy"], s["wd"] = normal((m, d), 1.0, t), normal((d, f), f ** -0.5, t)
        s["gu"], s["h"] = normal((m, 2 * f), 1.0, t), normal((m, f), 0.6, t)
    return s


def prepare(case, seed):
    s = _make(case, seed)
    op, out = case["op"], DT.get(case.get("out"))

    def room(rows, cols, dtype):
        return torch.zeros(rows, _ld(cols), device="cuda", dtype=dtype)[:, :cols]

    s["case"] = case
    s["workspace"] = torch.zeros(SCRATCH // 4, device="cuda", dtype=torch.int32)
    if op == "clip":
        s["out"] = [torch.empty_like(g) for g in s["grads"]]
        s["norm"] = torch.empty(1, device="cuda")
    elif op == "linear":
        s["y"] = room(case["m"], case["n"], out)
        s["zout"] = room(case["m"], case["n"], out) if case["keep"] else None
    elif op == "linear_bwd":
        t = DT[case["dtype"]]
        s["dz"] = room(case["m"], case["n"], t) if case["act"] != "none" else None
        s["dx"], s["dw"] = room(case["m"], case["k"], t), room(case["n"], case["k"], out)
        s["db"] = torch.empty(case["n"], device="cuda") if case["bias"] else None
    elif op == "glu":
        s["hout"] = room(case["m"], case["f"], out)
        s["guout"] = room(case["m"], 2 * case["f"], out) if case["keep"] else None
    else:
        m, f, d = case["m"], case["f"], case["d"]
        s["dgu"], s["dx"] = room(m, 2 * f, out), room(m, d, out)
        s["dw"], s["dwd"] = room(2 * f, d, out), room(d, f, out)
    return s


# ---------------------------------------------------------------- plain forms


def _act(name, x):
    if name == "none":
        return x
    if name == "relu":
        return x * (x > 0)
    if name == "silu":
        return x / (1 + torch.exp(-x))
    if name == "gelu":
        return 0.5 * x * (1 + torch.erf(x * 0.5 ** 0.5))
    return 0.5 * x * (1 + torch.tanh((2 / math.pi) ** 0.5 * (x + 0.044715 * x * x * x)))


def _act_grad(name, x):
    if name == "none":
        return torch.ones_like(x)
    if name == "relu":
        return (x > 0).to(x.dtype)
    if name == "silu":
        p = 1 / (1 + torch.exp(-x))
        return p * (1 + x * (1 - p))
    if name == "gelu":
        return 0.5 * (1 + torch.erf(x * 0.5 ** 0.5)) + x * torch.exp(-0.5 * x * x) * (2 * math.pi) ** -0.5
    c = (2 / math.pi) ** 0.5
    t = torch.tanh(c * (x + 0.044715 * x * x * x))
    return 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * c * (1 + 3 * 0.044715 * x * x)


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "clip":
        norm = torch.stack([g.double().square().sum() for g in s["grads"]]).sum().sqrt()
        coef = torch.clamp(case["max_norm"] / (norm + EPS), max=1.0)
        return {"norm": norm.float().reshape(1), "out": [(g.float() * coef.float()).to(g.dtype) for g in s["grads"]]}
    out = DT[case["out"]]
    if op == "linear":
        z = (s["x"].float() @ s["w"].float().t()) * (s["scale_x"] * s["scale_w"])
        if s["bias"] is not None:
            z = z + s["bias"]
        y = _act(case["act"], z)
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return {"y": y.to(out), "z": z.to(out)} if case["keep"] else {"y": y.to(out)}
    if op == "linear_bwd":
        dz = s["dy"].float() * _act_grad(case["act"], s["z"].float())
        r = {"dx": (dz @ s["w"].float()).to(s["x"].dtype), "dw": (dz.t() @ s["x"].float()).to(out)}
        if case["bias"]:
            r["db"] = dz.sum(0)
        return r
    f = case["f"]
    if op == "glu":
        gu = (s["x"].float() @ s["w"].float().t()) * (s["scale_x"] * s["scale_w"])
        h = _act(case["act"], gu[:, :f]) * gu[:, f:]
        return {"h": h.to(out), "gu": gu.to(out)} if case["keep"] else {"h": h.to(out)}
    g, u, dy = s["gu"][:, :f].float(), s["gu"][:, f:].float(), s["dy"].float()
    dh = dy @ s["wd"].float()
    dgu = torch.cat([dh * u * _act_grad(case["act"], g), dh * _act(case["act"], g)], 1)
    return {"dx": (dgu @ s["w"].float()).to(out), "dw": (dgu.t() @ s["x"].float()).to(out), "dwd": (dy.t() @ s["h"].float()).to(out)}


def _own(s):
    import tile_level_gemm_02_amd as tg

    case = s["case"]
    op = case["op"]
    if op == "clip":
        tg.tg_clip_grads(s["grads"], case["max_norm"], out=s["out"], norm=s["norm"], eps=EPS, workspace=s["workspace"])
        return {"norm": s["norm"], "out": s["out"]}
    if op == "linear":
        tg.tg_linear(s["x"], s["w"], s["y"], bias=s["bias"], act=case["act"], residual=s["residual"], preact=s["zout"], scale_x=s["scale_x"],
                     scale_w=s["scale_w"], workspace=s["workspace"])
        return {"y": s["y"], "z": s["zout"]} if case["keep"] else {"y": s["y"]}
    if op == "linear_bwd":
        tg.tg_linear_backward(s["dy"], s["x"], s["w"], dx=s["dx"], dw=s["dw"], dbias=s["db"], preact=s["z"], act=case["act"], dz=s["dz"],
                              workspace=s["workspace"])
        r = {"dx": s["dx"], "dw": s["dw"]}
        if case["bias"]:
            r["db"] = s["db"]
        return r
    if op == "glu":
        tg.tg_glu(s["x"], s["w"], s["hout"], act=case["act"], gate_up=s["guout"], scale_x=s["scale_x"], scale_w=s["scale_w"], workspace=s["workspace"])
        return {"h": s["hout"], "gu": s["guout"]} if case["keep"] else {"h": s["hout"]}
    tg.tg_glu_backward(s["dy"], s["wd"], s["x"], s["w"], s["gu"], s["h"], s["dgu"], dx=s["dx"], dw_gate_up=s["dw"], dw_down=s["dwd"], act=case["act"],
                       workspace=s["workspace"])
    return {"dx": s["dx"], "dw": s["dw"], "dwd": s["dwd"]}


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    op = case["op"]
    if op == "clip":
        b = sum(n * SIZE[t] for n, t in zip(_sizes(case), _types(case)))
        return {"bytes": 2 * b + 4, "flops": 3 * sum(_sizes(case))}
    t, o = SIZE[case["dtype"]], SIZE[case["out"]]
    if op == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": (m + n) * k * t + m * n * o * (1 + case["residual"] + case["keep"]) + 4 * n * case["bias"], "flops": 2 * m * n * k}
    if op == "linear_bwd":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": (m * n * (1 + (case["act"] != "none")) + 2 * m * k + n * k) * t + n * k * o + 4 * n * case["bias"], "flops": 4 * m * n * k}
    m, f, d = case["m"], case["f"], case["d"]
    if op == "glu":
        return {"bytes": (m + 2 * f) * d * t + m * f * o * (3 if case["keep"] else 1), "flops": 4 * m * f * d}
    return {"bytes": (3 * m * d + 3 * m * f + 6 * f * d) * t, "flops": 12 * m * f * d}


# ------------------------------------------------- the definitions in 64 bits


def _phi(name, v):
    """(value, slope) of an activation in 64 bits."""
    if name == "none":
        return v, torch.ones_like(v)
    if name == "relu":
        return v.clamp(min=0), torch.heaviside(v, torch.zeros_like(v))
    if name == "silu":
        p = torch.sigmoid(v)
        return v * p, p + v * p * (1 - p)
    if name == "gelu":
        cdf = 0.5 * torch.special.erfc(-v / math.sqrt(2))
        return v * cdf, cdf + v * torch.exp(-v.square() / 2) / math.sqrt(2 * math.pi)
    # 0.5 * (1 + tanh(a)) is the logistic function of 2a
    a = 2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v.pow(3))
    p = torch.sigmoid(a)
    return v * p, p + v * p * (1 - p) * 2 * math.sqrt(2 / math.pi) * (1 + 0.134145 * v.square())


def exact(case, seed):
    s, op = _make(case, seed), case["op"]
    if op == "clip":
        total = sum(torch.dot(g.double(), g.double()) for g in s["grads"])
        norm = math.sqrt(float(total))
        c = min(1.0, case["max_norm"] / (norm + EPS))
        return {"norm": torch.tensor([norm], dtype=torch.float64), "out": [g.double() * c for g in s["grads"]]}
    x, w = s["x"].double(), s["w"].double()
    if op == "linear":
        z = torch.mm(x, w.t()) * s["scale_x"] * s["scale_w"]
        z = z if s["bias"] is None else z + s["bias"].double()
        y = _phi(case["act"], z)[0]
        y = y if s["residual"] is None else y + s["residual"].double()
        return {"y": y, "z": z} if case["keep"] else {"y": y}
    if op == "linear_bwd":
        dz = s["dy"].double() * _phi(case["act"], s["z"].double())[1]
        r = {"dx": torch.mm(dz, w), "dw": torch.mm(dz.t(), x)}
        if case["bias"]:
            r["db"] = torch.mv(dz.t(), torch.ones(case["m"], device="cuda", dtype=torch.float64))
        return r
    f = case["f"]
    if op == "glu":
        g, u = (torch.mm(x, half.t()) * s["scale_x"] * s["scale_w"] for half in (w[:f], w[f:]))
        h = _phi(case["act"], g)[0] * u
        return {"h": h, "gu": torch.cat([g, u], 1)} if case["keep"] else {"h": h}
    g, u, dy = s["gu"][:, :f].double(), s["gu"][:, f:].double(), s["dy"].double()
    dh = torch.mm(dy, s["wd"].double())
    value, slope = _phi(case["act"], g)
    dg, du = dh * u * slope, dh * value
    return {"dx": torch.mm(dg, w[:f]) + torch.mm(du, w[f:]), "dw": torch.cat([torch.mm(dg.t(), x), torch.mm(du.t(), x)], 0),
            "dwd": torch.mm(dy.t(), s["h"].double())}
