"""The feed-forward operators at the edges of their range: pre-activations whose
square leaves fp32's range and infinite ones, on every kernel."""
import pytest
import torch

from _ops_ref import ACTS, U, act, act_bound, product, rounding, slope_bound
from test_gpu_ops import DT, FP8_INNER, bwd_case, clean, glu_bwd_case, out, rand, tg, ws  # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu

INF = float("inf")


def agrees(got, want, tol, what):
    """NaN and infinities where the definition has them, within tol elsewhere."""
    got = got.double()
    for name, a, b in (("NaN", got.isnan(), want.isnan()), ("inf", got == INF, want == INF), ("-inf", got == -INF, want == -INF)):
        assert torch.equal(a, b), f"{what}: {int((a != b).sum())} values differ in being {name}"
    r = torch.where(torch.isfinite(want) & (got != want), (got - want).abs() / tol.clamp(min=1e-300), torch.zeros_like(want))
    assert float(r.max()) <= 1.0, f"{what}: {float(r.max()):.3g} of its bound"


# few rows (one slice and two), the 64 and 128 tiles, the 256 tile, the generic tile
EDGE_SHAPES = [(6, 136, 128), (23, 72, 136), (130, 201, 272), (1270, 1281, 72), (4090, 4097, 200), (50, 70, 33)]
LARGE = (INF, -INF, 1e30, -1e30, 2e19, -2e19)  # rows 0 to 5 (fp16 holds the infinities alone)


def edge_rows(M, N, K, t, seed):
    """x whose first rows hold one of LARGE and zeros, and W."""
    x, w = rand(M, K, t, seed), rand(N, K, t, seed + 1, K ** -0.5)
    for r, v in enumerate(LARGE):
        x[r] = 0.0
        x[r, 0] = v if t != torch.float16 or abs(v) == INF else 6e4 * (1 if v > 0 else -1)
    return x, w


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("dt,od", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16")])
def test_linear_large_and_infinite(tg, ws, name, dt, od):
    for M, N, K in EDGE_SHAPES:
        x, w = edge_rows(M, N, K, DT[dt], 1)
        s, y = out(M, N, DT[od])
        print(f"linear {M}x{N}x{K} {dt}->{od} {name}", flush=True)
        tg.tg_linear(x, w, y, act=name, workspace=ws)
        z, tol = product(x[:12], w)
        v = act(name, z)[0]
        agrees(y[:12], v, act_bound(name, z, v, tol) * (1 + 2.0 ** -7) + rounding(v, DT[od]), "y")
        assert bool(torch.isfinite(y[6:]).all())
        clean(s, M, N, "y")


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_glu_large_and_infinite(tg, ws, name, dt):
    t = DT[dt]
    for M, F, D in EDGE_SHAPES:
        x, w = edge_rows(M, 2 * F, D, t, 1)
        if t == torch.bfloat16:
            w[F:, 0] *= 2.0 ** -100  # finite rows: an up projection of ordinary size beside the large gate
        else:
            w[:, 0] *= 2.0 ** -10
        s, h = out(M, F, t)
        print(f"glu {M}x{F}x{D} {dt} {name}", flush=True)
        tg.tg_glu(x, w, h, act=name, workspace=ws)
        p, b = product(x[:12], w)
        g, u, eg, eu = p[:, :F], p[:, F:], b[:, :F], b[:, F:]
        v = act(name, g)[0]
        ev = act_bound(name, g, v, eg)
        y = v * u
        agrees(h[:12], y, (ev * u.abs() + (v.abs() + ev) * eu) + 2 * U * y.abs() + rounding(y, t), "h")
        assert bool(torch.isfinite(h[6:]).all())
        clean(s, M, F, "h")


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("M,N,K", [(6, 136, 128), (130, 208, 272), (1270, 1288, 272), (50, 70, 33)])
def test_large_from_scales_and_bias(tg, ws, name, M, N, K):
    """8-bit inputs with large scales, and an fp32 bias beside 16-bit inputs."""
    x, w = rand(M, K, DT["fp8"], 1), rand(N, K, DT["fp8"], 2)
    alpha = 2.0 ** 100
    for od in ("bf16", "f32"):
        y = out(M, N, DT[od])[1]
        tg.tg_linear(x, w, y, act=name, scale_x=2.0 ** 50, scale_w=2.0 ** 50, workspace=ws)
        z, tol = product(x, w, alpha, FP8_INNER)
        v = act(name, z)[0]
        agrees(y, v, act_bound(name, z, v, tol) * (1 + 2.0 ** -7) + rounding(v, DT[od]), f"y {od}")
    F = N // 2
    h = out(M, F, DT["bf16"])[1]
    wide = w[:2 * F].float()
    wide[F:] = 0.0
    wide[F:, 0] = 2.0 ** -9  # (the squares of many g leave fp32's range, g * u stays in it)
    w[:2 * F].copy_(wide)
    tg.tg_glu(x, w[:2 * F], h, act=name, scale_x=2.0 ** 31, scale_w=2.0 ** 30, workspace=ws)
    p, b = product(x, w[:2 * F], 2.0 ** 61, FP8_INNER)
    g, u, eg, eu = p[:, :F], p[:, F:], b[:, :F], b[:, F:]
    v = act(name, g)[0]
    ev = act_bound(name, g, v, eg)
    agrees(h, v * u, (ev * u.abs() + (v.abs() + ev) * eu) + 2 * U * (v * u).abs() + rounding(v * u, DT["bf16"]), "h")
    x, w = rand(M, K, DT["f16"], 3), rand(N, K, DT["f16"], 4, K ** -0.5)
    bias = torch.tensor([1e20, -1e20, 3e38, -3e38, 2e19, -2e19, 1.0, -1.0], device="cuda").repeat(N // 8 + 1)[:N].contiguous()
    y = out(M, N, DT["f32"])[1]
    tg.tg_linear(x, w, y, bias=bias, act=name, workspace=ws)
    z, tol = product(x, w)
    z = z + bias.double()
    tol = tol + 4 * U * z.abs() + 2 * U * bias.double().abs()
    v = act(name, z)[0]
    agrees(y, v, act_bound(name, z, v, tol) * (1 + 2.0 ** -7) + rounding(v, DT["f32"]), "y, bias")


@pytest.mark.parametrize("name", ACTS)
def test_slopes_at_large_preactivations(tg, ws, name):
    t = torch.bfloat16
    M, N, K = 40, 64, 72
    dy, x, w, z = rand(M, N, t, 1), rand(M, K, t, 2), rand(N, K, t, 3), rand(M, N, t, 4)
    for r, v in enumerate(LARGE[2:]):
        z[r] = v
    dz, db = out(M, N, t)[1], torch.empty(N, device="cuda")
    tg.tg_linear_backward(dy, x, w, dbias=db, preact=z, act=name, dz=dz, workspace=ws)
    want = dy.double() * act(name, z.double())[1]
    agrees(dy if name == "none" else dz, want, dy.double().abs() * slope_bound(name) + U * want.abs() + rounding(want, t), "dz")


@pytest.mark.parametrize("in_place", [False, True])
def test_infinite_max_norm_clips_nothing(tg, ws, in_place):
    """Whatever the norm, infinity included; only a NaN still reaches every output."""
    norm = torch.empty(1, device="cuda")
    for bad in (0.0, 3e38, INF, -INF):
        grads = [torch.randn(9001, device="cuda"), torch.randn(77, device="cuda", dtype=torch.bfloat16), torch.zeros(3, device="cuda")]
        grads[0][8] = bad
        before = [g.clone() for g in grads]
        outs = grads if in_place else [torch.full_like(g, float("nan")) for g in grads]
        tg.tg_clip_grads(grads, INF, out=None if in_place else outs, norm=norm, workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(outs, before)), bad
        assert (float(norm) == INF) == (abs(bad) == INF)
    grads[0][8] = float("nan")
    tg.tg_clip_grads(grads, INF, norm=norm, workspace=ws)
    assert bool(norm.isnan().all()) and all(bool(g.isnan().all()) for g in grads)
    a = torch.ones(5, device="cuda")  # a finite max_norm takes an infinite norm to the factor 0
    a[2] = INF
    tg.tg_clip_grads([a], 1e30, norm=norm, workspace=ws)
    assert float(norm) == INF and bool(a[2].isnan()) and not a[:2].any() and not a[3:].any()


def one_row(cols, t, seed):
    """A row of a 16-bit matrix whose stride is off the 16-byte grid, NaN around it."""
    s = torch.full((10, -(-cols // 16) * 16 + 1), float("nan"), device="cuda").to(t)
    r = s[8:9, :cols]  # (starts on the grid)
    r.copy_(rand(1, cols, t, seed))
    return r


@pytest.mark.parametrize("K", [8, 33, 64, 200, 4104])
def test_one_token_with_any_stride(tg, ws, K):
    """A token taken out of a matrix with unaligned rows, and contiguous rows of odd width."""
    t, N = torch.bfloat16, 77
    x, w = one_row(K, t, 1), rand(N, K, t, 2, K ** -0.5)
    res, pre, y = (one_row(N, t, 3 + i) for i in range(3))
    tg.tg_linear(x, w, y, act="silu", residual=res, preact=pre, workspace=ws)
    z, tol = product(x, w)
    v = act("silu", z)[0]
    agrees(pre, z, tol + rounding(z, t), "preact")
    agrees(y, v + res.double(), (act_bound("silu", z, v, tol) + 2 * U * (v + res.double()).abs()) * (1 + 2.0 ** -7) + rounding(v + res.double(), t), "y")
    h = torch.empty(1, 38, device="cuda", dtype=t)
    tg.tg_glu(x, w[:76], h, workspace=ws)
    g, u, eg, eu = z[:, :38], z[:, 38:76], tol[:, :38], tol[:, 38:76]
    v = act("silu", g)[0]
    ev = act_bound("silu", g, v, eg)
    agrees(h, v * u, (ev * u.abs() + (v.abs() + ev) * eu) + 2 * U * (v * u).abs() + rounding(v * u, t), "h")
    dx, dw = one_row(K, t, 6), rand(N, K, t, 7)
    tg.tg_linear_backward(y, x, w, dx=dx, dw=dw, workspace=ws)
    p, b = product(y, w.t())
    agrees(dx, p, b + rounding(p, t), "dx")
    p = y.double().t() @ x.double()
    agrees(dw, p, 4 * U * p.abs() + rounding(p, t), "dw")


# weight gradients of one, two and three K steps that fill whole rounds of 256 tiles, the last ones with ragged edges
@pytest.mark.parametrize("M,N,K", [(64, 4096, 4096), (1, 8192, 2048), (100, 8192, 8192), (130, 8192, 8184), (40, 4088, 4096)])
@pytest.mark.parametrize("dt,od", [("bf16", "bf16"), ("f16", "f32")])
def test_linear_backward_whole_rounds(tg, ws, M, N, K, dt, od):
    bwd_case(tg, M, N, K, dt, od, "none", ws)


@pytest.mark.parametrize("M,F,D", [(16, 4096, 4096), (60, 4096, 4096), (130, 8192, 4096), (60, 4088, 4096)])
def test_glu_backward_whole_rounds(tg, ws, M, F, D):
    glu_bwd_case(tg, M, F, D, "bf16", "bf16", "silu", ws)


@pytest.mark.parametrize("M", [8, 40, 200])
def test_gelu_tail_holds_its_digits(tg, ws, M):
    """gelu over its whole negative tail, relative to its value: the pre-activation is an fp32 bias beside a product
    of zeros, so that it is exact.  Phi's fit is off by 1.5e-6 of it at most; beside that come the roundings of its
    seven coefficients and steps, the reciprocal and the exponential (under 24 u together) and three roundings of the
    exponent x^2/2.  Below -13 Phi leaves fp32's normal range."""
    N = 4096
    z = torch.linspace(-12.5, 12.5, N, device="cuda")
    x, w = torch.zeros(M, 64, device="cuda", dtype=torch.float16), torch.zeros(N, 64, device="cuda", dtype=torch.float16)
    want = act("gelu", z.double())[0]
    rel = 1.6e-6 + U * (24 + 1.5 * z.double().square())
    for od in (torch.float32, torch.float16):
        y = torch.empty(M, N, device="cuda", dtype=od)
        tg.tg_linear(x, w, y, bias=z, act="gelu", workspace=ws)
        tol = rel * want.abs() + rounding(want, od)
        agrees(y, want.expand(M, N), tol.expand(M, N), str(od))
    x, w, y = x.bfloat16(), w.bfloat16(), torch.empty(M, N, device="cuda", dtype=torch.bfloat16)
    tg.tg_linear(x, w, y, bias=z, act="gelu", workspace=ws)
    agrees(y, want.expand(M, N), (rel * want.abs() + rounding(want, torch.bfloat16)).expand(M, N), "bf16")


def test_gradients_through_weights_past_2_gib(tg, ws):
    """dX = dZ . W and dH = dY . Wd with row-major weights that span more than one buffer descriptor: another kernel
    takes them."""
    t = torch.bfloat16
    M, N, K = 24, 131_080, 8200  # W: 2.15 GB
    dy, x, w = rand(M, N, t, 1), rand(M, K, t, 2), rand(N, K, t, 3, K ** -0.5)
    s, dx = out(M, K, t)
    tg.tg_linear_backward(dy, x, w, dx=dx, workspace=ws)
    want, size = 0.0, 0.0
    for i in range(0, N, 16_384):
        a, b = dy[:, i:i + 16_384].double(), w[i:i + 16_384].double()
        want, size = want + a @ b, size + a.abs() @ b.abs()
    agrees(dx, want, 2 * N * U * size + 4 * U * want.abs() + rounding(want, t), "dx")
    clean(s, M, K, "dx")
    del w, x
    F, D = 131_080, 8200  # Wd: D x F
    dy, wd, gu = rand(M, D, t, 4), rand(D, F, t, 5, F ** -0.5), rand(M, 2 * F, t, 6)
    s, dgu = out(M, 2 * F, t)
    w, x = torch.empty(2 * F, D, device="cuda", dtype=t), rand(M, D, t, 7)  # (not read: no dx, no dw)
    tg.tg_glu_backward(dy, wd, x, w, gu, None, dgu, workspace=ws)
    for i in range(0, F, 16_384):
        j = min(F, i + 16_384)
        g, u = gu[:, i:j].double(), gu[:, F + i:F + j].double()
        dh, e = product(dy, wd[:, i:j].t())
        v, slope = act("silu", g)
        es, ev = slope_bound("silu"), act_bound("silu", g, v, torch.zeros_like(g))
        dg, du = dh * u * slope, dh * v
        agrees(dgu[:, i:j], dg, (e * slope.abs() + (dh.abs() + e) * es) * u.abs() + 3 * U * dg.abs() + rounding(dg, t), "dg")
        agrees(dgu[:, F + i:F + j], du, e * v.abs() + (dh.abs() + e) * ev + U * du.abs() + rounding(du, t), "du")
    clean(s, M, 2 * F, "dgate_up")
