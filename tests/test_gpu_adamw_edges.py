"""tg_adamw on the GPU at the ends of its numbers: gradients that are not finite
beside 8-bit states' other values, and second moments below fp32's normal
numbers."""
import pytest
import torch

from _train_ref import U, rounded
from test_gpu_adamw import BF, F16, F32, Tensor, step_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import tile_level_gemm_02_amd as tg

    return tg


def bits(t):
    return t.contiguous().view(torch.uint8).view(t.numel(), -1)


AT = 300  # in the second block of 256


@pytest.mark.parametrize("p,g,master", [(F32, F32, False), (BF, BF, False), (BF, BF, True), (F16, F32, False)])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), 1e20])
@pytest.mark.parametrize("eight", [False, True])
def test_one_gradient_spoils_its_own_element_alone(tg, p, g, master, bad, eight):
    """Two steps against the same ones with a gradient of 0 there, whose m and v are 0: every other element's weight and root
    is the same bit for bit, and its m too unless a finite value sets the block's scale of m."""
    made = []
    for value in (bad, 0.0):
        t = Tensor(1000, p, g, master, eight, 11)
        for k in ("m", "v"):
            t.t[k].view(torch.uint8).view(1000, -1)[AT] = 0
        for step in (1, 2):
            t.t["g"][AT] = value if step == 1 else 0.25
            step_of(tg, [t], step)
            made.append({k: v.clone() for k, v in t.t.items()})
    other = torch.arange(1000, device="cuda") != AT
    for step in (0, 1):
        a, b = made[step], made[2 + step]
        for k in a:
            if k in ("sm", "sv"):
                # (the second step's own 0.25 counts only where nothing was spoilt)
                same = torch.tensor([True, step == 0 and not (k == "sm" and bad == 1e20), True, True], device="cuda")
                assert bool(a[k].isfinite().all()) and torch.equal(a[k][same], b[k][same]), (step, k)
            elif eight and (k == "m" and bad == 1e20 or step == 1):
                assert bool(a[k].float()[other].isfinite().all()), (step, k)
                far = torch.cat([other[:256].nonzero(), 512 + other[512:].nonzero()]).flatten()
                assert torch.equal(bits(a[k])[far], bits(b[k])[far]), (step, k)
            else:
                assert torch.equal(bits(a[k])[other], bits(b[k])[other]), (step, k)
        name = "w" if master else "p"
        if bad != 1e20:
            assert bool(a[name][AT].isnan()) and bool(a["m"].float()[AT].isnan() if eight else a["m"][AT].isinf() or step == 1)
        if eight:
            assert bool(a["v"].float()[AT].isnan())
    # the spoilt block's other weights are finite after the second step, which reads what the first one held
    w = made[1]["w" if master else "p"].float()[other]
    assert bool(w.isfinite().all())


@pytest.mark.parametrize("eps", [0.0, 1e-22, 1e-20, 1e-8])
@pytest.mark.parametrize("p", [F32, BF])
def test_roots_of_subnormal_second_moments(tg, p, eps):
    """fp32 states whose v' runs from a few of the smallest steps to normal numbers: the update against its definition of the m' and v'
    that the step wrote (12 u of it, and the weight's own roundings)."""
    n = 3000
    t = Tensor(n, p, F32, False, False, 7)
    t.t["g"].copy_(10.0 ** torch.linspace(-22, -18, n, device="cuda"))  # v' = 0.05 g^2: 5e-46 (0 or a step) to 5e-38
    for k in ("m", "v"):
        t.t[k].zero_()
    t.t["p"].fill_(0.5)
    h = dict(lr=1e-2, b1=0.9, b2=0.95, wd=0.0)
    tg.tg_adamw([t.t["p"]], [t.t["g"]], [t.t["m"]], [t.t["v"]], 3, h["lr"], betas=(h["b1"], h["b2"]), eps=eps, weight_decay=0.0)
    m, v = t.t["m"].double(), t.t["v"].double()
    step = 2.0 ** -149
    want = (0.05 * t.t["g"].double() ** 2)
    assert bool(((v - want).abs() <= step / 2 * (1 + 2.0 ** -20) + 4 * U * want).all()) and int((v < 2.0 ** -126).sum()) > n // 2
    some = v > 0
    up = h["lr"] / (1 - h["b1"] ** 3) * m / ((v / (1 - h["b2"] ** 3)).sqrt() + eps)
    w = t.t["p"].double()
    off = (w - (0.5 - up)).abs() - (12 * U * up.abs() + 4 * U * 0.5 + rounded(0.5 - up, p))
    assert bool((off[some] <= 0).all()), float(off[some].max())


def test_8_bit_roots_of_subnormal_second_moments(tg):
    """A block whose sqrt(v') is above 2^-100 is held by its roots, though v' is subnormal."""
    t = Tensor(512, F32, F32, False, True, 1)
    for k in ("m", "v"):
        t.t[k].view(torch.uint8).zero_()
    t.t["g"].fill_(1e-20)
    t.t["g"][256:] = 3e-21
    g = t.t["g"][::256].cpu()
    step_of(tg, [t], 3)
    omb2 = torch.tensor(1 - 0.95, dtype=torch.float64).float()
    v = (g * omb2 * g).double()  # (5e-42 and 4.5e-43, each rounded to a multiple of 2^-149)
    sv = t.t["sv"].cpu().double()
    assert bool(((sv / (v.sqrt() / 448) - 1).abs() <= 6 * U).all()), sv
    assert bool((t.t["v"].float() == 448).all())


@pytest.mark.parametrize("eps", [1e-320, 1e-45, 1e-40, 2.0 ** -126, 1e-30])
@pytest.mark.parametrize("eight", [False, True])
def test_a_small_eps_leaves_weights_without_gradients(tg, eps, eight):
    """m' = v' = 0 over eps > 0 is 0: rows of an embedding that no token took keep their weights."""
    t = Tensor(600, F32, F32, False, eight, 5)
    for k in ("g", "m", "v"):
        t.t[k].view(torch.uint8).zero_()
    h = dict(exp_avg_scales=[t.t["sm"]], exp_avg_sq_scales=[t.t["sv"]]) if eight else {}
    tg.tg_adamw([t.t["p"]], [t.t["g"]], [t.t["m"]], [t.t["v"]], 3, 1e-2, eps=eps, weight_decay=0.0, **h)
    assert torch.equal(t.t["p"], t.before["p"])
