"""tg_adamw on the GPU at the ends of its numbers: gradients that are not finite
beside 8-bit states' other values."""
import pytest
import torch

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
