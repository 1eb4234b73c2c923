"""The vocabulary loss's gradient on the GPU beside values that are not finite."""
import pytest
import torch

from _train_ref import rounded, within, xent_grad
from test_gpu_xent import BF, F16, F32, IGNORE, gen, problem, space

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import tile_level_gemm_02_amd as tg

    return tg


@pytest.mark.parametrize("dtype", [F16, BF])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("M", [70, 3000])
def test_a_factor_that_is_not_finite_spoils_its_own_row_alone(tg, dtype, bad, M):
    """Every other row's dx is that of the call in which the row is ignored, bit for bit, and within its bound."""
    V, D, z = 500, 64, 1e-3
    x, w, target = problem(M, V, D, dtype)
    target[5] = 7
    lse = torch.logsumexp(x.double() @ w.double().t().contiguous(), 1).float()
    dloss = (torch.rand(M, device="cuda", generator=gen(9)) + 0.1) * 100
    ws = space(tg.tg_linear_xent_backward_workspace_bytes(dtype, M, V, D))

    def call(target, dloss):
        dx = torch.empty(M, D, device="cuda", dtype=dtype)
        tg.tg_linear_xent_backward(x, w, target, lse, dx=dx, dloss=dloss, ignore_index=IGNORE, z_loss=z, grad_scale=1e-3, workspace=ws)
        return dx

    spoilt = dloss.clone()
    spoilt[5] = bad
    without = target.clone()
    without[5] = IGNORE
    a, b = call(target, spoilt), call(without, dloss)
    other = torch.arange(M, device="cuda") != 5
    assert not bool(a[5].isfinite().any()) and torch.equal(a[other], b[other])
    want, _, bound, _ = xent_grad(x, w, without, 1.0, IGNORE, z, lse, 1e-3 * dloss.double(), dtype)
    within(b, want, bound + rounded(want, dtype), "dx")
