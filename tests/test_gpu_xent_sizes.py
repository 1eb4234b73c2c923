"""The vocabulary loss on the GPU at the ends of its range of sizes."""
import pytest
import torch

from test_gpu_xent import BF, F16, MARK, free, space

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import tile_level_gemm_02_amd as tg

    return tg


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("V", [0, 10, 32000])
def test_no_rows_in_the_querys_bytes(tg, dtype, V):
    """An empty batch's total is two zeros, in a workspace of exactly the query's bytes."""
    w, e = torch.zeros(V, 16, device="cuda", dtype=dtype), torch.zeros(0, device="cuda")
    x, target = torch.zeros(0, 16, device="cuda", dtype=dtype), torch.zeros(0, device="cuda", dtype=torch.int64)
    ws = space(tg.tg_linear_xent_workspace_bytes(dtype, 0, V, 16))
    for _ in range(2):
        total = torch.full((4,), MARK, device="cuda")
        tg.tg_linear_xent(x, w, target, e, e, total[:2], workspace=ws)
        assert total.tolist() == [0.0, 0.0, MARK, MARK]
        free(ws)
