"""The vocabulary loss on the GPU at the ends of its range of sizes."""
import pytest
import torch

from _train_ref import within, xent
from test_gpu_xent import BF, F16, IGNORE, MARK, free, gen, space

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


def test_more_rows_than_a_launch_of_the_join_has_lanes_for(tg):
    """2^28 rows and a few, 16 to a workgroup of 256 lanes: 2^32 lanes and more, and a total over all of them."""
    M, V, D = (1 << 28) + 5003, 8, 8
    need = tg.tg_linear_xent_workspace_bytes(BF, M, V, D)
    if torch.cuda.mem_get_info()[0] < need + (24 << 30):
        pytest.skip("device memory")
    x = torch.empty(M, D, device="cuda", dtype=BF).normal_(generator=gen(1))
    w = torch.empty(V, D, device="cuda", dtype=BF).normal_(generator=gen(2))
    target = torch.randint(0, V, (M,), device="cuda", generator=gen(3))
    target[::5] = IGNORE
    loss, lse, total = (torch.empty(n, device="cuda") for n in (M, M, 2))
    ws = torch.zeros(need // 4, dtype=torch.int32, device="cuda")
    tg.tg_linear_xent(x, w, target, loss, lse, total, scale=0.9, ignore_index=IGNORE, workspace=ws)
    free(ws)
    want, off = 0.0, 0.0
    for i in range(0, M, 1 << 24):
        rows = slice(i, min(M, i + (1 << 24)))
        a, lse64, dl, de = xent(x[rows], w, target[rows], 0.9, IGNORE, 0.0)
        within(lse[rows], lse64, de, "lse")
        within(loss[rows], a, dl, "loss")
        want, off = want + float(a.sum()), off + float(dl.sum())
    # (the counted rows as the nearest fp32 number)
    count = torch.tensor(float((target != IGNORE).sum()))
    assert float(total[1]) == float(count) and abs(float(total[0]) - want) <= off + 2.0 ** -23 * want
    again = torch.empty(2, device="cuda")
    tg.tg_linear_xent(x, w, target, None, None, again, scale=0.9, ignore_index=IGNORE, workspace=ws)
    assert torch.equal(again, total)
