"""The 8-bit integer layers on the GPU past the sizes that one launch has lanes
for.  Sums of 16 products of int8 are whole numbers below 2^24, so an fp32
product gives them exactly, and the epilogue's fp32 operations, each rounded
once in the same order, give the same bits."""
import pytest
import torch

from test_gpu_int8 import BF, F32, I8, MARK, gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import tile_level_gemm_02_amd as tg

    return tg


def ints(rows, cols, seed):
    return torch.randint(-128, 128, (rows, cols), device="cuda", dtype=I8, generator=gen(seed))


def layer(tg, M, N, od, residual):
    """All of Y against its definition, in parts; K = 16."""
    ld = -(-N // 16) * 16
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 24 * (M + N) + 2 * M * ld * od.itemsize + (16 << 30):
        pytest.skip("device memory")
    print(f"i8 {M}x{N}x16 {od}", flush=True)
    x, w = ints(M, 16, 1), ints(N, 16, 2)
    sx, sw = (torch.rand(n, device="cuda", generator=gen(3)) + 0.5 for n in (M, N))
    bias = torch.rand(N, device="cuda", generator=gen(4))
    y = torch.full((M, ld), float(MARK), device="cuda", dtype=od)
    r = torch.rand(M, ld, device="cuda", dtype=od, generator=gen(5))[:, :N] if residual else None
    tg.tg_linear_i8(x, w, y[:, :N], sx, sw, bias=bias, residual=r, workspace=tg.tg_ops_workspace())
    rows, cols = min(M, 1 << 22), min(N, 1 << 24)
    for i in range(0, M, rows):
        for j in range(0, N, cols):
            a, b = slice(i, i + rows), slice(j, min(N, j + cols))
            z = (x[a].float() @ w[b].float().t().contiguous()) * (sx[a, None] * sw[b]) + bias[b]
            if residual:
                z = z + r[a, b].float()
            assert torch.equal(y[a, b], z.to(od)), (i, j)
    assert bool((y[:, N:] == MARK).all())


def test_few_rows_and_more_columns_than_a_launch_has_lanes_for(tg):
    for N in ((1 << 28) - 16, (1 << 28) + 40):
        layer(tg, 3, N, BF, False)
    layer(tg, 20, (1 << 28) + 40, BF, False)


def test_sizes_that_go_in_parts(tg):
    """Past 2^30 rows, of x and of W."""
    layer(tg, (1 << 30) + 300, 8, BF, True)
    layer(tg, 2, (1 << 30) + 50, F32, True)
