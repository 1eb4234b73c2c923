"""The vocabulary loss on the GPU at the ends of its range of sizes."""
import pytest
import torch

from _train_ref import U, adds, logits, within, xent
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


@pytest.fixture(autouse=True)
def _room():
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def far_ends(tg, M, V, D, rows, ends, room=24):
    """The loss of M x V logits at `rows`, whose targets take the columns in `ends` and others, against sums in 64 bits."""
    need = tg.tg_linear_xent_workspace_bytes(BF, M, V, D)
    if torch.cuda.mem_get_info()[0] < need + 2 * D * (M + V) + (room << 30):
        pytest.skip("device memory")
    print(f"xent {M}x{V}x{D}", flush=True)
    x = torch.empty(M, D, device="cuda", dtype=BF).normal_(generator=gen(1))
    w = torch.empty(V, D, device="cuda", dtype=BF)
    for i in range(0, V, 1 << 26):
        w[i:i + (1 << 26)].normal_(generator=gen(2))
    w[-1] = x[rows[0]] * 2  # (a last column that its row's sum would miss)
    target = torch.randint(0, V, (M,), device="cuda", generator=gen(3))
    rows = torch.tensor(rows, device="cuda")
    target[rows] = torch.tensor([ends[i % len(ends)] for i in range(len(rows))], device="cuda")
    target[rows[-1]] = IGNORE
    loss, lse, total = (torch.empty(n, device="cuda") for n in (M, M, 2))
    ws = torch.zeros(need // 4, dtype=torch.int32, device="cuda")
    tg.tg_linear_xent(x, w, target, loss, lse, total, ignore_index=IGNORE, workspace=ws)
    free(ws)
    del ws
    # rows' sums over parts of the vocabulary; the bound of each logit and of its exponential as _train_ref's, their largest
    part, a = max(1 << 16, (1 << 28) // len(rows)), x[rows]
    sums, off, tops = [], 0.0, 0.0
    for i in range(0, V, part):
        t, dt = logits(a, w[i:i + part], 1.0)
        sums.append(torch.logsumexp(t, 1))
        off, tops = torch.clamp(dt.amax(1), min=off), torch.clamp(t.abs().amax(1), min=tops)
    lse64 = torch.logsumexp(torch.stack(sums), 0)
    de = off + 4 * U * (tops + lse64.abs()) + 4 * U + 2 * adds(V) * U + 2 * U * lse64.abs()
    within(lse[rows], lse64, de, "lse")
    counts = target[rows] != IGNORE
    tt = (a.double() * w[target[rows].clamp(min=0)].double()).sum(1)
    within(loss[rows], torch.where(counts, lse64 - tt, 0.0), de + off + 4 * U * (lse64.abs() + tt.abs()), "loss")
    # all of them: the total is their sum
    assert float(total[1]) == float(torch.tensor(float((target != IGNORE).sum())))
    want = float(loss.double().sum())
    assert abs(float(total[0]) - want) <= 2.0 ** -23 * want and bool(loss.isfinite().all())


def test_more_tiles_than_a_launch_has_lanes_for(tg):
    """2^39 logits and more: the rows go in two launches of 2^23 tiles of 512 lanes, the second from row 8355840 on."""
    M, V = (1 << 23) + 301, (1 << 16) + 64
    cut = 8355840
    rows = list(range(40)) + list(range(cut - 40, cut + 40)) + list(range(M - 40, M))
    far_ends(tg, M, V, 8, rows, [0, V - 1, V - 2, 65535, 65536, 777])


def test_wide_vocabularies(tg):
    """Few rows against more columns than the few-rows kernel's launch has lanes for, and more than 2^30 columns, which go in parts."""
    for V in ((1 << 27) - 16, (1 << 27) + 77):
        far_ends(tg, 3, V, 8, [0, 1, 2], [V - 1, 0])
    V = (1 << 30) + 300
    far_ends(tg, 33, V, 8, list(range(33)), [V - 1, 0, (1 << 30) - 1, 1 << 30, (1 << 30) + 63, (1 << 30) + 64, 12345])
