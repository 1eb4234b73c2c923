"""The vocabulary loss and its gradient on the GPU against their 64-bit
definitions: every kernel variant (few rows, each tile plan, pieces of the
vocabulary, K splits), both types, ragged sizes, rows that do not count, and
the values and calls that its contract names."""
import pytest
import torch

from _train_ref import rounded, within, xent, xent_grad

pytestmark = pytest.mark.gpu

BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
IGNORE = -100
MARK = 7.0


@pytest.fixture(scope="module")
def tg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import tile_level_gemm_02_amd as tg

    return tg


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def padded(rows, cols, dtype, fill, extra=8):
    s = torch.full((rows + 2, -(-cols // 8) * 8 + extra), fill, device="cuda", dtype=dtype)
    return s, s[:rows, :cols]


def rand(rows, cols, dtype, seed, std):
    _, t = padded(rows, cols, dtype, float("nan"), 16)
    return t.copy_(torch.empty(rows, cols, device="cuda").normal_(0.0, std, generator=gen(seed)))


def problem(M, V, D, dtype, seed=1, ignored=0.2):
    x, w = rand(M, D, dtype, seed, 1.0), rand(V, D, dtype, seed + 1, 2.0 * max(D, 1) ** -0.5)
    target = torch.randint(0, V, (M,), device="cuda", generator=gen(seed + 2))
    target[torch.rand(M, device="cuda", generator=gen(seed + 3)) < ignored] = IGNORE
    if M > 2:
        target[0], target[1] = V - 1, 0
    return x, w, target


def space(n):
    """A workspace whose scratch holds NaN."""
    ws = torch.full(((n + 3) // 4,), -1, dtype=torch.int32, device="cuda")
    ws[:16384] = 0
    return ws


def free(ws):
    assert int(ws[:16384].count_nonzero()) == 0, "arrival counters not zero after the call"


def vector(n):
    return torch.full((n + 2,), MARK, device="cuda")


def forward(tg, x, w, target, scale=1.0, z=0.0, ws=None):
    M, D = x.shape
    ws = space(tg.tg_linear_xent_workspace_bytes(x.dtype, M, w.shape[0], D)) if ws is None else ws
    loss, lse, total = vector(M), vector(M), vector(2)
    tg.tg_linear_xent(x, w, target, loss[:M], lse[:M], total[:2], scale=scale, ignore_index=IGNORE, z_loss=z, workspace=ws)
    torch.cuda.synchronize()
    for v, n in ((loss, M), (lse, M), (total, 2)):
        assert bool((v[n:] == MARK).all())
    free(ws)
    return loss[:M], lse[:M], total[:2]


def check_forward(tg, M, V, D, dtype, scale=0.9, z=1e-3, seed=1):
    print(f"xent {M}x{V}x{D} {dtype}", flush=True)
    x, w, target = problem(M, V, D, dtype, seed)
    loss, lse, total = forward(tg, x, w, target, scale, z)
    want, lse64, dl, de = xent(x, w, target, scale, IGNORE, z)
    within(lse, lse64, de, "lse")
    within(loss, want, dl, "loss")
    within(total[0], want.sum(), dl.sum() + 2.0 ** -23 * want.abs().sum(), "total")
    assert int(total[1]) == int((target != IGNORE).sum())
    return x, w, target, lse, total


# few rows (one and two slices, wide and narrow workgroups); 128 tiles with both rings; 256 x 128; 256; a short last round in
# 256 x 128 and 128 parts (also where the plan asks for 64)
@pytest.mark.parametrize("M,V,D", [(1, 1, 8), (1, 17, 64), (2, 1000, 136), (8, 4097, 200), (9, 8300, 72), (16, 333, 1032), (17, 1500, 264),
                                   (32, 65, 8), (33, 63, 64), (40, 200, 520), (65, 129, 72), (130, 5003, 136), (1270, 1281, 72),
                                   (2300, 2290, 136), (3580, 3570, 72), (777, 32003, 136), (4600, 5300, 72), (4352, 4352, 64),
                                   (4360, 4350, 136), (140000, 40, 8)])
@pytest.mark.parametrize("dtype", [BF, F16])
def test_loss(tg, M, V, D, dtype):
    check_forward(tg, M, V, D, dtype)


def backward_case(tg, M, V, D, dtype, dw_dtype, piece=0, weighted=False, counted=True, z=1e-3, scale=0.9, gs=3.0, ldw=None, seed=1):
    print(f"xent backward {M}x{V}x{D} {dtype} piece {piece}", flush=True)
    x, w, target = problem(M, V, D, dtype, seed)
    t = scale * (x.double() @ w.double().t().contiguous())
    lse = torch.logsumexp(t, 1).float()
    dloss = torch.rand(M, device="cuda", generator=gen(9)) * 2 - 0.5 if weighted else None
    if weighted:
        dloss[target == IGNORE] = float("nan")  # not read
    total = torch.tensor([0.0, float((target != IGNORE).sum())], device="cuda") if counted else None
    n = tg.tg_linear_xent_backward_workspace_bytes(dtype, M, V, D, piece)
    ws = space(n)
    sx, dx = padded(M, D, dtype, MARK)
    sw, dw = padded(V, D, dw_dtype, MARK)
    tg.tg_linear_xent_backward(x, w, target, lse, dx=dx, dw=dw, dloss=dloss, total=total, grad_scale=gs, scale=scale, ignore_index=IGNORE,
                               z_loss=z, workspace=ws)
    torch.cuda.synchronize()
    free(ws)
    g = torch.full((M,), gs / (max(1.0, float(total[1])) if counted else 1.0), device="cuda", dtype=torch.float64)
    if weighted:
        g = g * torch.nan_to_num(dloss.double())
    wx, ww, bx, bw = xent_grad(x, w, target, scale, IGNORE, z, lse, g, dtype)
    within(dx, wx, bx + rounded(wx, dtype), "dx")
    within(dw, ww, bw + rounded(ww, dw_dtype), "dw")
    for s, rows in ((sx, M), (sw, V)):
        assert bool((s[rows:] == MARK).all()) and bool((s[:, D:] == MARK).all()), "wrote outside its matrix"


# one piece and several (a last one of one column, of 8 k + 1, of whole chunks), a row and many, K split and tiles of every size
@pytest.mark.parametrize("M,V,D,piece", [(1, 1, 8, 0), (1, 300, 64, 0), (5, 257, 72, 1), (33, 1000, 136, 256), (100, 769, 520, 1),
                                         (300, 5003, 264, 1024), (777, 3201, 136, 0), (1270, 1281, 72, 512), (200, 70003, 64, 0),
                                         (512, 9000, 1032, 4096), (2300, 2290, 136, 0), (4100, 513, 256, 0), (4352, 4400, 64, 0),
                                         # one piece, which has no sums of dx, needs less than two
                                         (160, 452, 1256, 512), (160, 452, 1256, 1),
                                         # the rows' largest factor in several passes of its workgroups
                                         (140000, 40, 8, 0),
                                         # dx's K, the vocabulary, over workgroups whose partial tiles a kernel adds; over pieces as well
                                         (600, 70003, 264, 0), (600, 70003, 264, 65536), (129, 131080, 520, 0)])
@pytest.mark.parametrize("dtype,dw_dtype", [(BF, BF), (BF, F32), (F16, F16), (F16, F32)])
def test_gradients(tg, M, V, D, piece, dtype, dw_dtype):
    backward_case(tg, M, V, D, dtype, dw_dtype, piece, weighted=piece == 0, counted=M % 2 == 1)


def test_gradients_of_a_weight_whose_rows_lie_far_apart(tg, monkeypatch):
    """4500 rows over 2 GiB take two pieces, and dx's sums, in a workspace whose query had one piece in mind."""
    M, V, D = 160, 4500, 1256
    w = torch.empty(V, 240000, device="cuda", dtype=BF)[:, :D]
    near = problem

    def far(*a):
        x, v, target = near(*a)
        return x, w.copy_(v), target

    monkeypatch.setitem(globals(), "problem", far)
    for piece in (0, 1, 4608):
        backward_case(tg, M, V, D, BF, F32, piece)


def test_gradients_of_small_probabilities_and_large_factors(tg):
    """fp16: factors far from 1 (loss scaling, a mean over many rows) do not cost the small probabilities their digits."""
    for gs in (65536.0, 2.0 ** -8):
        backward_case(tg, 200, 4000, 64, F16, F32, gs=gs, counted=True)
    backward_case(tg, 70, 500, 64, F16, F16, z=0.5)  # 1 + 2 z lse about 8
    backward_case(tg, 70, 500, 64, BF, BF, scale=-1.3)


def test_gradient_against_differences(tg):
    """Along the gradient's own signs a difference of the loss does not cancel.  The loss in 64 bits at x +- e s: the
    difference is e^2 / 6 of a third derivative off (bounded by scale^3 |W|^3-sized terms, under 1e-4 here), the
    gradient by its own bound."""
    M, V, D = 40, 300, 64
    x, w, target = problem(M, V, D, BF)
    _, lse, total = forward(tg, x, w, target)
    dx, dw = torch.empty(M, D, device="cuda", dtype=BF), torch.empty(V, D, device="cuda")
    ws = space(tg.tg_linear_xent_backward_workspace_bytes(BF, M, V, D))
    tg.tg_linear_xent_backward(x, w, target, lse, dx=dx, dw=dw, total=total, ignore_index=IGNORE, workspace=ws)

    def mean(a, b):
        t = a @ b.t().contiguous()
        counts = target != IGNORE
        loss = torch.logsumexp(t, 1) - t.gather(1, target.clamp(min=0)[:, None])[:, 0]
        return float(torch.where(counts, loss, 0.0).sum() / counts.sum())

    a, b, e = x.double(), w.double(), 1e-4
    for grad, shift in ((dx, lambda s, k: mean(a + k * e * s, b)), (dw, lambda s, k: mean(a, b + k * e * s))):
        s = grad.double().sign()
        slope, want = float((grad.double() * s).sum()), (shift(s, 1) - shift(s, -1)) / (2 * e)
        assert abs(slope / want - 1) < 2 * 2.0 ** -8, (slope, want)


def test_rows_that_do_not_count(tg):
    M, V, D = 70, 500, 64
    x, w, target = problem(M, V, D, BF)
    target[:] = IGNORE
    loss, lse, total = forward(tg, x, w, target, z=1e-2)
    assert bool((loss == 0).all()) and total.tolist() == [0.0, 0.0] and bool(torch.isfinite(lse).all())
    dx, dw = torch.full((M, D), MARK, device="cuda", dtype=BF), torch.full((V, D), MARK, device="cuda", dtype=BF)
    ws = space(tg.tg_linear_xent_backward_workspace_bytes(BF, M, V, D, 1))
    tg.tg_linear_xent_backward(x, w, target, lse, dx=dx, dw=dw, total=total, ignore_index=IGNORE, workspace=ws)
    assert bool((dx == 0).all()) and bool((dw == 0).all())
    # an ignored row's NaN stays in its lse and reaches neither the total nor its dx
    target[5] = 3
    x[7] = float("nan")
    loss, lse, total = forward(tg, x, w, target)
    assert bool(lse[7].isnan()) and float(loss[7]) == 0.0 and total[1] == 1 and abs(float(total[0] - loss[5])) <= 1e-6 * float(loss[5])
    tg.tg_linear_xent_backward(x, w, target, lse, dx=dx, dw=None, total=total, ignore_index=IGNORE, workspace=ws)
    assert bool((dx[7] == 0).all()) and bool(dx[5].isfinite().all()) and float(dx[5].abs().max()) > 0


@pytest.mark.parametrize("M", [3, 300])
def test_targets_out_of_range_and_logits_that_are_not_finite(tg, M):
    V, D = 700, 64
    x, w, target = problem(M, V, D, F16, ignored=0.0)
    target[1], target[2] = V, -1
    loss, lse, total = forward(tg, x, w, target)
    assert loss.isnan().tolist()[:3] == [False, True, True] and bool(lse.isfinite().all()) and bool(total[0].isnan()) and total[1] == M
    dx = torch.empty(M, D, device="cuda", dtype=F16)
    ws = space(tg.tg_linear_xent_backward_workspace_bytes(F16, M, V, D))
    tg.tg_linear_xent_backward(x, w, target, lse, dx=dx, ignore_index=IGNORE, workspace=ws)
    assert bool(dx[1:3].isnan().all()) and bool(dx[0].isfinite().all())
    # minus infinity is a probability of 0: a whole wave's columns, all but one column
    target[:] = 5
    x.fill_(1.0)
    w.fill_(0.0)
    w[:] = -65504.0  # D of them: -4.2 million, e^t = 0 beside t = 0
    w[5] = 0.0
    loss, lse, _ = forward(tg, x, w, target)
    assert bool((loss == 0).all()) and bool((lse == 0).all())
    w[100:300, 0] = float("-inf")
    loss, lse, _ = forward(tg, x, w, target)
    assert bool((loss == 0).all()) and bool((lse == 0).all())
    w[:, 0] = float("-inf")  # no finite logit at all
    assert bool(forward(tg, x, w, target)[0].isnan().all())
    w[:] = 0.0
    w[3, 0] = float("inf")
    assert bool(forward(tg, x, w, target)[0].isnan().all())


def test_large_logits(tg):
    """Logits of +-2000, whose exponentials leave fp32: the sums are relative to each row's largest."""
    for scale in (300.0, -300.0):
        check_forward(tg, 70, 1000, 64, BF, scale=scale, z=0.0)
        check_forward(tg, 5, 1000, 64, BF, scale=scale, z=0.0)


def test_sizes_of_nothing(tg):
    w = torch.zeros(10, 16, device="cuda", dtype=BF)
    e = torch.zeros(0, device="cuda")
    x, target = torch.zeros(0, 16, device="cuda", dtype=BF), torch.zeros(0, device="cuda", dtype=torch.int64)
    total, dw = torch.full((2,), MARK, device="cuda"), torch.full((10, 16), MARK, device="cuda")
    ws = tg.tg_ops_workspace()
    tg.tg_linear_xent(x, w, target, e, e, total, workspace=ws)
    assert total.tolist() == [0.0, 0.0]
    ws = space(tg.tg_linear_xent_backward_workspace_bytes(BF, 0, 10, 16))
    tg.tg_linear_xent_backward(x, w, target, e, dx=x, dw=dw, total=total, workspace=ws)
    assert bool((dw == 0).all())
    # no width: every logit is 0
    x, w = torch.zeros(3, 0, device="cuda", dtype=BF), torch.zeros(50, 0, device="cuda", dtype=BF)
    loss = torch.empty(3, device="cuda")
    tg.tg_linear_xent(x, w, torch.tensor([1, 49, IGNORE], device="cuda"), loss, None, None, workspace=tg.tg_ops_workspace())
    want = torch.tensor([50.0, 50.0, 1.0], dtype=torch.float64).log()
    assert float((loss.cpu().double() - want).abs().max()) < 8 * 2.0 ** -24 * 4


def test_outputs_left_out_and_repeated_calls(tg):
    M, V, D = 300, 3000, 136
    x, w, target = problem(M, V, D, BF)
    loss, lse, total = forward(tg, x, w, target, z=1e-3)
    ws = space(tg.tg_linear_xent_workspace_bytes(BF, M, V, D))
    only = torch.empty(M, device="cuda")
    for k in ("loss", "lse"):
        tg.tg_linear_xent(x, w, target, **{k: only}, z_loss=1e-3, workspace=ws)
        assert torch.equal(only, loss if k == "loss" else lse)
    ws = space(tg.tg_linear_xent_backward_workspace_bytes(BF, M, V, D, 1024))

    def grads(dx, dw):
        tg.tg_linear_xent_backward(x, w, target, lse, dx=dx, dw=dw, total=total, z_loss=1e-3, workspace=ws)
        return dx, dw

    room = lambda n: torch.empty(n, D, device="cuda", dtype=BF)  # noqa: E731
    dx, dw = grads(room(M), room(V))
    assert torch.equal(grads(room(M), None)[0], dx) and torch.equal(grads(None, room(V))[1], dw)
    again = grads(room(M), room(V))
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


def test_captured_and_on_another_stream(tg):
    """A captured forward and backward replayed on new contents, eager calls between the replays, on their own workspaces."""
    M, V, D = 300, 5003, 136
    x, w, target = problem(M, V, D, BF)
    n = max(tg.tg_linear_xent_workspace_bytes(BF, M, V, D), tg.tg_linear_xent_backward_workspace_bytes(BF, M, V, D, 2048))
    side = torch.cuda.Stream()

    def state():
        return dict(loss=torch.empty(M, device="cuda"), lse=torch.empty(M, device="cuda"), total=torch.empty(2, device="cuda"),
                    dx=torch.empty(M, D, device="cuda", dtype=BF), dw=torch.empty(V, D, device="cuda"), ws=space(n))

    def call(s):
        tg.tg_linear_xent(x, w, target, s["loss"], s["lse"], s["total"], workspace=s["ws"])
        tg.tg_linear_xent_backward(x, w, target, s["lse"], dx=s["dx"], dw=s["dw"], total=s["total"], workspace=s["ws"])

    a, b, c = state(), state(), state()
    call(a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(b)
    for k in range(3):
        x.copy_(torch.empty(M, D, device="cuda").normal_(generator=gen(50 + k)))
        call(a)
        torch.cuda.synchronize()
        graph.replay()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            call(c)
        call(a)
        torch.cuda.synchronize()
        for name in ("loss", "lse", "total", "dx", "dw"):
            assert torch.equal(a[name], b[name]) and torch.equal(a[name], c[name]), (k, name)


def test_logits_and_weights_past_32_bit_offsets(tg):
    """2^31 logits, and a weight of 2.2 GiB whose gradient is as large."""
    M, V, D = 24, 150000, 7872
    w = torch.empty(V, D, device="cuda", dtype=BF).normal_(0.0, 0.02, generator=gen(2))
    x = torch.empty(M, D, device="cuda", dtype=BF).normal_(generator=gen(1))
    target = torch.randint(0, V, (M,), device="cuda", generator=gen(3))
    target[:4] = torch.tensor([V - 1, 0, V - 2, 136500])
    loss, lse, total = forward(tg, x, w, target)
    rows = torch.cat([target, torch.arange(0, V, 997, device="cuda")])
    t = torch.cat([x.float() @ w[i:i + 30000].float().t() for i in range(0, V, 30000)], 1).double()
    lse64 = torch.logsumexp(t, 1)
    # (t itself fp32 here: 2 D u S of each side, S about 1.3 x 0.02 x 0.64 D = 100 at most)
    assert float((lse - lse64).abs().max()) < 4 * D * 2.0 ** -24 * 200
    dw = torch.empty(V, D, device="cuda", dtype=BF)
    dx = torch.empty(M, D, device="cuda", dtype=BF)
    ws = space(tg.tg_linear_xent_backward_workspace_bytes(BF, M, V, D))
    tg.tg_linear_xent_backward(x, w, target, lse, dx=dx, dw=dw, total=total, workspace=ws)
    d = torch.exp(t - lse64[:, None])
    d[torch.arange(M, device="cuda"), target] -= 1
    d /= M
    want = d[:, rows].t().contiguous() @ x.double()
    off = (dw[rows].double() - want).norm() / want.norm()
    assert float(off) < 2 * 2.0 ** -8
    wx = sum(d[:, i:i + 30000] @ w[i:i + 30000].double() for i in range(0, V, 30000))
    assert float((dx.double() - wx).norm() / wx.norm()) < 2 * 2.0 ** -8
    # more than 2^31 logits
    M, V, D = 33000, 66000, 8
    x, w = rand(M, D, BF, 1, 1.0), rand(V, D, BF, 2, 0.7)
    target = torch.randint(0, V, (M,), device="cuda", generator=gen(3))
    loss, lse, total = forward(tg, x, w, target)
    for at in (0, 16000, M - 300):
        want, lse64, dl, de = xent(x[at:at + 300], w, target[at:at + 300], 1.0, IGNORE, 0.0)
        within(lse[at:at + 300], lse64, de, "lse")
        within(loss[at:at + 300], want, dl, "loss")
