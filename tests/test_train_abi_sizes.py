"""Sizes and numbers at the ends of what the training operators and the int8
layers take: queries and refusals (CPU only: nothing here launches)."""
import pytest
import torch

A = 0x10000  # a fake aligned device address: never dereferenced on these paths
W = 1 << 20  # a fake workspace


@pytest.fixture(scope="module")
def tg():
    import tile_level_gemm_02_amd as tg

    return tg


@pytest.fixture(scope="module")
def train(tg):
    from tile_level_gemm_02_amd import train

    return train._lib()


@pytest.mark.parametrize("V,D", [(8, 8), (0, 8), (8, 0), (32000, 2048), (1000, 1 << 25)])
def test_loss_of_no_rows_takes_its_querys_bytes(tg, train, V, D):
    """The query of an empty batch covers the total's two zeros: a byte less, or no workspace, is refused."""

    def call(total, ws, nb):
        return train.tg_linear_xent(1, 0, V, D, None, D, None, D, 1.0, None, -100, 0.0, None, None, total, ws, nb, None)

    need = tg.tg_linear_xent_workspace_bytes(torch.bfloat16, 0, V, D)
    assert need > 65536 and need % 256 == 0
    assert call(A, W, need - 1) == tg.TG_ERR_INVALID_VALUE
    assert call(A, None, 0) == tg.TG_ERR_INVALID_VALUE
    # without a total there is nothing to write, whatever the workspace
    assert call(None, None, 0) == call(None, W, 256) == tg.TG_OK


@pytest.mark.parametrize("scale", [2.4e38, -2.4e38, 3.4e38, float("nan")])
def test_a_scale_whose_exponentials_have_no_fp32_factor(tg, train, scale):
    """Exponentials are base 2: a scale whose product with log2(e) is past fp32 would make 0 x infinity of a logit of 0."""
    big = 1 << 40
    assert train.tg_linear_xent(1, 8, 8, 8, A, 8, A, 8, scale, A, -100, 0.0, A, A, A, W, big, None) == tg.TG_ERR_INVALID_VALUE
    assert train.tg_linear_xent_backward(1, 8, 8, 8, A, 8, A, 8, scale, A, -100, 0.0, A, A, 1.0, A, A, 8, A, 8, 2, W, big,
                                         None) == tg.TG_ERR_INVALID_VALUE


def test_rows_too_long_for_32_bit_offsets(tg, train):
    """The limits that the header states, on their far side; the queries know no leading dimension but the width."""
    big, bf = 1 << 50, torch.bfloat16

    def loss(D, ldx, ldw):
        return train.tg_linear_xent(1, 8, 8, D, A, ldx, A, ldw, 1.0, A, -100, 0.0, A, A, A, W, big, None)

    def grad(D, ldx, ldw):
        return train.tg_linear_xent_backward(1, 8, 8, D, A, ldx, A, ldw, 1.0, A, -100, 0.0, A, A, 1.0, A, A, D, A, D, 2, W, big, None)

    ld = (2 ** 31 - 16 - 16) // 512 // 8 * 8 + 8  # 512 ld + 16 just past the limit
    assert 512 * ld + 16 >= 2 ** 31 - 16
    for f in (loss, grad):
        assert f(8, ld, 8) == f(8, 8, ld) == tg.TG_ERR_NOT_SUPPORTED
    assert grad(8, 8, 1398104) == tg.TG_ERR_NOT_SUPPORTED
    assert tg.tg_linear_xent_workspace_bytes(bf, 8, 8, 1 << 22) == tg.tg_linear_xent_backward_workspace_bytes(bf, 8, 8, 1 << 22) == 0
    assert tg.tg_linear_xent_backward_workspace_bytes(bf, 8, 8, 1398104) == 0 < tg.tg_linear_xent_backward_workspace_bytes(bf, 8, 8, 1398096)


def test_int8_rows_too_long_for_32_bit_offsets(tg):
    from tile_level_gemm_02_amd import int8

    def layer(ldx, ldw):
        return int8._lib().tg_linear_i8(33, 40, 16, A, ldx, A, ldw, A, A, None, 0, None, 0, A, 40, 2, None, 0, None)

    ld = (2 ** 31 - 16 - 16) // 256 // 16 * 16 + 16
    assert layer(ld, 16) == layer(16, ld) == tg.TG_ERR_NOT_SUPPORTED


def test_scales_whose_product_is_past_fp32(tg, train):
    """It is the gradients' common factor: infinite, it would make the zeros of ignored rows NaN."""
    for scale, gs in ((10.0, 1e38), (-1e20, 1e19), (2.0, -3e38)):
        assert train.tg_linear_xent_backward(1, 8, 8, 8, A, 8, A, 8, scale, A, -100, 0.0, A, A, gs, A, A, 8, A, 8, 2, W, 1 << 40,
                                             None) == tg.TG_ERR_INVALID_VALUE
