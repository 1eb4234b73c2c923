"""The example block (examples/ffn_block.py): its gradients against torch's
autograd in 64 bits on the same weights, and its loss falls."""
import os
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ffn():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import ffn_block

    return ffn_block


def test_gradients_of_the_whole_block(ffn):
    """Each stored 16-bit value (h, y, z, dz, dy, dg, du) is off by up to 2^-8
    of itself; a gradient sums products of such values with independent
    roundings, so relative to the gradient's norm the errors of the seven stages
    add to at most 7 x 2^-8 = 0.027 (were they all aligned)."""
    tokens, width, hidden, out = 300, 136, 200, 72
    b = ffn.Block(tokens, width, hidden, out)
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.empty(tokens, width, device="cuda").normal_(generator=g).to(torch.bfloat16)
    dz = torch.empty(tokens, out, device="cuda").normal_(generator=g).to(torch.bfloat16)
    b.forward(x)
    b.dz.copy_(dz)
    b.backward(x, b.dz, float("inf"))
    w = [t.double().requires_grad_() for t in (b.w_gate_up, b.w_down, b.w_head, b.bias)]
    x64 = x.double()
    gu = x64 @ w[0].t()
    h = torch.nn.functional.silu(gu[:, :hidden]) * gu[:, hidden:]
    y = x64 + h @ w[1].t()
    z = torch.nn.functional.gelu(y @ w[2].t() + w[3])
    (z * dz.double()).sum().backward()
    for got, want in zip(b.grads, w):
        off = (got.double() - want.grad).norm() / want.grad.norm()
        assert float(off) < 7 * 2.0 ** -8, float(off)


def test_the_loss_falls_and_a_token_alone_agrees(ffn):
    losses, off = ffn.train(tokens=512, width=256, hidden=704, out=128, steps=12, say=lambda *a: None)
    assert losses[-1] < losses[0] and all(b < a * 1.02 for a, b in zip(losses, losses[1:]))
    # one token takes other kernels: another order of the fp32 sums can move the
    # stored h, y and z by a step of their type (2^-7 of values up to about 4)
    assert off <= 3 * 2.0 ** -7 * 4
