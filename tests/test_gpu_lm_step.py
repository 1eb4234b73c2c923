"""The training operators together (examples/lm_step.py): the loss and all
gradients of a small model against torch's autograd in 64 bits on the same
weights, an update against the formula, and the head served in 8 bits."""
import os
import sys

import pytest
import torch

from _train_ref import U, adamw

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import lm_step

    return lm_step


def setup(lm, states):
    tokens, width, hidden, vocab = 300, 136, 200, 1003
    m = lm.Model(tokens, width, hidden, vocab, states)
    g = torch.Generator(device="cuda").manual_seed(5)
    ids, targets = (torch.randint(0, vocab, (tokens,), device="cuda", generator=g) for _ in range(2))
    targets[-20:] = lm.PAD
    return m, ids, targets, hidden


def test_loss_and_gradients_of_the_whole_model(lm):
    """The stored 16-bit values h, y, dt, dy, [dg | du], dx and the gradient itself are each off by up to 2^-8 of
    themselves; a gradient sums products of such values with independent roundings, so relative to the gradient's norm
    the errors of the seven stages add to at most 7 x 2^-8 = 0.027 (were they all aligned).  The embedding's gradient
    adds one more rounding (dx + dy, and its sums in bf16): 9."""
    m, ids, targets, hidden = setup(lm, 32)
    m.backward(ids, targets, z_loss=1e-3)
    w = [t.double().requires_grad_() for t in m.params]
    x = w[0][ids]
    gu = x @ w[1].t()
    y = x + (torch.nn.functional.silu(gu[:, :hidden]) * gu[:, hidden:]) @ w[2].t()
    t = y @ w[3].t()
    lse, counts = torch.logsumexp(t, 1), targets != lm.PAD
    loss = torch.where(counts, lse - t.gather(1, targets.clamp(min=0)[:, None])[:, 0] + 1e-3 * lse * lse, 0.0)
    (loss.sum() / counts.sum()).backward()
    # y is off by 2 x 2^-8 of itself, so a logit by that of its norm: |y| |w| / sqrt(width) a token, averaged over the tokens
    assert abs(float(m.total[0]) - float(loss.detach().sum())) < 2 * 2.0 ** -8 * float(counts.sum()) and int(m.total[1]) == int(counts.sum())
    for i, (got, want) in enumerate(zip(m.grads, w)):
        off = float((got.double() - want.grad).norm() / want.grad.norm())
        assert off < (9 if i == 0 else 7) * 2.0 ** -8, (i, off)


@pytest.mark.parametrize("states", [32, 8])
def test_an_update_after_the_gradients(lm, states):
    """Two steps: the first's states are zero before, so its update is known whatever the states' type."""
    m, ids, targets, _ = setup(lm, states)
    m.backward(ids, targets)
    before = [t.clone() for t in m.masters]
    grads = [g.clone() for g in m.grads]
    m.update(1e-2, max_norm=0.5)
    norm = float(sum(g.double().square().sum() for g in grads)) ** 0.5
    assert abs(float(m.norm) / norm - 1) < 2.0 ** -23 and all(torch.equal(a, b) for a, b in zip(grads, m.grads))
    for w0, g, w, p in zip(before, grads, m.masters, m.params):
        zero = torch.zeros_like(w0)
        want, _, _, up = adamw(w0, g, zero, zero, 1, 1e-2, 0.9, 0.95, 1e-8, 0.1, norm, 0.5)
        # as tests/test_gpu_adamw.py: 12 u of the update and 6 + 9 / 2 of its m and v, 4 u of the weight
        assert bool(((w.double() - want).abs() <= 24 * U * up.abs() + 5 * U * want.abs()).all())
        assert torch.equal(p, w.to(p.dtype))
    m.backward(ids, targets)
    m.update(1e-2)
    assert all(bool(t.isfinite().all()) for t in m.masters)


@pytest.mark.parametrize("states", [32, 8])
def test_the_example_runs_and_serves(lm, states):
    losses, off = lm.train(tokens=512, width=256, hidden=704, vocab=5003, steps=4, states=states, say=lambda *a: None)
    assert all(v == v and v < 1e3 for v in losses)
    # tokens and channels are off by up to half a step of amax / 127 a value, uniformly: amax is at most about 5 standard
    # deviations here, so each operand's relative error is at most 5 / 127 / sqrt(12) = 0.0114, and the logits' sqrt(2) of it
    # (2 times that for rows with larger extremes)
    assert off < 2 * 2 ** 0.5 * 0.0114
