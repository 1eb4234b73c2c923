"""One gated feed-forward block trained for a few steps, and run for one token.

    python examples/ffn_block.py [--tokens 2048 --width 1024 --hidden 2816 --steps 20]

The block is y = x + down(act(gate(x)) * up(x)) with a small head on it,
z = gelu(y . Wh^T + b), fitted to random targets by plain gradient descent.
Every matrix product, activation, residual, gradient and the clipping is one
of the library's feed-forward operators; torch holds the memory, makes the
data and applies the updates.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import tile_level_gemm_02_amd as tg  # noqa: E402


class Block:
    def __init__(self, tokens: int, width: int, hidden: int, out: int, dtype=torch.bfloat16):
        gen = torch.Generator(device="cuda").manual_seed(1)

        def weight(rows, cols):
            return torch.empty(rows, cols, device="cuda").normal_(0.0, cols ** -0.5, generator=gen)

        # fp32 weights for the updates and their 16-bit copies for the products
        self.master = [weight(2 * hidden, width), weight(width, hidden), weight(out, width), torch.zeros(out, device="cuda")]
        self.w_gate_up, self.w_down, self.w_head = (m.to(dtype) for m in self.master[:3])
        self.bias = self.master[3]
        self.grads = [torch.empty_like(m) for m in self.master]
        self.norm = torch.empty(1, device="cuda")
        self.ws = tg.tg_ops_workspace()

        def room(cols):
            return torch.empty(tokens, cols, device="cuda", dtype=dtype)

        self.h, self.gate_up, self.y, self.z, self.pre = room(hidden), room(2 * hidden), room(width), room(out), room(out)
        self.dz, self.dy = room(out), room(width)

    def forward(self, x):
        n = x.shape[0]
        h, gu, y, z, pre = self.h[:n], self.gate_up[:n], self.y[:n], self.z[:n], self.pre[:n]
        tg.tg_glu(x, self.w_gate_up, h, act="silu", gate_up=gu, workspace=self.ws)
        tg.tg_linear(h, self.w_down, y, residual=x, workspace=self.ws)
        tg.tg_linear(y, self.w_head, z, bias=self.bias, act="gelu", preact=pre, workspace=self.ws)
        return z

    def backward(self, x, dz, max_norm: float):
        """Gradients of all weights from dz (overwritten), clipped to max_norm in place."""
        g_gate_up, g_down, g_head, g_bias = self.grads
        tg.tg_linear_backward(dz, self.y, self.w_head, dx=self.dy, dw=g_head, dbias=g_bias, preact=self.pre, act="gelu", dz=dz,
                              workspace=self.ws)
        # the residual's gradient is dy itself; [dg | du] may replace [g | u]
        tg.tg_glu_backward(self.dy, self.w_down, x, self.w_gate_up, self.gate_up, self.h, self.gate_up, dw_gate_up=g_gate_up,
                           dw_down=g_down, act="silu", workspace=self.ws)
        tg.tg_clip_grads(self.grads, max_norm, norm=self.norm, workspace=self.ws)

    def update(self, rate: float):
        for m, g in zip(self.master, self.grads):
            m.sub_(g, alpha=rate)
        for w, m in zip((self.w_gate_up, self.w_down, self.w_head), self.master):
            w.copy_(m)


def train(tokens=2048, width=1024, hidden=2816, out=512, steps=20, rate=0.5, max_norm=1.0, say=print):
    """Mean squared error of each step."""
    block = Block(tokens, width, hidden, out)
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.empty(tokens, width, device="cuda").normal_(generator=gen).to(torch.bfloat16)
    target = torch.empty(tokens, out, device="cuda").normal_(0.0, 0.5, generator=gen)
    losses = []
    for step in range(steps):
        z = block.forward(x)
        error = z.float() - target
        losses.append(float(error.square().mean()))
        block.dz.copy_(error * (2.0 / tokens))
        block.backward(x, block.dz, max_norm)
        block.update(rate)
        say(f"step {step}: loss {losses[-1]:.5f}, gradient norm {float(block.norm):.4f}")
    one = block.forward(x[:1]).clone()  # a single token, the decode path
    every = block.forward(x)
    return losses, float((one.float() - every[:1].float()).abs().max())


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--width", type=int, default=1024)
    ap.add_argument("--hidden", type=int, default=2816)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args()
    losses, off = train(a.tokens, a.width, a.hidden, steps=a.steps)
    print(f"loss {losses[0]:.5f} -> {losses[-1]:.5f}; one token alone differs from the batch by at most {off:.3g}")


if __name__ == "__main__":
    main()
