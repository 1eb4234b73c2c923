"""A small language model's training steps, and its head served in 8-bit integers.

    python examples/lm_step.py [--tokens 2048 --width 1024 --hidden 2816 --vocab 32000 --steps 10 --states 8]

The model is an embedding, one gated block y = x + down(act(gate(x)) * up(x))
and a vocabulary head, trained on random next tokens: the loss and its gradient
over the vocabulary, the block's gradients, the gradients' norm and the AdamW
update are the library's operators; torch holds the memory, makes the data and
gathers and scatters the embedding's rows.  Afterwards the head's weight is
quantized with a scale per channel, and logits of a few tokens are taken with
tokens quantized on the way.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import tile_level_gemm_02_amd as tg  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32
PAD = -100


class Model:
    def __init__(self, tokens: int, width: int, hidden: int, vocab: int, states: int = 32, seed: int = 1):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def weight(rows, cols, std):
            return torch.empty(rows, cols, device="cuda").normal_(0.0, std, generator=gen)

        # fp32 masters, their bf16 copies for the products, gradients in bf16
        self.masters = [weight(vocab, width, 1.0), weight(2 * hidden, width, width ** -0.5), weight(width, hidden, hidden ** -0.5),
                        weight(vocab, width, width ** -0.5)]
        self.params = [m.to(BF) for m in self.masters]
        self.embed, self.w_gate_up, self.w_down, self.w_head = self.params
        self.grads = [torch.empty_like(p) for p in self.params]
        if states == 8:
            self.exp_avg = [torch.zeros(p.shape, device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn) for p in self.params]
            self.exp_avg_sq = [m.clone() for m in self.exp_avg]
            self.scales = [[torch.zeros(-(-p.numel() // 256), device="cuda") for p in self.params] for _ in range(2)]
        else:
            self.exp_avg, self.exp_avg_sq = ([torch.zeros_like(m) for m in self.masters] for _ in range(2))
            self.scales = [None, None]
        self.ws = tg.tg_ops_workspace()
        need = max(tg.tg_linear_xent_workspace_bytes(BF, tokens, vocab, width), tg.tg_linear_xent_backward_workspace_bytes(BF, tokens, vocab, width))
        self.loss_ws = torch.zeros(-(-need // 4), dtype=torch.int32, device="cuda")

        def room(cols):
            return torch.empty(tokens, cols, device="cuda", dtype=BF)

        self.h, self.gate_up, self.y, self.dy, self.dx = room(hidden), room(2 * hidden), room(width), room(width), room(width)
        self.loss, self.lse = (torch.empty(tokens, device="cuda") for _ in range(2))
        self.total, self.norm = torch.empty(2, device="cuda"), torch.empty(1, device="cuda")
        self.steps = 0

    def forward(self, tokens):
        """The block's output for each token."""
        n = tokens.shape[0]
        x, h, gu, y = self.embed[tokens], self.h[:n], self.gate_up[:n], self.y[:n]
        tg.tg_glu(x, self.w_gate_up, h, act="silu", gate_up=gu, workspace=self.ws)
        tg.tg_linear(h, self.w_down, y, residual=x, workspace=self.ws)
        return x, y

    def backward(self, tokens, targets, z_loss: float = 1e-4):
        """Gradients of the mean loss; the loss stays on the GPU (self.total)."""
        x, y = self.forward(tokens)
        g_embed, g_gate_up, g_down, g_head = self.grads
        tg.tg_linear_xent(y, self.w_head, targets, self.loss, self.lse, self.total, ignore_index=PAD, z_loss=z_loss, workspace=self.loss_ws)
        tg.tg_linear_xent_backward(y, self.w_head, targets, self.lse, dx=self.dy, dw=g_head, total=self.total, ignore_index=PAD, z_loss=z_loss,
                                   workspace=self.loss_ws)
        tg.tg_glu_backward(self.dy, self.w_down, x, self.w_gate_up, self.gate_up, self.h, self.gate_up, dx=self.dx, dw_gate_up=g_gate_up,
                           dw_down=g_down, act="silu", workspace=self.ws)
        g_embed.zero_().index_add_(0, tokens, self.dx + self.dy)  # (the residual passes dy on)

    def update(self, lr: float, max_norm: float = 1.0):
        self.steps += 1
        tg.tg_clip_grads(self.grads, float("inf"), norm=self.norm, workspace=self.ws)  # the norm alone
        tg.tg_adamw(self.params, self.grads, self.exp_avg, self.exp_avg_sq, self.steps, lr, betas=(0.9, 0.95), weight_decay=0.1,
                    masters=self.masters, exp_avg_scales=self.scales[0], exp_avg_sq_scales=self.scales[1], norm=self.norm, max_norm=max_norm)

    def serve(self):
        """A function from tokens to logits whose head is held in 8 bits."""
        q, scale = torch.empty(self.w_head.shape, device="cuda", dtype=torch.int8), torch.empty(self.w_head.shape[0], device="cuda")
        tg.tg_quantize_i8(self.w_head, q, scale)

        def logits(tokens):
            y = self.forward(tokens)[1]
            yq, ys = torch.empty(y.shape, device="cuda", dtype=torch.int8), torch.empty(y.shape[0], device="cuda")
            out = torch.empty(y.shape[0], -(-q.shape[0] // 16) * 16, device="cuda")[:, :q.shape[0]]
            tg.tg_quantize_i8(y, yq, ys)
            tg.tg_linear_i8(yq, q, out, ys, scale, workspace=self.ws)
            return out

        return logits


def train(tokens=2048, width=1024, hidden=2816, vocab=32000, steps=10, states=32, lr=1e-3, say=print):
    """Mean loss of each step, and how far the 8-bit head's logits of four tokens are from the bf16 head's, relative to their norm."""
    model = Model(tokens, width, hidden, vocab, states)
    gen = torch.Generator(device="cuda").manual_seed(2)
    ids = torch.randint(0, vocab, (tokens,), device="cuda", generator=gen)
    targets = torch.randint(0, vocab, (tokens,), device="cuda", generator=gen)
    targets[-tokens // 16:] = PAD
    losses = []
    for step in range(steps):
        model.backward(ids, targets)
        model.update(lr)
        losses.append(float(model.total[0] / model.total[1]))
        say(f"step {step}: loss {losses[-1]:.4f}, gradient norm {float(model.norm):.4f}")
    few = ids[:4]
    y = model.forward(few)[1].clone()
    full = torch.empty(4, -(-vocab // 16) * 16, device="cuda")[:, :vocab]
    tg.tg_linear(y, model.w_head, full, workspace=model.ws)
    eight = model.serve()(few)
    return losses, float((eight - full).norm() / full.norm())


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 2048), ("width", 1024), ("hidden", 2816), ("vocab", 32000), ("steps", 10), ("states", 32)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    losses, off = train(a.tokens, a.width, a.hidden, a.vocab, a.steps, a.states)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f}; the 8-bit head's logits are {off:.3g} off")


if __name__ == "__main__":
    main()
