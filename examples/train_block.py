"""A small language model trained on one GPU with every operator of the library: feed-forward blocks
(forward, gate and up kept in 8 bits, backward), their inputs as 8-bit checkpoints, the linear cross
entropy under a tied embedding, micro-step accumulation with the clip statistics, and AdamW on the
flat shard, whose bf16 round-out is the next step's weights.

    python examples/train_block.py [steps]

The model is x <- x + block(rmsnorm(x)), the data a fixed successor for each of 64 tokens, so the
loss has to fall from ln(vocab) towards 0. Normalisation and the embedding lookup are plain torch.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import zero_sharded_optimizer_flat_gb300 as Z  # noqa: E402
from zero_sharded_optimizer_flat_gb300 import build_lib  # noqa: E402

DIM, HIDDEN, LAYERS, VOCAB, TOKENS, MICRO_STEPS = 256, 768, 2, 4096, 500, 2


def rmsnorm(x):
    return (x.float() * torch.rsqrt(x.float().square().mean(1, keepdim=True) + 1e-6)).bfloat16()


def rmsnorm_backward(dy, x):
    x, dy = x.float(), dy.float()
    r = torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-6)
    return dy * r - x * (dy * x).mean(1, keepdim=True) * r ** 3


class Trainer:
    def __init__(self, seed: int = 0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.shapes = [(VOCAB, DIM)] + [s for _ in range(LAYERS) for s in ((DIM, 2 * HIDDEN), (HIDDEN, DIM))]
        numel = [a * b for a, b in self.shapes]
        self.layout = Z.ShardLayout(numel, [True] * len(numel), bucket=1 << 25, world=1, rank=0)
        self.table, n = self.layout.device_table(), self.layout.shard_len
        self.master = torch.zeros(n, device="cuda")
        self.master[:sum(numel)] = torch.randn(sum(numel), generator=g, device="cuda") * 0.02
        self.m, self.v, self.grad = (torch.zeros(n, device="cuda") for _ in range(3))
        self.weights, self.micro = (torch.zeros(n, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.weights.copy_(self.master)
        self.w, self.dw, at = [], [], 0
        for (a, b), k in zip(self.shapes, numel):  # matrices of the flat arrays, no copies
            self.w.append(self.weights[at:at + k].view(a, b))
            self.dw.append(self.micro[at:at + k].view(a, b))
            at += k
        self.clip, self.state, self.ws = Z.new_clip_stats(), Z.new_adam_state(), Z.new_norm_workspace(n)
        new = lambda *s, dtype=torch.bfloat16: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
        self.kept = [Z.new_act8(TOKENS, 2 * HIDDEN, parts=2) for _ in range(LAYERS)]
        self.inputs = [Z.new_act8(TOKENS, DIM) for _ in range(LAYERS)]
        self.y, self.dx = new(TOKENS, DIM), new(TOKENS, DIM)
        self.loss, self.lse = (new(TOKENS, dtype=torch.float32) for _ in range(2))
        self.ws_ffn = Z.new_ffn_workspace(self.inputs[0], self.w[1], self.w[2])
        self.ws_ce = Z.new_linear_ce_workspace(self.y, self.w[0])

    def micro_step(self, tokens, targets):
        """The micro-step's loss; its bf16 gradient is in self.micro."""
        x, stack = self.w[0][tokens], []
        for l in range(LAYERS):
            n = rmsnorm(x)
            Z.act_pack(n, self.inputs[l])
            Z.ffn_forward(n, self.w[1 + 2 * l], self.w[2 + 2 * l], self.y, self.ws_ffn, kept=self.kept[l])
            stack.append(x)
            x = x + self.y
        last = rmsnorm(x)
        Z.linear_ce_forward(last, self.w[0], targets, self.loss, self.lse, self.ws_ce)
        live = targets != -100
        dloss = live.float() / (live.sum() * MICRO_STEPS)
        Z.linear_ce_backward(last, self.w[0], targets, self.lse, dloss, self.dx, self.dw[0], self.ws_ce)
        dx = rmsnorm_backward(self.dx, x)
        for l in reversed(range(LAYERS)):
            Z.ffn_backward(dx.bfloat16(), self.inputs[l], self.kept[l], self.w[1 + 2 * l], self.w[2 + 2 * l], self.dx,
                           self.dw[1 + 2 * l], self.dw[2 + 2 * l], self.ws_ffn)
            dx = dx + rmsnorm_backward(self.dx, stack[l])
        embed = torch.zeros(VOCAB, DIM, device="cuda").index_add_(0, tokens, dx)
        self.dw[0].copy_(self.dw[0].float() + embed)
        return self.loss.sum() / live.sum()

    def step(self, batches, lr: float = 2e-3):
        total = 0.0
        for k, (tokens, targets) in enumerate(batches):
            total += self.micro_step(tokens, targets)
            Z.grad_accumulate(self.grad, self.micro, first=k == 0, last=k == len(batches) - 1, max_norm=1.0, ws=self.ws,
                              stats=self.clip)
        Z.adamw_step(self.layout, self.table, self.master, self.m, self.v, self.grad, self.weights, lr=lr,
                     clip_stats=self.clip, adam_state=self.state)
        return total / len(batches)


def batch(g):
    tokens = torch.randint(0, 64, (TOKENS,), generator=g, device="cuda") * 61
    targets = (tokens * 5 + 61 * 7) % (64 * 61)
    targets[torch.rand(TOKENS, generator=g, device="cuda") < 0.1] = -100  # prompt tokens: no loss
    return tokens, targets


def main(steps: int = 40):
    build_lib.build()
    t, g = Trainer(), torch.Generator(device="cuda").manual_seed(1)
    losses = []
    for i in range(steps):
        losses.append(float(t.step([batch(g) for _ in range(MICRO_STEPS)])))
        if i % 5 == 0 or i == steps - 1:
            s = Z.read_clip_stats(t.clip)
            print(f"step {i:3d}  loss {losses[-1]:.4f}  gradient norm {float(s['norm']):.3f}  found_inf {s['found_inf']}")
    return losses


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 40)
