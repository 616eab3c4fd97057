"""A small language model of experts trained on one GPU: each block routes its tokens (zopt_route_*) and runs
the experts' feed-forward block (zopt_experts_*), the loss is the linear cross entropy under a tied
embedding, AdamW steps embedding and routers on the flat shard, Muon the experts' matrices, a batch of
equal ones for each of the two shapes.

    python examples/train_experts.py [steps]

The model is x <- x + experts(rmsnorm(x)) with logistic scores and a bias for balance, which moves towards the
experts that get fewer slots; the data a fixed successor for each of 64 tokens and some padding.
Normalisation, the routers' own product and the embedding lookup are plain torch.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import zero_sharded_optimizer_flat_gb300 as Z  # noqa: E402
from zero_sharded_optimizer_flat_gb300 import build_lib  # noqa: E402

DIM, HIDDEN, EXPERTS, TOP_K, LAYERS, VOCAB, TOKENS, PADDING = 256, 256, 8, 2, 2, 4096, 500, 20
HOW = dict(score="sigmoid", renormalise=True, scale=1.0)


def rmsnorm(x):
    return (x.float() * torch.rsqrt(x.float().square().mean(1, keepdim=True) + 1e-6)).bfloat16()


def rmsnorm_backward(dy, x):
    x, dy = x.float(), dy.float()
    r = torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-6)
    return dy * r - x * (dy * x).mean(1, keepdim=True) * r ** 3


class Layer:
    """A block's buffers: the routing of its tokens, what the backward keeps, the experts' gradients."""

    def __init__(self, g):
        new = lambda *s, dtype=torch.bfloat16: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
        draw = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        self.index, self.weight = new(TOKENS, TOP_K, dtype=torch.int32), new(TOKENS, TOP_K, dtype=torch.float32)
        self.counts, self.bias = new(EXPERTS, dtype=torch.int32), torch.zeros(EXPERTS, device="cuda")
        self.dweight, self.dlogits = torch.empty_like(self.weight), new(TOKENS, EXPERTS, dtype=torch.float32)
        self.kept = new(TOKENS * TOP_K, 2 * HIDDEN)
        self.master = [draw(EXPERTS, DIM, 2 * HIDDEN) * DIM ** -0.5, draw(EXPERTS, HIDDEN, DIM) * 0.3 * HIDDEN ** -0.5]
        self.momentum = [torch.zeros_like(m) for m in self.master]
        self.w, self.dw = [m.bfloat16() for m in self.master], [new(*m.shape) for m in self.master]
        self.stats = [Z.new_muon_stats(EXPERTS) for _ in self.master]


class Trainer:
    def __init__(self, seed: int = 0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.layers = [Layer(g) for _ in range(LAYERS)]
        self.shapes = [(VOCAB, DIM)] + [(DIM, EXPERTS)] * LAYERS
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
        self.live = torch.arange(TOKENS, device="cuda") < TOKENS - PADDING
        new = lambda *s, dtype=torch.bfloat16: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
        self.y, self.dx = new(TOKENS, DIM), new(TOKENS, DIM)
        self.loss, self.lse = (new(TOKENS, dtype=torch.float32) for _ in range(2))
        layer = self.layers[0]
        self.ws_experts = Z.new_experts_workspace(self.y, layer.index, *layer.w)
        self.ws_ce = Z.new_linear_ce_workspace(self.y, self.w[0])
        self.ws_muon = Z.new_muon_workspace_many([(DIM, 2 * HIDDEN, EXPERTS), (HIDDEN, DIM, EXPERTS)] * LAYERS)

    def micro_step(self, tokens, targets):
        """The micro-step's loss; its bf16 gradients are in self.micro and the layers' dw."""
        x, stack = self.w[0][tokens], []
        for layer, router in zip(self.layers, self.w[1:]):
            n = rmsnorm(x)
            logits = n.float() @ router.float()
            Z.route_forward(logits, layer.index, layer.weight, layer.counts, bias=layer.bias, live=self.live, **HOW)
            Z.experts_forward(n, layer.index, layer.weight, *layer.w, self.y, self.ws_experts, kept=layer.kept)
            stack.append((x, n, logits))
            x = x + self.y
        last = rmsnorm(x)
        Z.linear_ce_forward(last, self.w[0], targets, self.loss, self.lse, self.ws_ce)
        counted = targets != -100
        dloss = counted.float() / counted.sum()
        Z.linear_ce_backward(last, self.w[0], targets, self.lse, dloss, self.dx, self.dw[0], self.ws_ce)
        dx = rmsnorm_backward(self.dx, x)
        for layer, router, drouter, (x, n, logits) in reversed(list(zip(self.layers, self.w[1:], self.dw[1:], stack))):
            Z.experts_backward(dx.bfloat16(), n, layer.index, layer.weight, layer.kept, *layer.w, self.dx, layer.dweight, *layer.dw,
                               self.ws_experts)
            Z.route_backward(logits, layer.index, layer.weight, layer.dweight, layer.dlogits, **HOW)
            drouter.copy_(n.float().t() @ layer.dlogits)
            dx = dx + rmsnorm_backward(self.dx.float() + layer.dlogits @ router.float().t(), x)
        embed = torch.zeros(VOCAB, DIM, device="cuda").index_add_(0, tokens, dx)
        self.dw[0].copy_(self.dw[0].float() + embed)
        return self.loss.sum() / counted.sum()

    def step(self, tokens, targets, lr: float = 2e-3, muon_lr: float = 1e-3):
        loss = self.micro_step(tokens, targets)
        Z.grad_accumulate(self.grad, self.micro, first=True, last=True, max_norm=1.0, ws=self.ws, stats=self.clip)
        Z.adamw_step(self.layout, self.table, self.master, self.m, self.v, self.grad, self.weights, lr=lr, clip_stats=self.clip,
                     adam_state=self.state)
        Z.muon_step_many([(layer.master[k], layer.momentum[k], layer.dw[k], layer.w[k], layer.stats[k])
                          for layer in self.layers for k in range(2)], self.ws_muon, lr=muon_lr)
        for layer in self.layers:  # the experts that got fewer slots become a little easier to choose
            layer.bias += 1e-3 * torch.sign(layer.counts.float().mean() - layer.counts)
        return loss


def batch(g):
    tokens = torch.randint(0, 64, (TOKENS,), generator=g, device="cuda") * 61
    targets = (tokens * 5 + 61 * 7) % (64 * 61)
    targets[TOKENS - PADDING:] = -100
    return tokens, targets


def main(steps: int = 40):
    build_lib.build()
    t, g = Trainer(), torch.Generator(device="cuda").manual_seed(1)
    losses = []
    for i in range(steps):
        losses.append(float(t.step(*batch(g))))
        if i % 5 == 0 or i == steps - 1:
            most = max(int(layer.counts.max()) for layer in t.layers)
            print(f"step {i:3d}  loss {losses[-1]:.4f}  most slots of an expert {most} of {(TOKENS - PADDING) * TOP_K}")
    return losses


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 40)
