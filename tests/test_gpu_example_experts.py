"""The example with experts runs, and its gradients are those of the model that it states: the same model in
fp64 under automatic differentiation, with the experts that its routing chose.

Tolerance, fixed before the first run: some sixteen roundings to bf16 lie between a parameter's gradient and its
inputs (norms, h, parts, dx and dgate_up of two blocks, the loss's gradient, the result), each at most 2^-8 of what it
rounds: 6.2e-2 of the norm if all of them added up."""
import importlib.util
import math
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


def load():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_experts.py")
    spec = importlib.util.spec_from_file_location("train_experts", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_train_experts_runs(zopt):
    m = load()
    losses = m.main(4)
    assert len(losses) == 4 and all(math.isfinite(x) for x in losses)


def test_train_experts_gradients(zopt):
    m = load()
    t = m.Trainer(3)
    tokens, targets = m.batch(torch.Generator(device="cuda").manual_seed(4))
    loss = t.micro_step(tokens, targets)
    torch.cuda.synchronize()
    w = [a.double().requires_grad_() for a in t.w]
    layers = [[a.double().requires_grad_() for a in layer.w] for layer in t.layers]
    norm = lambda x: x * torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-6)  # noqa: E731
    x = w[0][tokens]
    for layer, router, (wgu, wd) in zip(t.layers, w[1:], layers):
        n = norm(x)
        score = torch.sigmoid(n @ router)
        index = layer.index.long()
        weight = score.gather(1, index.clamp(min=0)) * (index >= 0)
        weight = weight / weight.sum(1, keepdim=True).clamp(min=1e-30)
        y = torch.zeros_like(x)
        for e in range(m.EXPERTS):
            z = n @ wgu[e]
            part = (torch.nn.functional.silu(z[:, :m.HIDDEN]) * z[:, m.HIDDEN:]) @ wd[e]
            y = y + part * (weight * (index == e)).sum(1, keepdim=True)
        x = x + y
    ref = torch.nn.functional.cross_entropy(norm(x) @ w[0].t(), targets)
    assert abs(float(loss) - float(ref)) <= 1e-2 * float(ref)
    ref.backward()
    for got, want in [(a, b.grad) for a, b in zip(t.dw, w)] + [(a, b.grad) for layer, r in zip(t.layers, layers) for a, b in zip(layer.dw, r)]:
        assert float((got.double() - want).norm()) <= 6.2e-2 * float(want.norm())
    for layer in t.layers:
        assert bool((layer.index[m.TOKENS - m.PADDING:] == -1).all()) and int(layer.counts.sum()) == (m.TOKENS - m.PADDING) * m.TOP_K
