"""Pins of the routing's and the experts' oracle: torch's own softmax, sigmoid and topk, autograd, and
central differences."""
import numpy as np
import pytest
import torch

from oracle import experts as OE
from oracle import lm


def case(seed, t=23, e=12):
    g = np.random.default_rng(seed)
    return g.normal(size=(t, e)), 0.1 * g.normal(size=e), g


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_route_forward_is_topk_of_torch(kind, biased):
    l, bias, _ = case(1)
    s = torch.softmax(torch.tensor(l), 1) if kind == "softmax" else torch.sigmoid(torch.tensor(l))
    rank = s + torch.tensor(bias) if biased else s
    want = rank.topk(4, dim=1).indices
    index, weight, counts = OE.route_forward(l, 4, kind, bias if biased else None, scale=2.5)
    assert np.array_equal(index, want.numpy())
    w = s.gather(1, want)
    assert np.allclose(weight, 2.5 * (w / w.sum(1, keepdim=True)).numpy(), rtol=1e-13)
    plain = OE.route_forward(l, 4, kind, bias if biased else None, renormalise=False)[1]
    assert np.allclose(plain, w.numpy(), rtol=1e-13)
    assert np.array_equal(counts, torch.bincount(want.flatten(), minlength=12).numpy())


def test_route_forward_ties_groups_and_what_is_left():
    l = np.zeros((1, 8))
    assert OE.route_forward(l, 3)[0].tolist() == [[0, 1, 2]]
    assert OE.route_forward(l, 3, groups=4, top_groups=2)[0].tolist() == [[0, 1, 2]]
    l[0] = [0, 5, 0, 0, 3, 3.5, 0, 0]  # runs of two: the scores' sums, not the largest one, decide
    assert OE.route_forward(l, 2, "sigmoid", groups=4, top_groups=1)[0].tolist() == [[5, 4]]
    l[0, 1:] = -np.inf
    index, weight, counts = OE.route_forward(l, 3)
    assert index.tolist() == [[0, -1, -1]] and weight.tolist() == [[1, 0, 0]] and counts.sum() == 1
    assert OE.route_forward(l, 2, groups=2, top_groups=1)[0].tolist() == [[0, -1]]
    assert OE.route_forward(np.full((1, 8), -np.inf), 2)[0].tolist() == [[-1, -1]]
    assert OE.route_forward(np.zeros((2, 8)), 2, live=[False, True])[0].tolist() == [[-1, -1], [0, 1]]


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [False, True])
def test_route_backward_against_differences(kind, renormalise):
    l, bias, g = case(2, t=5, e=7)
    index, _, _ = OE.route_forward(l, 3, kind, bias)
    index[2, 1] = -1
    dw = g.normal(size=(5, 3))

    def value(l):
        total = 0.0
        for r in range(5):
            on = index[r] >= 0
            w = OE.scores(l[r], kind)[index[r][on]]
            total += (dw[r][on] * 1.5 * (w / w.sum() if renormalise else w)).sum()
        return total

    got, h = OE.route_backward(l, index, dw, kind, renormalise, 1.5), 1e-6
    for r in range(5):
        for i in range(7):
            up, down = l.copy(), l.copy()
            up[r, i] += h
            down[r, i] -= h
            assert abs((value(up) - value(down)) / (2 * h) - got[r, i]) < 1e-8


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_experts_against_autograd(act):
    g = torch.Generator().manual_seed(3)
    t, k, e, d, f = 9, 3, 4, 6, 5
    new = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    x, wgu, wd, dy = new(t, d), new(e, d, 2 * f), new(e, f, d), new(t, d)
    w = torch.rand(t, k, generator=g, dtype=torch.float64)
    index = torch.randint(-1, e, (t, k), generator=g)
    for a in (x, wgu, wd, w):
        a.requires_grad_()
    a = torch.nn.functional.silu if act == "silu" else lambda z: torch.nn.functional.gelu(z, approximate="tanh")
    z = torch.einsum("td,tkdf->tkf", x, wgu[index.clamp(min=0)])
    parts = torch.einsum("tkf,tkfd->tkd", a(z[..., :f]) * z[..., f:], wd[index.clamp(min=0)])
    y = (parts * (w * (index >= 0))[..., None]).sum(1)
    y.backward(dy)
    n = [v.detach().numpy() for v in (x, index.int(), w, wgu, wd)]
    got, gu, size = OE.experts_forward(*n, act)
    assert np.allclose(got, y.detach().numpy(), rtol=1e-12, atol=1e-12) and (size >= np.abs(got) - 1e-12).all()
    back = OE.experts_backward(dy.numpy(), n[0], n[1], n[2], gu, n[3], n[4], act)
    for name, ref in (("dx", x), ("dweight", w), ("dw_gate_up", wgu), ("dw_down", wd)):
        assert np.allclose(back[name][0], ref.grad.numpy(), rtol=1e-10, atol=1e-12)
        assert (back[name][1] >= np.abs(back[name][0]) - 1e-12).all()


def test_one_expert_is_the_dense_block():
    g = np.random.default_rng(4)
    x, wgu, wd, dy = g.normal(size=(7, 6)), g.normal(size=(1, 6, 10)), g.normal(size=(1, 5, 6)), g.normal(size=(7, 6))
    index, w = np.zeros((7, 1), np.int32), np.ones((7, 1))
    y, gu, _ = OE.experts_forward(x, index, w, wgu, wd, "silu")
    ref, kept, _ = lm.ffn_forward(x, wgu[0], wd[0], "silu")
    assert np.allclose(y, ref) and np.allclose(gu, kept)
    back = OE.experts_backward(dy, x, index, w, gu, wgu, wd, "silu")
    for got, want in zip((back["dx"][0], back["dw_gate_up"][0][0], back["dw_down"][0][0]), lm.ffn_backward(dy, x, kept, wgu[0], wd[0], "silu")):
        assert np.allclose(got, want)
    assert np.allclose(back["dweight"][0][:, 0], (y * dy).sum(1))
