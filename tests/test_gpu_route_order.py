"""The order of the routing's choices where sums of scores and biases are hard to tell apart or far apart: index
for index the choice of decimal numbers (oracle/choice.py)."""
import numpy as np
import pytest
import torch

from oracle.choice import choose

pytestmark = pytest.mark.gpu


def chosen(Z, logits, top_k, score, bias, groups=1, top_groups=1):
    t, e = logits.shape
    index = torch.full((t, top_k), -7, dtype=torch.int32, device="cuda")
    weight, counts = torch.empty(t, top_k, device="cuda"), torch.empty(e, dtype=torch.int32, device="cuda")
    Z.route_forward(logits, index, weight, counts, bias=bias, score=score, groups=groups, top_groups=top_groups)
    torch.cuda.synchronize()
    got = index.cpu().numpy()
    assert np.array_equal(counts.cpu().numpy(), np.bincount(got.flatten(), minlength=e))
    return got


def same(Z, logits, top_k, score, bias, groups=1, top_groups=1):
    want = choose(logits.double().cpu().numpy(), top_k, score, None if bias is None else bias.double().cpu().numpy(), groups, top_groups)
    assert np.array_equal(chosen(Z, logits, top_k, score, bias, groups, top_groups), want)


def logits_of(t, e, seed, sigma=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(t, e, generator=g, device="cuda") * sigma


def masks(e, low):
    """A third of the experts pushed out of the way, the others' biases as a balance has them."""
    bias = 0.01 * torch.randn(e, generator=torch.Generator().manual_seed(e))
    bias[::3] = low
    return bias.cuda()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e", [24, 60, 256])
@pytest.mark.parametrize("low", [-1e4, -8e37])
def test_biases_far_larger_than_scores(zopt, e, score, low):
    """Where every rank is closer to the next than its error, and that error passes 31 bits."""
    l = logits_of(12, e, e)
    same(zopt, l, 6, score, masks(e, low))
    same(zopt, l, 6, score, masks(e, low), 4, 2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e", [8, 24, 32, 60, 256])
@pytest.mark.parametrize("low", [-1e38, torch.finfo(torch.float32).min])
def test_biases_of_the_lowest_value(zopt, e, score, low):
    """The range's reciprocal is no normal number: no fixed point holds such ranks."""
    l = logits_of(12, e, e)
    same(zopt, l, 3, score, masks(e, low))
    if e >= 24:
        same(zopt, l, 3, score, masks(e, low), 4, 2)
