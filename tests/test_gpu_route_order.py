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
    l = logits_of(4, e, e)
    same(zopt, l, 6, score, masks(e, low))
    same(zopt, l, 6, score, masks(e, low), 4, 2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e", [8, 24, 32, 60, 256])
@pytest.mark.parametrize("low", [-1e38, torch.finfo(torch.float32).min])
def test_biases_of_the_lowest_value(zopt, e, score, low):
    """The range's reciprocal is no normal number: no fixed point holds such ranks."""
    l = logits_of(4, e, e)
    same(zopt, l, 3, score, masks(e, low))
    if e >= 24:
        same(zopt, l, 3, score, masks(e, low), 4, 2)


def close_pairs(t, e, seed, sigma):
    """Half of the experts an fp32 step or two from their neighbours in the first rows."""
    l = logits_of(t, e, seed, sigma)
    l[:t // 2, 1:e // 2 * 2:2] = l[:t // 2, :e // 2 * 2:2] * (1 + 2.0 ** -22)
    return l


BIASES = {
    "none": lambda e: None,
    "zeros": lambda e: torch.zeros(e),
    "equal, large": lambda e: torch.full((e,), 1e10),
    "tiny": lambda e: 1e-30 * (torch.arange(e) % 2),
    "a few of the highest": lambda e: torch.where(torch.arange(e) % 5 == 0, torch.finfo(torch.float32).max, 0.0),
    "spread": lambda e: 0.05 * torch.randn(e, generator=torch.Generator().manual_seed(e)),
    "spread, shifted": lambda e: 100.0 + 0.1 * torch.rand(e, generator=torch.Generator().manual_seed(e)),
}


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", BIASES)
@pytest.mark.parametrize("e", [8, 60, 160])
def test_sums_that_fp64_does_not_tell_apart(zopt, e, bias, score):
    """Logits up to some 100: logistic scores that are 1 in fp64, softmax scores far below a bias's last bit."""
    for sigma in (1.0, 30.0):
        l = close_pairs(4, e, e, sigma)
        b = BIASES[bias](e)
        b = None if b is None else b.float().cuda()
        same(zopt, l, 5, score, b)
        same(zopt, l, 2, score, b, 4, 2)
        same(zopt, l.bfloat16(), 5, score, b)


def test_saturated_scores_by_their_logits(zopt):
    l = torch.tensor([[0.0, 40.0, 50.0, 1.0, 60.0, 45.0], [-730.0, -705.0, -740.0, 0.0, -710.0, -800.0]], device="cuda")
    for bias in (None, torch.zeros(6, device="cuda"), torch.full((6,), -3e5, device="cuda")):
        assert chosen(zopt, l, 4, "sigmoid", bias).tolist() == [[4, 2, 5, 1], [3, 1, 4, 0]]
        assert chosen(zopt, l, 4, "softmax", bias).tolist() == [[4, 2, 5, 1], [3, 1, 4, 0]]
    assert chosen(zopt, l[:1], 2, "sigmoid", None, 3, 1).tolist() == [[4, 5]]
