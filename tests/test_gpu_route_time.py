"""Rows that need no second look do not get one: a balance's bias costs the same wherever it lies."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def microseconds(call, times=20, tries=7):
    """The least of a few means: a call among others."""
    best = float("inf")
    for _ in range(tries):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        call()
        a.record()
        for _ in range(times):
            call()
        b.record()
        b.synchronize()
        best = min(best, 1e3 * a.elapsed_time(b) / times)
    return best


def forward(Z, logits, bias, top_k, **how):
    t, e = logits.shape
    index, weight = torch.empty(t, top_k, dtype=torch.int32, device="cuda"), torch.empty(t, top_k, device="cuda")
    counts = torch.empty(e, dtype=torch.int32, device="cuda")
    return lambda: Z.route_forward(logits, index, weight, counts, bias=bias, **how)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e", [8, 60, 160, 384])
def test_a_common_shift_of_the_bias_costs_nothing(zopt, e, score):
    """Lanes behind the last expert, where experts do not fill a warp, stay out of a row's checks."""
    g = torch.Generator(device="cuda").manual_seed(e)
    logits = torch.randn(8192, e, generator=g, device="cuda")
    spread = 0.04 * torch.rand(e, generator=g, device="cuda")
    centred = microseconds(forward(zopt, logits, spread - 0.02, 4, score=score))
    for shift in (0.01, -0.05):
        shifted = microseconds(forward(zopt, logits, spread + shift, 4, score=score))
        assert shifted <= 1.5 * centred + 2.0, (shifted, centred)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_rows_ranked_from_all_experts(zopt, score):
    """Biases whose spread leaves no fixed point send every row to the ranking of all its experts, which a lane goes
    through once or twice, not for every choice: in the time of a few choices, not of all eight."""
    logits = torch.randn(8192, 256, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    bias = torch.zeros(256, device="cuda")
    bias[::8] = torch.finfo(torch.float32).min
    one, eight = (microseconds(forward(zopt, logits, bias, k, score=score)) for k in (1, 8))
    assert eight <= 4.0 * one, (one, eight)
