"""Routing tokens to experts on the GPU (zopt_route_forward, zopt_route_backward) against the fp64 oracle.

Tolerances, fixed before the first run: indices and counts equal; weights within
oracle.experts.weight_bound; dlogits within the result's own rounding (fp32 2^-24, bf16 2^-8) and
weight_bound of the magnitudes that it is the difference of; repeated calls bit for bit.
"""
import numpy as np
import pytest
import torch

from oracle import experts as OE

pytestmark = pytest.mark.gpu

# tokens, experts, top_k, score, bias, groups, top_groups, renormalise, scale, dtype
CASES = [
    (1, 1, 1, "softmax", False, 1, 1, True, 1.0, torch.float32),
    (1, 64, 6, "softmax", False, 1, 1, True, 1.0, torch.float32),
    (1, 64, 6, "sigmoid", True, 1, 1, True, 2.5, torch.float32),
    (33, 7, 7, "softmax", False, 1, 1, False, 1.0, torch.float32),
    (100, 33, 4, "softmax", True, 1, 1, False, 1.0, torch.bfloat16),
    (65, 32, 32, "sigmoid", False, 1, 1, False, 0.5, torch.float32),
    (257, 60, 4, "softmax", False, 1, 1, False, 1.0, torch.float32),
    (130, 256, 8, "sigmoid", True, 8, 4, True, 2.5, torch.float32),
    (130, 256, 8, "softmax", True, 8, 3, True, 1.0, torch.bfloat16),
    (70, 130, 5, "softmax", False, 2, 1, True, 1.0, torch.bfloat16),
    (64, 96, 3, "sigmoid", False, 32, 2, True, 1.0, torch.float32),
    (50, 24, 2, "sigmoid", True, 24, 5, False, 1.0, torch.float32),
    (31, 500, 8, "softmax", True, 4, 2, False, 1.0, torch.float32),
    (29, 1024, 32, "sigmoid", True, 32, 32, True, 1.0, torch.bfloat16),
    (1500, 16, 2, "softmax", False, 1, 1, True, 1.0, torch.bfloat16),
]


def make(t, e, top_k, score, bias, groups, top_groups, renorm, scale, dtype, ld=None, seed=0, live=False):
    g = torch.Generator(device="cuda").manual_seed(seed + t + e)
    logits = (torch.randn(t, e, generator=g, device="cuda") * 1.5).to(dtype)
    if ld is not None:
        whole = torch.full((t, ld), float("nan"), dtype=dtype, device="cuda")
        whole[:, :e] = logits
        logits = whole[:, :e]
    b = 0.1 * torch.randn(e, generator=g, device="cuda") if bias else None
    on = torch.rand(t, generator=g, device="cuda") < 0.8 if live else None
    how = dict(score=score, renormalise=renorm, scale=scale)
    return logits, b, on, dict(groups=groups, top_groups=top_groups), how, torch.randn(t, top_k, generator=g, device="cuda")


def forward(Z, logits, top_k, b, on, groups, how, counts=True):
    t, e = logits.shape
    index = torch.full((t, top_k), -7, dtype=torch.int32, device="cuda")
    weight = torch.full((t, top_k), float("nan"), device="cuda")
    n = torch.full((e,), -5, dtype=torch.int32, device="cuda") if counts else None
    Z.route_forward(logits, index, weight, n, bias=b, live=on, **groups, **how)
    torch.cuda.synchronize()
    return index, weight, n


def oracle_of(logits, top_k, b, on, groups, how):
    return OE.route_forward(logits.double().cpu().numpy(), top_k, how["score"], None if b is None else b.double().cpu().numpy(),
                            groups["groups"], groups["top_groups"], how["renormalise"], how["scale"],
                            None if on is None else on.cpu().numpy())


def check_backward(Z, logits, index, weight, dw, how, ld=None):
    t, e = logits.shape
    whole = torch.full((t + 1, ld or e), 777.0, dtype=logits.dtype, device="cuda")
    dl = whole[:t, :e]
    Z.route_backward(logits, index, weight, dw, dl, **how)
    first = dl.clone()
    Z.route_backward(logits, index, weight, dw, dl, **how)
    torch.cuda.synchronize()
    assert torch.equal(first, dl) and bool((whole[t:] == 777.0).all()) and bool((whole[:t, e:] == 777.0).all())
    l, i, g = logits.double().cpu().numpy(), index.cpu().numpy(), dw.double().cpu().numpy()
    ref = OE.route_backward(l, i, g, **how_oracle(how))
    # what dlogits is the difference of: each chosen weight's own term, and the sum's
    w = np.abs(weight.double().cpu().numpy())
    size = np.zeros_like(ref)
    for r in range(t):
        total = (w[r] * np.abs(g[r])).sum()
        for j in range(i.shape[1]):
            if i[r, j] >= 0:
                size[r, i[r, j]] += w[r, j] * (np.abs(g[r, j]) + total / how["scale"])
        if how["score"] == "softmax" and not how["renormalise"] and (i[r] >= 0).any():
            size[r] += OE.scores(l[r], "softmax") * total
    own = (2.0 ** -8 if logits.dtype == torch.bfloat16 else 2.0 ** -24) * np.abs(ref)
    err = np.abs(dl.double().cpu().numpy() - ref)
    assert (err <= own * 1.01 + OE.weight_bound(size)).all(), float((err / (own * 1.01 + OE.weight_bound(size))).max())


def how_oracle(how):
    return dict(kind=how["score"], renormalise=how["renormalise"], scale=how["scale"])


@pytest.mark.parametrize("live", [False, True])
@pytest.mark.parametrize("case", CASES)
def test_route(zopt, case, live):
    t, e, top_k = case[:3]
    ld = e + 3 if live else None
    logits, b, on, groups, how, dw = make(*case, ld=ld, live=live)
    index, weight, counts = forward(zopt, logits, top_k, b, on, groups, how)
    ref_i, ref_w, ref_n = oracle_of(logits, top_k, b, on, groups, how)
    assert np.array_equal(index.cpu().numpy(), ref_i) and np.array_equal(counts.cpu().numpy(), ref_n)
    assert (np.abs(weight.double().cpu().numpy() - ref_w) <= OE.weight_bound(ref_w)).all()
    again = forward(zopt, logits, top_k, b, on, groups, how)
    assert all(torch.equal(a, c) for a, c in zip((index, weight, counts), again))
    assert forward(zopt, logits, top_k, b, on, groups, how, counts=False)[2] is None
    check_backward(zopt, logits, index, weight, dw, how, ld)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_scores_closer_than_fp32_tells_apart(zopt, score):
    """s + bias of neighbours 1e-9 apart, in an order against the index's: 400 rows of such pairs."""
    t, e = 400, 48
    g = torch.Generator(device="cuda").manual_seed(5)
    logits = torch.randn(t, e, generator=g, device="cuda")
    bias = torch.zeros(e, device="cuda")
    logits[:, 24:] = logits[:, :24] + (2.0 ** -22) * (torch.randint(-2, 3, (t, 24), generator=g, device="cuda"))
    bias[24:] = 1e-9
    how, groups = dict(score=score, renormalise=True, scale=1.0), dict(groups=1, top_groups=1)
    index = forward(zopt, logits, 6, bias, None, groups, how)[0]
    assert np.array_equal(index.cpu().numpy(), oracle_of(logits, 6, bias, None, groups, how)[0])
    for n in (4, 12):  # runs whose sums are as close
        groups = dict(groups=n, top_groups=n // 2)
        index = forward(zopt, logits, 3, bias, None, groups, how)[0]
        assert np.array_equal(index.cpu().numpy(), oracle_of(logits, 3, bias, None, groups, how)[0])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_ties_go_to_the_lowest_index(zopt, score, biased):
    logits = torch.zeros(9, 70, device="cuda")
    logits[1, ::2] = 1.0
    logits[2] = -0.0
    logits[2, 5:] = 0.0
    bias = torch.full((70,), 0.25, device="cuda") if biased else None
    how = dict(score=score, renormalise=True, scale=1.0)
    for groups in (dict(groups=1, top_groups=1), dict(groups=7, top_groups=2)):
        index, weight, _ = forward(zopt, logits, 4, bias, None, groups, how)
        assert index[0].tolist() == [0, 1, 2, 3] and index[1].tolist() == [0, 2, 4, 6] and index[2].tolist() == [0, 1, 2, 3]
        assert torch.allclose(weight, torch.full_like(weight, 0.25), rtol=1e-6)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masked_and_extreme_logits(zopt, score, dtype):
    """-inf is never chosen; the type's lowest value is, last; large logits of either sign keep their weights."""
    low, inf = torch.finfo(dtype).min, float("inf")
    l = torch.full((6, 40), -inf, dtype=dtype, device="cuda")
    l[1, 3] = 2.0
    l[2, :] = low
    l[2, 7], l[2, 9] = 1.0, 1.0
    l[3, :] = -200.0
    l[3, 30] = -199.0
    l[4, :] = 300.0
    l[5, ::2] = low
    how, groups = dict(score=score, renormalise=True, scale=2.0), dict(groups=1, top_groups=1)
    for bias in (None, torch.zeros(40, device="cuda")):
        index, weight, counts = forward(zopt, l, 3, bias, None, groups, how)
        assert index[0].tolist() == [-1, -1, -1] and weight[0].tolist() == [0, 0, 0]
        assert index[1].tolist() == [3, -1, -1] and weight[1].tolist() == [2.0, 0, 0]
        assert index[4].tolist() == [0, 1, 2] and int(counts.sum()) == 13
        if bias is None:  # (with one, 1 + 0 and 1e-87 + 0 are ranked as the numbers they are, in fp64)
            assert index[2].tolist() == [7, 9, 0] and weight[2].tolist() == [1.0, 1.0, 0.0]
            assert index[3].tolist() == [30, 0, 1]
            w = np.exp([0.0, -1.0, -1.0])
            assert np.allclose(weight[3].double().cpu().numpy(), 2 * w / w.sum(), rtol=1e-5)
            assert index[5].tolist() == [0, 2, 4]
    dl = torch.empty_like(l)
    index, weight, _ = forward(zopt, l, 3, None, None, groups, how)
    zopt.route_backward(l, index, weight, torch.ones(6, 3, device="cuda"), dl, **how)
    assert bool((dl[0] == 0).all()) and bool(torch.isfinite(dl[:4]).all())
    plain = dict(how, renormalise=False)
    index, weight, _ = forward(zopt, l[:4], 3, None, None, groups, plain)
    zopt.route_backward(l[:4], index, weight, torch.ones(4, 3, device="cuda"), dl[:4], **plain)
    assert bool(torch.isfinite(dl[:4]).all()) and bool((dl[0] == 0).all())


def test_nan_and_infinite_logits_reach_the_weights(zopt):
    l = torch.randn(5, 20, device="cuda")
    l[1, 4], l[2, 6] = float("nan"), float("inf")
    l[3] = float("nan")
    groups = dict(groups=1, top_groups=1)
    for renorm in (True, False):
        index, weight, _ = forward(zopt, l, 2, None, None, groups, dict(score="softmax", renormalise=renorm, scale=1.0))
        assert index[1, 0] == 4 and index[2, 0] == 6 and index[3].tolist() == [0, 1]
        assert bool(torch.isnan(weight[1:4]).all()) and bool(torch.isfinite(weight[[0, 4]]).all())
    index, weight, _ = forward(zopt, l, 2, None, None, groups, dict(score="sigmoid", renormalise=False, scale=1.0))
    assert index[1, 0] == 4 and torch.isnan(weight[1, 0]) and torch.isfinite(weight[1, 1])
    assert index[2, 0] == 6 and weight[2, 0] == 1.0
    live = torch.tensor([True, False, False, False, True], device="cuda")  # padding hides them
    for bias in (None, torch.zeros(20, device="cuda")):
        index, weight, _ = forward(zopt, l, 2, bias, live, groups, dict(score="softmax", renormalise=True, scale=1.0))
        assert bool((index[1:4] == -1).all()) and bool((weight[1:4] == 0).all())
        dl = torch.empty_like(l)
        for renorm in (True, False):
            zopt.route_backward(l, index, weight, torch.full((5, 2), float("nan"), device="cuda"), dl, renormalise=renorm)
            assert bool((dl[1:4] == 0).all())


def test_an_index_out_of_range_poisons_its_row(zopt):
    l = torch.randn(4, 20, device="cuda")
    how, groups = dict(score="softmax", renormalise=True, scale=1.0), dict(groups=1, top_groups=1)
    index, weight, _ = forward(zopt, l, 2, None, None, groups, how)
    index[1, 0], index[2, 1] = 20, -2
    dl = torch.empty_like(l)
    zopt.route_backward(l, index, weight, torch.ones(4, 2, device="cuda"), dl, **how)
    assert bool(torch.isnan(dl[1:3]).all()) and bool(torch.isfinite(dl[[0, 3]]).all())


def test_no_tokens(zopt):
    l = torch.empty(0, 8, device="cuda")
    index, weight, counts = forward(zopt, l, 2, None, None, dict(groups=1, top_groups=1), dict(score="softmax", renormalise=True, scale=1.0))
    assert bool((counts == 0).all())
    zopt.route_backward(l, index, weight, torch.empty(0, 2, device="cuda"), torch.empty_like(l))
    torch.cuda.synchronize()


def test_captured_and_replayed_on_new_logits(zopt):
    case = CASES[7]
    logits, b, _, groups, how, dw = make(*case)
    t, top_k = case[0], case[2]
    index, weight, counts = forward(zopt, logits, top_k, b, None, groups, how)
    dl = torch.empty_like(logits)
    zopt.route_backward(logits, index, weight, dw, dl, **how)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        zopt.route_forward(logits, index, weight, counts, bias=b, **groups, **how)
        zopt.route_backward(logits, index, weight, dw, dl, **how)
    for seed in (1, 2):
        logits.copy_(make(*case, seed=seed)[0])
        g.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in (index, weight, counts, dl)]
        want = forward(zopt, logits, top_k, b, None, groups, how)
        zopt.route_backward(logits, *want[:2], dw, dl, **how)
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(got, (*want, dl)))


def test_on_a_stream_of_its_own(zopt):
    case = CASES[8]
    logits, b, _, groups, how, _ = make(*case)
    want = forward(zopt, logits, case[2], b, None, groups, how)
    s = torch.cuda.Stream()
    got = [torch.empty_like(x) for x in want]
    s.wait_stream(torch.cuda.current_stream())
    zopt.route_forward(logits, *got, bias=b, **groups, **how, stream=s)
    s.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(want, got))


def test_many_rows(zopt):
    """More rows than one wave of warps, every one's choice."""
    logits, b, on, groups, how, dw = make(40000, 64, 6, "sigmoid", True, 1, 1, True, 1.0, torch.float32, live=True)
    index, weight, counts = forward(zopt, logits, 6, b, on, groups, how)
    c = torch.sigmoid(logits.double()) + b.double()
    want = c.sort(dim=1, descending=True, stable=True).indices[:, :6].int()
    assert torch.equal(index, torch.where(on[:, None], want, -1))
    assert torch.equal(counts, torch.bincount(want[on].flatten(), minlength=64).int())
    s = torch.sigmoid(logits.double()).gather(1, want.long())
    w = torch.where(on[:, None], s / s.sum(1, keepdim=True), 0.0)
    assert bool(((weight.double() - w).abs() <= 2.0 ** -16 * w).all())


def test_refusals(zopt):
    l = torch.randn(4, 8, device="cuda")
    index, weight = torch.empty(4, 2, dtype=torch.int32, device="cuda"), torch.empty(4, 2, device="cuda")
    with pytest.raises(ValueError, match="index"):
        zopt.route_forward(l, index.long(), weight)
    with pytest.raises(ValueError, match="weight"):
        zopt.route_forward(l, index, weight.bfloat16())
    with pytest.raises(ValueError, match="bias"):
        zopt.route_forward(l, index, weight, bias=torch.zeros(7, device="cuda"))
    with pytest.raises(ValueError, match="live"):
        zopt.route_forward(l, index, weight, live=torch.zeros(4, device="cuda"))
    with pytest.raises(ValueError, match="counts"):
        zopt.route_forward(l, index, weight, torch.zeros(8, device="cuda"))
    for bad in (l.half(), l.double(), l.int()):
        with pytest.raises(zopt.ZoptError, match="dtype"):
            zopt.route_forward(bad, index, weight)
    with pytest.raises(zopt.ZoptError, match="score"):
        zopt.route_forward(l, index, weight, score="tanh")
    with pytest.raises(zopt.ZoptError, match="dtype"):
        zopt.route_backward(l, index, weight, weight, l.bfloat16())
