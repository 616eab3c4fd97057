"""The training operators' results in norm, and at extremes entry by entry, against the fp64 oracle.

Tolerances, fixed before the first run:
* in norm: a rounding to bf16 (8 significant bits) is uniform in a step of 2^-7 of a mantissa that is at
  least 1: 2^-7 / sqrt(12) = 2.26e-3 rms at most. A gradient takes two, its operand's and its own, which
  are independent: sqrt(2) times that;
* a row by itself may be one term's: 2^-8 for each of the two roundings;
* at large logits: p = exp(l - lse) with l and lse off by d = 2^-20 of (1 + the largest |x||w| sum) and
  2^-23 of lse, so p by (exp(d) - 1) p, on top of oracle.lm.product_bound.
"""
import numpy as np
import pytest
import torch

from oracle import lm
from tests.test_gpu_lm import ce_case, check_ffn, f64, ffn_case, rows, run_ce, run_ffn, within

pytestmark = pytest.mark.gpu

TWO = 2 ** 0.5 * 2.0 ** -7 / 12 ** 0.5


def off(got, ref):
    return float(np.linalg.norm(f64(got) - ref) / np.linalg.norm(ref))


def row_off(got, ref):
    n = np.linalg.norm(ref, axis=1)
    return float((np.linalg.norm(f64(got) - ref, axis=1)[n > 0] / n[n > 0]).max())


@pytest.mark.parametrize("weights", ["random", "mean"])
@pytest.mark.parametrize("t,d,v", [(510, 128, 2000), (777, 264, 4099), (300, 72, 777)])
def test_cross_entropy_gradients_in_norm(zopt, t, d, v, weights):
    """Also where every row has the same weight, 1 / 255, half a step beyond a bf16 value: rounded along
    with it, every target's entry, near -1, would carry the same 2^-8 (3.8e-3 of dx and dw)."""
    x, w, target, dloss = ce_case(t, t, d, v)
    if weights == "mean":
        dloss.fill_(1 / 255)
    _, lse, dx, dw = run_ce(zopt, x, w, target, dloss)
    X, W, y = f64(x), f64(w), target.cpu().numpy()
    rx, rw = lm.ce_backward(X, W, y, lm.ce_forward(X, W, y)[1], f64(dloss))
    assert off(dx, rx) <= TWO and off(dw, rw) <= TWO
    assert row_off(dx, rx) <= 2 * 2.0 ** -8


@pytest.mark.parametrize("keep", ["bf16", "e4m3"])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("t,d,f", [(513, 264, 520), (300, 100, 1030), (1023, 256, 768)])
def test_block_in_norm(zopt, t, d, f, act, keep):
    x, dy, wgu, wd = ffn_case(t + f, t, d, f)
    got, kept, x8 = run_ffn(zopt, x, dy, wgu, wd, act, keep)
    y = lm.ffn_forward(f64(x), f64(wgu), f64(wd), act)[0]
    if x8 is None:
        K, XK = f64(kept), f64(x)
    else:
        K = lm.act8_unpack(kept.q.cpu().numpy(), kept.scale.cpu().numpy(), 2)
        XK = lm.act8_unpack(x8.q.cpu().numpy(), x8.scale.cpu().numpy())
    ref = dict(zip(("dx", "dw_gate_up", "dw_down"), lm.ffn_backward(f64(dy), XK, K, f64(wgu), f64(wd), act)), y=y)
    for n in ref:
        assert off(got[n], ref[n]) <= TWO, n


@pytest.mark.parametrize("keep", ["bf16", "e4m3"])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("t", [2, 40])
def test_block_of_extreme_gates(zopt, t, act, keep):
    """Gates of thousands, either sign, where a ends at 0 or z and a' at 0 or 1."""
    x, dy, wgu, wd = ffn_case(3, t, 64, 96)
    wgu = wgu.clone()
    wgu[:, :96] *= 4000
    got, kept, x8 = run_ffn(zopt, x, dy, wgu, wd, act, keep)
    check_ffn(x, dy, wgu, wd, act, got, kept, x8)


def test_cross_entropy_gradients_of_large_logits(zopt):
    """Logits of +-2e4: one entry of a row has all of its weight, or two share it."""
    gen = torch.Generator(device="cuda").manual_seed(9)
    x, w = rows(gen, 50, 64, 40.0), rows(gen, 700, 64, 40.0)
    x[7] = 0
    target = torch.randint(0, 700, (50,), generator=gen, device="cuda")
    target[::2] = (x[::2].float() @ w.float().T).argmax(1)  # rows with next to no loss, and rows with much
    _, lse, dx, dw = run_ce(zopt, x, w, target, torch.ones(50, device="cuda"))
    X, W, y = f64(x), f64(w), target.cpu().numpy()
    rl = lm.ce_forward(X, W, y)[1]
    dl = lm.ce_dlogits(X, W, y, rl, np.ones(50))
    p = np.exp(X @ W.T - rl[:, None])
    d = 2.0 ** -20 * (1 + (np.abs(X) @ np.abs(W).T).max(axis=1)) + 2.0 ** -23 * np.abs(rl)
    slack = np.abs(dl) + 2.0 ** 8 * p * np.expm1(d)[:, None]  # (product_bound takes 2^-8 of it)
    within(dx, dl @ W, slack @ np.abs(W))
    within(dw, dl.T @ X, slack.T @ np.abs(X))
