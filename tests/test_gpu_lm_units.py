"""The block and the cross entropy at sizes where every CTA pair has several tiles, against fp64 torch on
the GPU: accumulators in turn, what a tile hands to the next one (the 8-bit blocks' exchange, gate, up
and powers on their way), tiles of either width, gate and up that start on and off 16 bytes, and the
gradients' units both dealt out by length and taken in turn.

Tolerances, fixed before the first run:
* entry by entry, oracle.lm.product_bound with the operands' own errors, as in test_gpu_lm.py;
* in norm: a rounding to bf16 (8 significant bits) is uniform in a step of 2^-7 of a mantissa that is at
  least 1, 2^-7 / sqrt(12) = 2.26e-3 rms at most. A result takes two, its operand's and its own, which
  are independent: sqrt(2) times that; what was kept takes one. Sums of hundreds of terms in the places
  of a few wrong ones would differ by percents.
"""
import numpy as np
import pytest
import torch

from oracle import lm
from tests.test_gpu_lm import ffn_case, run_ffn

pytestmark = pytest.mark.gpu

ONE = 2.0 ** -7 / 12 ** 0.5
TWO = 2 ** 0.5 * ONE

SHAPES = [  # tokens, dim, hidden
    (4099, 128, 2832),  # gate and up: 765 tiles of 64 columns (391 of 128 in 8 bits); dh: 204 of 256
    (4099, 136, 2732),  # rows off 16 bytes; gate and up: 374 tiles of 128 columns; dh: 374 of 128
    (5130, 72, 1303),   # odd rows; dh: 126 tiles of 256; the gradients' 55 units, one a pair
    (300, 2056, 5000),  # the gradients: 630 units, in turn
]


def gate64(z, act):
    if act == "silu":
        s = torch.sigmoid(z)
        return z * s, s * (1 + z * (1 - s))
    c = (2 / np.pi) ** 0.5
    t = torch.tanh(c * (z + 0.044715 * z ** 3))
    return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)


def close(got, ref, abs_product, norm):
    got = got.double()
    assert torch.isfinite(got).all()
    bound = 1.125 * 2.0 ** -8 * (ref.abs() + abs_product) + 1e-30  # (oracle.lm.product_bound)
    worst = float(((got - ref).abs() / bound).max())
    assert worst <= 1.0, worst
    off = float((got - ref).norm() / ref.norm())
    assert off <= norm, off


def unpacked(c):
    """What a checkpoint stands for, in fp64, from its bytes."""
    rows, width = c.rows, c.cols // c.parts
    nb = -(-width // 128)
    s = torch.exp2(c.scale.double().reshape(rows, c.parts, nb) - 127)
    s = s.repeat_interleave(128, 2)[:, :, :width].reshape(rows, c.cols)
    return torch.tensor(lm.e4m3_values(), device="cuda")[c.q.long()] * s, s


def check(x, dy, wgu, wd, act, got, kept, x8):
    X, DY, G, D, f = x.double(), dy.double(), wgu.double(), wd.double(), wd.shape[0]
    gu = X @ G
    g, u = gu[:, :f], gu[:, f:]
    h = gate64(g, act)[0] * u
    sg = X.abs() @ G.abs()
    # h's error before its rounding: the fp32 sums of g and u (2^-16 of sum |x||w| each, |a'| < 1.2)
    hs = h.abs() + 2.0 ** -7 * (sg[:, :f] * u.abs() * 1.2 + g.abs() * sg[:, f:])
    close(got["y"], h @ D, hs @ D.abs(), TWO)
    if x8 is None:
        close(kept, gu, 2.0 ** -4 * sg, ONE)
        K, XK = kept.double(), X
    else:
        K, s = unpacked(kept)
        # half a step of the format, and the fp32 sums' error
        assert ((K - gu).abs() <= torch.maximum(2.0 ** -4 * gu.abs(), 2.0 ** -10 * s) + 2.0 ** -16 * sg).all()
        pad = torch.nn.functional.pad
        nb = -(-f // 128)
        top = pad(gu.reshape(-1, 2, f), (0, 128 * nb - f)).reshape(-1, 2, nb, 128).abs().amax(3)
        power = torch.exp2(kept.scale.double().reshape(top.shape) - 127)
        assert (top <= 448 * power * (1 + 2.0 ** -12)).all() and (top >= 224 * power * (1 - 2.0 ** -12)).all()
        XK = unpacked(x8)[0]
        assert ((XK - X).abs() <= torch.maximum(2.0 ** -4 * X.abs(), 2.0 ** -10 * unpacked(x8)[1])).all()
    kg, ku = K[:, :f], K[:, f:]
    a, da = gate64(kg, act)
    dh = DY @ D.T
    dgu = torch.cat((dh * ku * da, dh * a), 1)
    sdh = 2.0 ** -7 * (DY.abs() @ D.abs().T) + 2.0 ** -10 * dh.abs()
    gs = dgu.abs() + torch.cat((sdh * ku.abs() * 1.2, sdh * kg.abs()), 1)
    close(got["dx"], dgu @ G.T, gs @ G.abs().T, TWO)
    close(got["dw_gate_up"], XK.T @ dgu, XK.abs().T @ gs, TWO)
    close(got["dw_down"], (a * ku).T @ DY, ((a * ku).abs() * (1 + 2.0 ** -10)).T @ DY.abs(), TWO)


@pytest.mark.parametrize("keep", ["bf16", "e4m3"])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("t,d,f", SHAPES)
def test_block_of_many_tiles(zopt, t, d, f, act, keep):
    args = ffn_case(t + d + f, t, d, f)
    got, kept, x8 = run_ffn(zopt, *args, act, keep)
    check(*args, act, got, kept, x8)
    again, kept2, _ = run_ffn(zopt, *args, act, keep)
    assert all(torch.equal(got[n], again[n]) for n in got)
    assert torch.equal(kept, kept2) if keep == "bf16" else torch.equal(kept.q, kept2.q) and torch.equal(kept.scale, kept2.scale)


@pytest.mark.parametrize("t,d,f", SHAPES[:3])
def test_block_of_many_tiles_keeps_nothing(zopt, t, d, f):
    x, dy, wgu, wd = ffn_case(t, t, d, f)
    kept = run_ffn(zopt, x, dy, wgu, wd, "silu", "bf16")[0]["y"]
    y = torch.empty(t, d, dtype=torch.bfloat16, device="cuda")
    zopt.ffn_forward(x, wgu, wd, y, zopt.new_ffn_workspace(x, wgu, wd, backward=False))
    torch.cuda.synchronize()
    assert torch.equal(y, kept)
