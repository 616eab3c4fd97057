"""CPU pins of the training operators' oracle: closed forms, torch's double-precision operators and
autograd, gradients against central differences, the e4m3 format against torch's own type."""
import math

import numpy as np
import pytest
import torch

from oracle import lm


@pytest.mark.parametrize("seed,t,d,v", [(0, 5, 7, 11), (1, 1, 3, 1), (2, 9, 4, 30)])
def test_cross_entropy_against_torch(seed, t, d, v):
    rng = np.random.default_rng(seed)
    x, w = rng.normal(size=(t, d)), rng.normal(size=(v, d))
    target = rng.integers(0, v, t)
    target[::4] = -100
    dloss = rng.normal(size=t)
    loss, lse = lm.ce_forward(x, w, target)
    tx, tw = torch.tensor(x, requires_grad=True), torch.tensor(w, requires_grad=True)
    tl = torch.nn.functional.cross_entropy(tx @ tw.T, torch.tensor(target), reduction="none")
    assert np.allclose(loss, tl.detach().numpy(), rtol=0, atol=1e-13)
    gx, gw = torch.autograd.grad((tl * torch.tensor(dloss)).sum(), (tx, tw))
    dx, dw = lm.ce_backward(x, w, target, lse, dloss)
    assert np.allclose(dx, gx.numpy(), rtol=0, atol=1e-13) and np.allclose(dw, gw.numpy(), rtol=0, atol=1e-13)


def test_cross_entropy_closed_forms():
    loss, lse = lm.ce_forward(np.zeros((2, 3)), np.ones((8, 3)), [5, -100])
    assert np.allclose(loss, [math.log(8), 0]) and np.allclose(lse, [math.log(8), 0])
    dx, dw = lm.ce_backward(np.zeros((1, 3)), np.ones((8, 3)), [5], [math.log(8)], [1.0])
    assert np.allclose(dx, 0) and np.allclose(dw, 0)
    x = np.array([[np.nan, 1.0], [0.5, 2.0]])  # an ignored row's values do not matter
    dx, dw = lm.ce_backward(x, np.eye(2), [-100, 1], lm.ce_forward(x, np.eye(2), [-100, 1])[1], [7.0, 1.0])
    assert np.all(dx[0] == 0) and np.isfinite(dw).all()


def _differences(f, a, step=1e-5):
    g = np.zeros_like(a)
    for i in np.ndindex(a.shape):
        up, down = a.copy(), a.copy()
        up[i] += step
        down[i] -= step
        g[i] = (f(up) - f(down)) / (2 * step)
    return g


def test_cross_entropy_gradient_against_differences():
    rng = np.random.default_rng(3)
    x, w, target, dloss = rng.normal(size=(4, 5)), rng.normal(size=(9, 5)), np.array([1, -100, 8, 0]), rng.normal(size=4)
    total = lambda x, w: (lm.ce_forward(x, w, target)[0] * dloss).sum()  # noqa: E731
    dx, dw = lm.ce_backward(x, w, target, lm.ce_forward(x, w, target)[1], dloss)
    # central differences of a smooth function: step^2 of its third derivative and 1e-16 / step
    assert np.allclose(dx, _differences(lambda a: total(a, w), x), rtol=0, atol=1e-8)
    assert np.allclose(dw, _differences(lambda a: total(x, a), w), rtol=0, atol=1e-8)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_block_against_torch_and_differences(act):
    rng = np.random.default_rng(4)
    x, wgu, wd = rng.normal(size=(3, 4)), rng.normal(size=(4, 10)), rng.normal(size=(5, 4))
    dy = rng.normal(size=(3, 4))
    y, gu, _ = lm.ffn_forward(x, wgu, wd, act)
    ts = [torch.tensor(a, requires_grad=True) for a in (x, wgu, wd)]
    g = ts[0] @ ts[1]
    a = torch.nn.functional.silu(g[:, :5]) if act == "silu" else torch.nn.functional.gelu(g[:, :5], approximate="tanh")
    ty = (a * g[:, 5:]) @ ts[2]
    assert np.allclose(y, ty.detach().numpy(), rtol=0, atol=1e-13)
    ref = torch.autograd.grad((ty * torch.tensor(dy)).sum(), ts)
    got = lm.ffn_backward(dy, x, gu, wgu, wd, act)
    for r, q in zip(ref, got):
        assert np.allclose(r.numpy(), q, rtol=0, atol=1e-12)
    total = lambda *p: (lm.ffn_forward(*p, act)[0] * dy).sum()  # noqa: E731
    assert np.allclose(got[0], _differences(lambda v: total(v, wgu, wd), x), rtol=0, atol=1e-7)
    assert np.allclose(got[1], _differences(lambda v: total(x, v, wd), wgu), rtol=0, atol=1e-7)
    assert np.allclose(got[2], _differences(lambda v: total(x, wgu, v), wd), rtol=0, atol=1e-7)


def test_gate_at_extremes():
    for act in ("silu", "gelu"):
        a, da = lm.gate(np.array([-200.0, 0.0, 200.0]), act)
        assert np.allclose(a, [0, 0, 200]) and np.allclose(da, [0, 0.5, 1])


def test_e4m3_is_torchs():
    bytes_ = np.arange(256, dtype=np.uint8)
    ref = torch.from_numpy(bytes_).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(lm.e4m3_values(), ref, equal_nan=True)
    rng = np.random.default_rng(5)
    z = np.concatenate([rng.normal(size=20000) * np.exp(rng.normal(size=20000) * 3), [0.0, -0.0, 448.0, -448.0]])
    z = z[np.abs(z) <= 448].astype(np.float32)
    pos = lm.e4m3_values()[:127]
    ties = ((pos[1:] + pos[:-1]) / 2).astype(np.float32)
    z = np.concatenate([z, ties, -ties, np.nextafter(ties, 0), np.nextafter(ties, 1000)])
    assert np.array_equal(lm.e4m3_bytes(z), torch.from_numpy(z).to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_checkpoint_closed_forms():
    x = np.zeros((1, 260))
    x[0, 0], x[0, 1], x[0, 130], x[0, 256] = 448.0, -1.0, 449.0, 2.0 ** -130
    q, scale = lm.act8_pack(x)
    assert list(scale[0]) == [127, 128, 1]  # 448 fits 2^0, 449 needs 2^1, a tiny block the smallest power
    v = lm.act8_unpack(q, scale)
    assert v[0, 0] == 448 and v[0, 1] == -1 and v[0, 130] == 448
    x[0, 5], x[0, 6] = np.inf, np.nan  # neither spoils its block
    q, scale = lm.act8_pack(x)
    v = lm.act8_unpack(q, scale)
    assert list(scale[0]) == [127, 128, 1] and np.isnan(v[0, 5]) and np.isnan(v[0, 6]) and v[0, 0] == 448


@pytest.mark.parametrize("parts,cols", [(1, 128), (1, 300), (2, 260), (2, 2), (1, 1)])
def test_checkpoint_error_is_half_a_step(parts, cols):
    rng = np.random.default_rng(cols)
    x = rng.normal(size=(6, cols)) * np.exp(2 * rng.normal(size=(6, 1)))
    q, scale = lm.act8_pack(x, parts)
    v = lm.act8_unpack(q, scale, parts)
    nb = -(-(cols // parts) // 128)
    s = np.repeat(2.0 ** (scale.reshape(6, parts, nb).astype(float) - 127), 128, axis=2)[:, :, :cols // parts].reshape(6, cols)
    assert np.all(np.abs(v - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * s))
    # packing what it stands for changes no value (a block whose largest entry was rounded down to
    # 224 2^e may take the next smaller power, on which every value still lies)
    assert np.array_equal(lm.act8_unpack(*lm.act8_pack(v, parts), parts), v)


def test_product_bound_holds_for_correctly_rounded_values_and_is_no_wider_than_it_says():
    """bf16 keeps 8 significant bits: a correctly rounded result is up to 2^-8 of itself off."""
    x = np.concatenate([1 + np.arange(1, 4096) * 2.0 ** -12, np.random.default_rng(6).normal(size=10000)])
    r = torch.tensor(x).to(torch.bfloat16).double().numpy()
    err = np.abs(r - x)
    assert np.all(err <= lm.product_bound(x, 0.0))
    assert (err / np.abs(x)).max() > 0.98 * 2.0 ** -8
    assert lm.product_bound(1.0, 1.0) < 2.3 * 2.0 ** -8
