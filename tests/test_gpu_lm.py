"""The training operators on the GPU (zopt_linear_ce_*, zopt_ffn_*, zopt_act_*) against the fp64
oracle.

Tolerances, fixed before the first run:
* a bf16 result of a product: oracle.lm.product_bound, entry by entry (its own rounding and the
  rounding of one operand to bf16, each bf16's unit roundoff 2^-8, with 1/8 on top);
* loss and lse (fp32): the logits' fp32 sums over D terms and the exponentials' 2^-22 leave an
  absolute error below 2^-20 of (1 + the largest |x||w| sum of the row), and a rounding of 2^-23 of
  the result;
* 8-bit checkpoints of bf16 input: bit for bit; of the block's own gate and up: half a step of the
  format on its own power of two, plus the fp32 sum's error;
* repeated calls: bit for bit.
"""
import numpy as np
import pytest
import torch

from oracle import lm

pytestmark = pytest.mark.gpu


def rows(gen, t, d, sigma=1.0, ld=None, offset=0):
    """A t x d bf16 matrix, optionally inside rows of ld elements filled with a sentinel."""
    a = (torch.randn(t, d, generator=gen, device="cuda") * sigma).bfloat16()
    return a if ld is None else framed(a, ld)


SENTINEL = 777.0


def framed(a, ld):
    whole = torch.full((a.shape[0] + 1, ld), SENTINEL, dtype=a.dtype, device="cuda")
    v = whole[:a.shape[0], :a.shape[1]]
    v.copy_(a)
    return v


def frame_of(t, d, ld=None):
    """An output matrix and what surrounds it."""
    ld = ld or d
    whole = torch.full((t + 1, ld), SENTINEL, dtype=torch.bfloat16, device="cuda")
    return whole, whole[:t, :d]


def untouched(whole, t, d):
    return bool((whole[:t, d:] == SENTINEL).all()) and bool((whole[t:] == SENTINEL).all())


def f64(t):
    return t.detach().double().cpu().numpy()


def within(got, ref, abs_product):
    bound = lm.product_bound(ref, abs_product)
    err = np.abs(f64(got) - ref)
    assert np.isfinite(f64(got)).all()
    worst = float((err / bound).max()) if err.size else 0.0
    assert worst <= 1.0, worst


# --------------------------------------------------------------------------- cross entropy

CE_SHAPES = [  # tokens, dim, vocab, row distance of x and w (None: contiguous)
    (1, 8, 1, None), (1, 256, 4096, None), (2, 64, 257, None), (31, 40, 129, None), (33, 100, 1000, None),
    (257, 96, 255, None), (300, 72, 777, 80), (129, 33, 300, None), (64, 50, 511, 61), (130, 264, 4099, None),
    (513, 128, 2049, None),
]


def ce_case(seed, t, d, v, ld=None, ignored=0.2):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x, w = rows(gen, t, d, ld=ld), rows(gen, v, d, 0.3, ld=ld)
    target = torch.randint(0, v, (t,), generator=gen, device="cuda")
    drop = torch.rand((t,), generator=gen, device="cuda") < ignored
    target[drop] = -100
    dloss = torch.randn((t,), generator=gen, device="cuda")
    return x, w, target, dloss


def run_ce(Z, x, w, target, dloss, ld_out=None, ignore=-100):
    t, d, v = x.shape[0], x.shape[1], w.shape[0]
    loss, lse = torch.empty(t, device="cuda"), torch.empty(t, device="cuda")
    ws = Z.new_linear_ce_workspace(x, w)
    ws.fill_(255)  # NaN in every type: nothing may be read before it is written
    (wdx, dx), (wdw, dw) = frame_of(t, d, ld_out), frame_of(v, d, ld_out)
    Z.linear_ce_forward(x, w, target, loss, lse, ws, ignore_index=ignore)
    Z.linear_ce_backward(x, w, target, lse, dloss, dx, dw, ws, ignore_index=ignore)
    torch.cuda.synchronize()
    assert Z.take_device_error() == 0
    assert untouched(wdx, t, d) and untouched(wdw, v, d)
    return loss, lse, dx, dw


def check_ce(x, w, target, dloss, got, ignore=-100):
    loss, lse, dx, dw = got
    X, W, y = f64(x), f64(w), target.cpu().numpy()
    rl, re = lm.ce_forward(X, W, y, ignore)
    size = 1 + (np.abs(np.nan_to_num(X)) @ np.abs(W).T).max(axis=1)
    assert np.all(np.abs(f64(loss) - rl) <= 2.0 ** -20 * size + 2.0 ** -23 * np.abs(rl))
    assert np.all(np.abs(f64(lse) - re) <= 2.0 ** -20 * size + 2.0 ** -23 * np.abs(re))
    assert np.all(f64(loss)[y == ignore] == 0) and np.all(f64(lse)[y == ignore] == 0)
    dl = lm.ce_dlogits(np.nan_to_num(X), W, y, re, f64(dloss), ignore)
    # p's own error (fp32 logits, exponential): relative 2^-20 of the row's size
    slack = 1.0 + 2.0 ** -10 * size[:, None]
    live = (y != ignore)[:, None]
    Xm = np.where(live, np.nan_to_num(X), 0.0)
    p = np.abs(dl) + np.where(live, 2.0 ** -11 * size[:, None] * np.abs(f64(dloss))[:, None] * (np.abs(dl) > 0) * np.abs(dl), 0)
    within(dx, dl @ W, (p * slack) @ np.abs(W))
    within(dw, dl.T @ Xm, (p * slack).T @ np.abs(Xm))
    assert np.all(f64(dx)[y == ignore] == 0)


@pytest.mark.parametrize("t,d,v,ld", CE_SHAPES)
def test_cross_entropy(zopt, t, d, v, ld):
    x, w, target, dloss = ce_case(t + d + v, t, d, v, ld)
    got = run_ce(zopt, x, w, target, dloss, ld_out=d + 3 if ld else None)
    check_ce(x, w, target, dloss, got)
    again = run_ce(zopt, x, w, target, dloss, ld_out=d + 3 if ld else None)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("t,d,v,ld", [(1, 1, 3, None), (1, 520, 20001, None), (2, 264, 5000, None), (1, 2049, 61, None),
                                      (2, 767, 2049, 771), (2, 100, 9, 104), (1, 250, 4863, 253)])
def test_cross_entropy_of_few_tokens(zopt, t, d, v, ld):
    """One and two tokens, rows of less and more than a warp's pieces, the last entry the target."""
    x, w, target, dloss = ce_case(40 + t + d + v, t, d, v, ld, ignored=0.0)
    target[0] = v - 1
    got = run_ce(zopt, x, w, target, dloss, ld_out=d + 3 if ld else None)
    check_ce(x, w, target, dloss, got)
    again = run_ce(zopt, x, w, target, dloss, ld_out=d + 3 if ld else None)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    if t == 2:  # the other row's overflow, and its being ignored, leave this one as it is
        x2, y2 = x.clone(), target.clone()
        x2[1] = float("inf")
        loss, lse = run_ce(zopt, x2, w, target, dloss)[:2]
        assert torch.equal(loss[0], got[0][0]) and torch.equal(lse[0], got[1][0]) and torch.isnan(loss[1])
        y2[1] = -100
        loss, lse = run_ce(zopt, x2, w, y2, dloss)[:2]
        assert torch.equal(loss[0], got[0][0]) and torch.equal(lse[0], got[1][0]) and loss[1] == 0 and lse[1] == 0


@pytest.mark.parametrize("t", [1, 2])
def test_cross_entropy_of_few_tokens_large_and_infinite_logits(zopt, t):
    """Logits of +-2e4, and weights of the lowest value and minus infinity: entries that take no part."""
    gen = torch.Generator(device="cuda").manual_seed(12 + t)
    x, w = rows(gen, t, 64, 40.0).abs(), rows(gen, 700, 64, 40.0)
    w[5], w[699] = float("-inf"), torch.finfo(torch.bfloat16).min
    target = torch.randint(6, 699, (t,), generator=gen, device="cuda")
    loss, lse = torch.empty(t, device="cuda"), torch.empty(t, device="cuda")
    zopt.linear_ce_forward(x, w, target, loss, lse, zopt.new_linear_ce_workspace(x, w, backward=False))
    keep = [v for v in range(700) if v not in (5, 699)]
    shifted = target.cpu().numpy() - 1  # (entry 5 lies below every target)
    rl, re = lm.ce_forward(f64(x), f64(w)[keep], shifted)
    size = 1 + (np.abs(f64(x)) @ np.abs(f64(w)[keep]).T).max(axis=1)
    assert np.all(np.abs(f64(loss) - rl) <= 2.0 ** -20 * size + 2.0 ** -23 * np.abs(rl))
    assert np.all(np.abs(f64(lse) - re) <= 2.0 ** -20 * size + 2.0 ** -23 * np.abs(re))


def test_cross_entropy_outputs_end_inside_a_16_byte_piece(zopt):
    """Rows whose distance the TMA could move but whose width it could not end at."""
    x, w, target, dloss = ce_case(5, 70, 44, 300)
    check_ce(x, w, target, dloss, run_ce(zopt, x, w, target, dloss, ld_out=64))


def test_cross_entropy_of_several_pieces(zopt):
    """Tokens times vocabulary beyond one piece: dx is summed over pieces, in a ragged last one too."""
    x, w, target, dloss = ce_case(6, 5000, 64, 30001)
    got = run_ce(zopt, x, w, target, dloss)
    X, W, y = x.double(), w.double(), target
    l = X @ W.T
    lse = torch.logsumexp(l, 1)
    live = y != -100
    assert ((got[1].double() - lse).abs()[live] <= 2.0 ** -20 * (1 + (X.abs() @ W.abs().T).amax(1))[live]).all()
    dl = torch.exp(l - got[1].double()[:, None])
    dl[torch.arange(len(y), device="cuda")[live], y[live]] -= 1
    dl = torch.where(live[:, None], dl * dloss.double()[:, None], 0.0)
    within(got[2], f64(dl @ W), f64(dl.abs() @ W.abs()))
    within(got[3], f64(dl.T @ X), f64(dl.abs().T @ X.abs()))


def test_cross_entropy_masked_rows_take_no_part(zopt):
    x, w, target, dloss = ce_case(7, 200, 64, 500)
    target[10:20] = -100
    clean = run_ce(zopt, x, w, target, dloss)
    x2, dloss2 = x.clone(), dloss.clone()
    x2[10:13] = float("nan")
    x2[13:16] = float("inf")
    x2[16] = torch.finfo(torch.bfloat16).min
    dloss2[10:20] = float("nan")
    got = run_ce(zopt, x2, w, target, dloss2)
    assert all(torch.equal(a, b) for a, b in zip(clean, got))
    check_ce(x, w, target, dloss, got)


@pytest.mark.parametrize("ignore", [-100, 0, 7])
def test_cross_entropy_every_row_ignored(zopt, ignore):
    x, w, target, dloss = ce_case(8, 40, 32, 100)
    target.fill_(ignore)
    loss, lse, dx, dw = run_ce(zopt, x, w, target, dloss, ignore=ignore)
    for a in (loss, lse, dx, dw):
        assert torch.all(a == 0)


def test_cross_entropy_large_and_equal_logits(zopt):
    """Logits of +-2e4 (nothing may overflow) and rows of equal ones."""
    gen = torch.Generator(device="cuda").manual_seed(9)
    x, w = rows(gen, 50, 64, 40.0), rows(gen, 700, 64, 40.0)
    x[7] = 0
    target = torch.randint(0, 700, (50,), generator=gen, device="cuda")
    loss, lse, dx, dw = run_ce(zopt, x, w, target, torch.ones(50, device="cuda"))
    rl, re = lm.ce_forward(f64(x), f64(w), target.cpu().numpy())
    size = 1 + (np.abs(f64(x)) @ np.abs(f64(w)).T).max(axis=1)
    assert np.all(np.abs(f64(loss) - rl) <= 2.0 ** -20 * size + 2.0 ** -23 * np.abs(rl))
    assert abs(float(lse[7]) - np.log(700)) < 1e-5
    assert torch.isfinite(dx).all() and torch.isfinite(dw).all()


def test_cross_entropy_invalid_targets_poison(zopt):
    x, w, target, dloss = ce_case(10, 30, 32, 100, ignored=0.0)
    for bad in (100, -1, 1 << 40):
        y = target.clone()
        y[3] = bad
        loss, lse, dx, dw = run_ce(zopt, x, w, y, dloss)
        assert torch.isnan(loss[3]) and torch.isfinite(torch.cat((loss[:3], loss[4:]))).all()
        assert torch.isnan(dx[3]).all() and torch.isfinite(dx[:3]).all() and torch.isnan(dw).any()


def test_cross_entropy_non_finite_rows_stay_their_own(zopt):
    x, w, target, dloss = ce_case(11, 30, 32, 100, ignored=0.0)
    x[5, 3] = float("nan")
    loss, lse, dx, dw = run_ce(zopt, x, w, target, dloss)
    assert torch.isnan(loss[5]) and torch.isnan(dx[5]).all()
    keep = [i for i in range(30) if i != 5]
    assert torch.isfinite(loss[keep]).all() and torch.isfinite(dx[keep]).all()


@pytest.mark.parametrize("scale", [1e-30, 1.0, 1e30])
def test_cross_entropy_gradient_scales_with_dloss(zopt, scale):
    x, w, target, dloss = ce_case(12, 60, 64, 300)
    a = run_ce(zopt, x, w, target, dloss)
    b = run_ce(zopt, x, w, target, dloss * 2.0 ** round(np.log2(scale)))
    f = 2.0 ** round(np.log2(scale))
    assert torch.equal(a[2].double() * f, b[2].double()) and torch.equal(a[3].double() * f, b[3].double())


def test_cross_entropy_gradient_against_differences(zopt):
    """dw and dx along random directions against central differences of the loss. Entries on a grid
    of 2^-6 move by one step and stay bf16 values; the loss is exact to about 1e-6, its third
    differences enter as step^2 = 2.4e-4 of the gradient's own size."""
    gen = torch.Generator(device="cuda").manual_seed(13)
    t, d, v, step = 64, 32, 200, 2.0 ** -6
    grid = lambda n: (torch.randint(-60, 61, (n, d), generator=gen, device="cuda").float() * step).bfloat16()  # noqa: E731
    x, w = grid(t), grid(v)
    target = torch.randint(0, v, (t,), generator=gen, device="cuda")
    _, _, dx, dw = run_ce(zopt, x, w, target, torch.ones(t, device="cuda"))
    total = lambda x, w: float(run_ce(zopt, x, w, target, torch.ones(t, device="cuda"))[0].double().sum())  # noqa: E731
    for which in range(2):
        u = torch.randint(-1, 2, ((t, v)[which], d), generator=gen, device="cuda").float()
        move = lambda s: total(*((x + s * step * u).bfloat16() if which == 0 else x,  # noqa: E731
                                 (w + s * step * u).bfloat16() if which == 1 else w))
        diff = (move(1) - move(-1)) / (2 * step)
        along = float(((dx, dw)[which].double() * u.double()).sum())
        size = float((dx, dw)[which].double().norm() * u.double().norm())
        assert abs(diff - along) <= 5e-3 * size + 1e-6 * t / step


def test_cross_entropy_one_gradient_alone(zopt):
    Z = zopt
    x, w, target, dloss = ce_case(14, 100, 64, 500)
    loss, lse, dx, dw = run_ce(Z, x, w, target, dloss)
    ws = Z.new_linear_ce_workspace(x, w)
    dx1, dw1 = torch.empty_like(dx), torch.empty_like(dw)
    Z.linear_ce_backward(x, w, target, lse, dloss, dx1, None, ws)
    Z.linear_ce_backward(x, w, target, lse, dloss, None, dw1, ws)
    torch.cuda.synchronize()
    dl = lm.ce_dlogits(f64(x), f64(w), target.cpu().numpy(), f64(lse), f64(dloss))
    within(dx1, dl @ f64(w), np.abs(dl) @ np.abs(f64(w)))
    within(dw1, dl.T @ f64(x), np.abs(dl).T @ np.abs(f64(x)))


def test_cross_entropy_no_tokens(zopt):
    Z = zopt
    x, w = torch.empty(0, 16, dtype=torch.bfloat16, device="cuda"), torch.ones(9, 16, dtype=torch.bfloat16, device="cuda")
    e, y = torch.empty(0, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda")
    ws = Z.new_linear_ce_workspace(x, w)
    dw = torch.ones_like(w)
    Z.linear_ce_forward(x, w, y, e, e, ws)
    Z.linear_ce_backward(x, w, y, e, e, torch.empty_like(x), dw, ws)
    torch.cuda.synchronize()
    assert torch.all(dw == 0)


# --------------------------------------------------------------------------- feed-forward block

FFN_SHAPES = [  # tokens, dim, hidden, row distances beyond the rows (None: contiguous)
    (1, 8, 8, None), (1, 256, 768, None), (3, 64, 128, None), (65, 40, 136, None), (130, 72, 200, 8),
    (257, 128, 384, None), (70, 50, 100, None), (64, 33, 97, None), (100, 96, 131, 3), (300, 264, 520, None),
    (1023, 256, 768, None),
]


def ffn_case(seed, t, d, f, pad=None):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    ld = (lambda n: None) if pad is None else (lambda n: n + pad)
    x, dy = rows(gen, t, d, ld=ld(d)), rows(gen, t, d, 0.1, ld=ld(d))
    wgu, wd = rows(gen, d, 2 * f, d ** -0.5, ld=ld(2 * f)), rows(gen, f, d, f ** -0.5, ld=ld(d))
    return x, dy, wgu, wd


def run_ffn(Z, x, dy, wgu, wd, act, keep, pad=None):
    t, d, f = x.shape[0], x.shape[1], wd.shape[0]
    pad = pad or 0
    x8 = Z.new_act8(t, d) if keep == "e4m3" else None
    kept = Z.new_act8(t, 2 * f, parts=2) if keep == "e4m3" else frame_of(t, 2 * f, 2 * f + pad)
    ws = Z.new_ffn_workspace(x if x8 is None else x8, wgu, wd, dy=dy)
    ws.fill_(255)
    outs = {"y": frame_of(t, d, d + pad), "dx": frame_of(t, d, d + pad), "dw_gate_up": frame_of(d, 2 * f, 2 * f + pad),
            "dw_down": frame_of(f, d, d + pad)}
    k = kept if x8 is not None else kept[1]
    Z.ffn_forward(x, wgu, wd, outs["y"][1], Z.new_ffn_workspace(x, wgu, wd, backward=False).fill_(255), kept=k, act=act)
    if x8 is not None:
        Z.act_pack(x, x8)
    Z.ffn_backward(dy, x if x8 is None else x8, k, wgu, wd, outs["dx"][1], outs["dw_gate_up"][1], outs["dw_down"][1],
                   ws, act=act)
    torch.cuda.synchronize()
    assert Z.take_device_error() == 0
    for whole, v in outs.values():
        assert untouched(whole, *v.shape)
    if x8 is None:
        assert untouched(kept[0], t, 2 * f)
    return {n: v for n, (_, v) in outs.items()}, k, x8


def check_ffn(x, dy, wgu, wd, act, got, kept, x8):
    X, DY, G, D, f = f64(x), f64(dy), f64(wgu), f64(wd), wd.shape[0]
    y, gu, h = lm.ffn_forward(X, G, D, act)
    sg = np.abs(X) @ np.abs(G)
    # h's error before its rounding: the fp32 sums of g and u (2^-16 of sum |x||w| each, |a'| < 1.2)
    hs = np.abs(h) + 2.0 ** -7 * (sg[:, :f] * np.abs(gu[:, f:]) * 1.2 + np.abs(gu[:, :f]) * sg[:, f:])
    within(got["y"], y, hs @ np.abs(D))
    if x8 is None:
        within(kept, gu, 2.0 ** -4 * sg)
        K, XK = f64(kept), X
    else:
        q, scale = kept.q.cpu().numpy(), kept.scale.cpu().numpy()
        K = lm.act8_unpack(q, scale, 2)
        nb = -(-f // 128)
        s = 2.0 ** (scale.reshape(len(X), 2, nb).astype(np.float64) - 127)
        top = np.stack([[np.abs(gu[:, p * f + 128 * b:p * f + min(128 * b + 128, f)]).max(axis=1) for b in range(nb)]
                        for p in range(2)]).transpose(2, 0, 1)
        assert np.all(top <= 448 * s * (1 + 2.0 ** -12)) and np.all((top >= 224 * s * (1 - 2.0 ** -12)) | (s <= 2.0 ** -126))
        s = np.repeat(s, 128, axis=2)[:, :, :f].reshape(len(X), 2 * f)
        assert np.all(np.abs(K - gu) <= np.maximum(2.0 ** -4 * np.abs(gu), 2.0 ** -10 * s) + 2.0 ** -16 * sg)
        xq, xs = lm.act8_pack(X)
        assert np.array_equal(x8.q.cpu().numpy(), xq) and np.array_equal(x8.scale.cpu().numpy().reshape(xs.shape), xs)
        XK = lm.act8_unpack(xq, xs)
    dx, dwgu, dwd = lm.ffn_backward(DY, XK, K, G, D, act)
    dgu, h, dh = lm.ffn_dgu(DY, K, D, act)
    # dg, du before their rounding: dh's fp32 sums (2^-16 of sum |dy||w|), the activation's 2^-20
    sdh = 2.0 ** -7 * (np.abs(DY) @ np.abs(D).T) + 2.0 ** -10 * np.abs(dh)
    gs = np.abs(dgu) + np.concatenate((sdh * np.abs(K[:, f:]) * 1.2, sdh * np.abs(K[:, :f])), axis=1)
    within(got["dx"], dx, gs @ np.abs(G).T)
    within(got["dw_gate_up"], dwgu, np.abs(XK).T @ gs)
    within(got["dw_down"], dwd, (np.abs(h) * (1 + 2.0 ** -10)).T @ np.abs(DY))


@pytest.mark.parametrize("keep", ["bf16", "e4m3"])
@pytest.mark.parametrize("t,d,f,pad", FFN_SHAPES)
def test_ffn(zopt, t, d, f, pad, keep):
    act = "gelu" if (t + d) % 2 else "silu"
    args = ffn_case(t + d + f, t, d, f, pad)
    got, kept, x8 = run_ffn(zopt, *args, act, keep, pad)
    check_ffn(*args, act, got, kept, x8)
    again, _, _ = run_ffn(zopt, *args, act, keep, pad)
    assert all(torch.equal(got[n], again[n]) for n in got)


@pytest.mark.parametrize("t,d,f", [(1, 64, 256), (77, 100, 130), (300, 128, 512)])
def test_ffn_forward_keeps_nothing(zopt, t, d, f):
    x, dy, wgu, wd = ffn_case(t, t, d, f)
    kept = run_ffn(zopt, x, dy, wgu, wd, "silu", "bf16")[0]["y"]
    y = torch.empty(t, d, dtype=torch.bfloat16, device="cuda")
    zopt.ffn_forward(x, wgu, wd, y, zopt.new_ffn_workspace(x, wgu, wd, backward=False))
    torch.cuda.synchronize()
    assert torch.equal(y, kept)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_ffn_extreme_gates(zopt, act):
    """Gates of thousands, either sign: a and a' end at 0, z and 1, and no infinity meets a zero."""
    x, dy, wgu, wd = ffn_case(3, 40, 64, 96)
    wgu = wgu.clone()
    wgu[:, :96] *= 4000
    for keep in ("bf16", "e4m3"):
        got, kept, x8 = run_ffn(zopt, x, dy, wgu, wd, act, keep)
        for a in got.values():
            assert torch.isfinite(a).all()


@pytest.mark.parametrize("keep", ["bf16", "e4m3"])
def test_ffn_non_finite_rows_stay_their_own(zopt, keep):
    x, dy, wgu, wd = ffn_case(4, 40, 64, 96)
    x[3, 5] = float("inf")
    got, _, _ = run_ffn(zopt, x, dy, wgu, wd, "silu", keep)
    others = [i for i in range(40) if i != 3]
    assert not torch.isfinite(got["y"][3]).any() and torch.isfinite(got["y"][others]).all()
    assert not torch.isfinite(got["dx"][3]).any() and torch.isfinite(got["dx"][others]).all()
    assert not torch.isfinite(got["dw_gate_up"]).all()  # found_inf sees it


def test_ffn_gradient_against_differences(zopt):
    """ddown along a random direction against central differences of <dy, y>, which is linear in
    down: only y's bf16 rounding (2^-8 at most, each way) is left, as a random sum over tokens x dim."""
    gen = torch.Generator(device="cuda").manual_seed(15)
    t, d, f, step = 64, 32, 96, 2.0 ** -3
    x, dy, wgu, _ = ffn_case(15, t, d, f)
    wd = (torch.randint(-8, 9, (f, d), generator=gen, device="cuda").float() * step).bfloat16()
    u = torch.randint(-1, 2, (f, d), generator=gen, device="cuda").float()
    got, _, _ = run_ffn(zopt, x, dy, wgu, wd, "silu", "bf16")
    ys = [run_ffn(zopt, x, dy, wgu, (wd + s * step * u).bfloat16(), "silu", "bf16")[0]["y"].double() for s in (1, -1)]
    diff = float(((ys[0] - ys[1]) * dy.double()).sum()) / (2 * step)
    along = float((got["dw_down"].double() * u.double()).sum())
    noise = 2.0 ** -9 * float(torch.sqrt(((ys[0] ** 2 + ys[1] ** 2) * dy.double() ** 2).sum())) / (2 * step)
    rounding = 2.0 ** -8 * float(got["dw_down"].double().norm() * u.double().norm())
    assert abs(diff - along) <= 6 * noise + rounding


def test_ffn_no_tokens(zopt):
    Z = zopt
    e = torch.empty(0, 16, dtype=torch.bfloat16, device="cuda")
    wgu, wd = torch.ones(16, 48, dtype=torch.bfloat16, device="cuda"), torch.ones(24, 16, dtype=torch.bfloat16, device="cuda")
    dwgu, dwd = torch.ones_like(wgu), torch.ones_like(wd)
    ws = Z.new_ffn_workspace(e, wgu, wd)
    kept = torch.empty(0, 48, dtype=torch.bfloat16, device="cuda")
    Z.ffn_forward(e, wgu, wd, e, ws, kept=kept)
    Z.ffn_backward(e, e, kept, wgu, wd, e, dwgu, dwd, ws)
    torch.cuda.synchronize()
    assert torch.all(dwgu == 0) and torch.all(dwd == 0)


def test_operators_on_a_stream_of_their_own_and_in_a_graph(zopt):
    Z = zopt
    x, dy, wgu, wd = ffn_case(16, 200, 64, 256)
    ref, _, _ = run_ffn(Z, x, dy, wgu, wd, "silu", "e4m3")
    ce = ce_case(17, 200, 64, 700)
    rce = run_ce(Z, *ce)
    kept, x8 = Z.new_act8(200, 512, parts=2), Z.new_act8(200, 64)
    ws, wce = Z.new_ffn_workspace(x8, wgu, wd), Z.new_linear_ce_workspace(ce[0], ce[1])
    out = {n: torch.zeros_like(v) for n, v in ref.items()}
    oce = [torch.zeros_like(v) for v in rce]

    def step():
        Z.ffn_forward(x, wgu, wd, out["y"], ws, kept=kept)
        Z.act_pack(x, x8)
        Z.ffn_backward(dy, x8, kept, wgu, wd, out["dx"], out["dw_gate_up"], out["dw_down"], ws)
        Z.linear_ce_forward(ce[0], ce[1], ce[2], oce[0], oce[1], wce)
        Z.linear_ce_backward(ce[0], ce[1], ce[2], oce[1], ce[3], oce[2], oce[3], wce)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    assert all(torch.equal(out[n], ref[n]) for n in ref) and all(torch.equal(a, b) for a, b in zip(oce, rce))
    for v in list(out.values()) + oce:
        v.zero_()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(out[n], ref[n]) for n in ref) and all(torch.equal(a, b) for a, b in zip(oce, rce))


# --------------------------------------------------------------------------- 8-bit checkpoints

@pytest.mark.parametrize("t,cols,parts,ld", [(1, 1, 1, None), (1, 128, 1, None), (3, 130, 1, None), (5, 256, 2, None),
                                             (33, 260, 2, None), (7, 514, 2, 520), (100, 1000, 1, 1001),
                                             (257, 2048, 1, None), (64, 11264, 2, None), (1, 3, 1, 8)])
def test_act8(zopt, t, cols, parts, ld):
    Z = zopt
    gen = torch.Generator(device="cuda").manual_seed(t + cols)
    x = torch.randn(t, cols, generator=gen, device="cuda") * torch.exp(3 * torch.randn(t, 1, generator=gen, device="cuda"))
    x[torch.rand(t, cols, generator=gen, device="cuda") < 0.02] = 0
    x = x.bfloat16()
    x[0, 0] = float("nan")
    if t > 1:
        x[1, cols // 2] = float("-inf")
        x[2] = 0
        x[2, 0] = 2.0 ** -133  # the smallest bf16 value
    if ld:
        x = framed(x, ld)
    c = Z.new_act8(t, cols, parts)
    c.q.fill_(255), c.scale.fill_(255)
    Z.act_pack(x, c)
    whole, out = frame_of(t, cols, ld)
    Z.act_unpack(c, out)
    torch.cuda.synchronize()
    q, scale = lm.act8_pack(f64(x), parts)
    gq = c.q.cpu().numpy()
    nan = ~np.isfinite(f64(x))
    assert np.all((gq[nan] & 127) == 127) and np.array_equal(gq[~nan], q[~nan])
    assert np.array_equal(c.scale.cpu().numpy().reshape(scale.shape), scale)
    v = lm.act8_unpack(q, scale, parts)
    assert np.array_equal(f64(out)[~nan], v[~nan]) and np.isnan(f64(out)[nan]).all()
    assert untouched(whole, t, cols)


def test_act8_every_byte(zopt):
    """Unpacking every e4m3 byte on powers from the smallest to 2^120 is exact."""
    Z = zopt
    c = Z.new_act8(247, 256)
    c.q.copy_(torch.arange(256, dtype=torch.uint8, device="cuda").repeat(247, 1))
    c.scale.copy_(torch.arange(1, 248, dtype=torch.uint8, device="cuda").repeat_interleave(2))
    out = torch.empty(247, 256, dtype=torch.bfloat16, device="cuda")
    Z.act_unpack(c, out)
    torch.cuda.synchronize()
    ref = lm.act8_unpack(c.q.cpu().numpy(), c.scale.cpu().numpy())
    small = np.abs(ref) < 2.0 ** -124  # four significant bits no longer fit bf16's subnormals
    got = f64(out)
    big = np.abs(ref) >= 2.0 ** 128
    ok = ~small & ~big & ~np.isnan(ref)
    assert np.array_equal(got[ok], ref[ok]) and np.array_equal(np.isnan(got), np.isnan(ref))
    assert np.all(np.abs(got - ref)[small] <= 2.0 ** -134)
