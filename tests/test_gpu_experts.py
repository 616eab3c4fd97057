"""The experts' feed-forward block on the GPU (zopt_experts_forward, zopt_experts_backward) against the fp64
oracle.

Tolerances, fixed before the first run: bf16 results entry by entry within oracle.experts.block_bound,
dweight within dweight_bound, kept gate and up in bf16 within their rounding (2^-8) and 2^-14 of their
terms, in 8 bits within half a step (2^-4 of the value; below the format's smallest normal value 2^-17
of the block's largest); repeated calls bit for bit.
"""
import numpy as np
import pytest
import torch

from oracle import experts as OE
from oracle import lm

pytestmark = pytest.mark.gpu

# tokens, dim, hidden, experts, top_k, act, keep, padding tokens
CASES = [
    (1, 8, 8, 1, 1, "silu", "bf16", 0),
    (1, 64, 40, 5, 3, "gelu", "e4m3", 0),
    (3, 256, 96, 4, 2, "silu", "e4m3", 1),
    (17, 72, 136, 6, 4, "silu", "bf16", 3),
    (40, 33, 47, 3, 2, "gelu", "bf16", 0),
    (40, 100, 130, 3, 1, "silu", "e4m3", 5),
    (130, 128, 128, 2, 2, "silu", "bf16", 0),
    (300, 64, 200, 2, 1, "gelu", "e4m3", 7),
    (90, 264, 72, 16, 6, "silu", "bf16", 2),
    (700, 40, 24, 3, 2, "silu", "e4m3", 0),
    (64, 300, 520, 4, 2, "gelu", "bf16", 0),
    (25, 17, 1, 2, 1, "silu", "bf16", 0),
    (25, 1, 9, 2, 2, "silu", "bf16", 0),
]
SENTINEL = 776.0  # (a bf16 value)


def frame(shape, extra, dtype=torch.bfloat16):
    """A tensor whose rows lie `extra` elements apart more than they are long, and what surrounds it."""
    whole = torch.full((*shape[:-2], shape[-2] + (1 if extra else 0), shape[-1] + extra), SENTINEL, dtype=dtype, device="cuda")
    return whole, whole[..., :shape[-2], :shape[-1]]


def untouched(whole, inner):
    mask = torch.ones_like(whole, dtype=torch.bool)
    mask[..., :inner.shape[-2], :inner.shape[-1]] = False
    return bool((whole[mask] == SENTINEL).all())


def framed(a, extra):
    whole, inner = frame(a.shape, extra, a.dtype)
    inner.copy_(a)
    return inner


class Block:
    def __init__(self, t, d, f, e, k, act, keep, padding, extra=0, seed=0, x8=False):
        g = torch.Generator(device="cuda").manual_seed(seed + t + d + f)
        new = lambda *s, sigma=1.0: (torch.randn(*s, generator=g, device="cuda") * sigma).bfloat16()  # noqa: E731
        self.t, self.d, self.f, self.e, self.k, self.act, self.keep, self.extra = t, d, f, e, k, act, keep, extra
        self.x, self.dy = framed(new(t, d), extra), framed(new(t, d), extra)
        self.wgu, self.wd = framed(new(e, d, 2 * f, sigma=d ** -0.5), extra), framed(new(e, f, d, sigma=f ** -0.5), extra)
        liking = torch.rand(t, e, generator=g, device="cuda")
        liking[:, 0] += 0.4  # some have many more slots than others
        self.index = liking.topk(k, dim=1).indices.int()
        self.weight = torch.rand(t, k, generator=g, device="cuda")
        if t > 2 and k > 1:
            self.index[1, 0] = -1  # a slot without an expert beside one with
        if padding:
            self.index[t - padding:] = -1
        off = (self.index < 0).all(dim=1)
        self.x[off], self.dy[off] = float("nan"), float("inf")
        self.weight[self.index < 0] = float("nan")
        self.off = off
        self.x8 = x8

    def forward(self, Z, ws=None, stream=None):
        self.whole_y, self.y = frame((self.t, self.d), self.extra)
        if self.keep == "e4m3":
            self.kept = Z.new_act8(self.t * self.k, 2 * self.f, parts=2)
            self.kept.q.fill_(99)
            self.kept.scale.fill_(99)
        elif self.keep == "bf16":
            self.whole_kept, self.kept = frame((self.t * self.k, 2 * self.f), self.extra)
        else:
            self.kept = None
        if ws is None:
            ws = Z.new_experts_workspace(self.x, self.index, self.wgu, self.wd)
            ws.fill_(255)
        Z.experts_forward(self.x, self.index, self.weight, self.wgu, self.wd, self.y, ws, kept=self.kept, act=self.act, stream=stream)

    def backward(self, Z, ws=None):
        self.whole_dx, self.dx = frame((self.t, self.d), self.extra)
        self.whole_dwgu, self.dwgu = frame((self.e, self.d, 2 * self.f), self.extra)
        self.whole_dwd, self.dwd = frame((self.e, self.f, self.d), self.extra)
        self.dweight = torch.full((self.t, self.k), float("nan"), device="cuda")
        x = self.x
        if self.x8:
            x = Z.new_act8(self.t, self.d)
            Z.act_pack(torch.where(self.off[:, None], 0.0, self.x).contiguous(), x)
            x.q[self.off], x.scale.view(self.t, -1)[self.off] = 127, 254
            self.packed = x
        if ws is None:
            ws = Z.new_experts_workspace(x, self.index, self.wgu, self.wd)
            ws.fill_(255)
        Z.experts_backward(self.dy, x, self.index, self.weight, self.kept, self.wgu, self.wd, self.dx, self.dweight, self.dwgu,
                           self.dwd, ws, act=self.act)

    def results(self):
        return [a.clone() for a in (self.y, self.dx, self.dweight, self.dwgu, self.dwd)]

    def kept_values(self):
        if self.keep == "e4m3":
            return lm.act8_unpack(self.kept.q.cpu().numpy(), self.kept.scale.cpu().numpy(), 2)
        return f64(self.kept)

    def check(self, Z):
        torch.cuda.synchronize()
        assert Z.take_device_error() == 0
        assert untouched(self.whole_y, self.y) and untouched(self.whole_dx, self.dx)
        assert untouched(self.whole_dwgu, self.dwgu) and untouched(self.whole_dwd, self.dwd)
        index, weight = self.index.cpu().numpy(), np.nan_to_num(f64(self.weight))
        x, dy = np.nan_to_num(f64(self.x)), np.where(self.off.cpu().numpy()[:, None], 0.0, f64(self.dy))
        wgu, wd = f64(self.wgu), f64(self.wd)
        y, gu, size = OE.experts_forward(x, index, weight, wgu, wd, self.act)
        close(self.y, y, OE.block_bound(y, size))
        on = index.reshape(-1) >= 0
        kept = self.kept_values()
        terms = np.zeros_like(gu)
        for s in np.nonzero(on)[0]:
            terms[s] = np.abs(x[s // self.k]) @ np.abs(wgu[index.reshape(-1)[s]])
        if self.keep == "bf16":
            assert (np.abs(kept - gu)[on] <= (2.0 ** -8 * np.abs(gu) + 2.0 ** -14 * terms)[on]).all()
            assert (kept[~on] == SENTINEL).all() and untouched(self.whole_kept, self.kept)
        else:
            top = np.abs(gu).max(axis=1, keepdims=True)
            assert (np.abs(kept - gu)[on] <= (2.0 ** -4 * np.abs(gu) + 2.0 ** -17 * top + 2.0 ** -13 * terms)[on]).all()
            assert (self.kept.q.cpu().numpy()[~on] == 99).all() and (self.kept.scale.cpu().numpy().reshape(len(on), -1)[~on] == 99).all()
        if self.x8:
            x = np.nan_to_num(lm.act8_unpack(self.packed.q.cpu().numpy(), self.packed.scale.cpu().numpy()))
        ref = OE.experts_backward(dy, x, index, weight, np.where(on[:, None], kept, 0.0), wgu, wd, self.act)
        close(self.dx, ref["dx"][0], OE.block_bound(*ref["dx"]))
        close(self.dweight, ref["dweight"][0], OE.dweight_bound(ref["dweight"][1], self.d, self.f))
        close(self.dwgu, ref["dw_gate_up"][0], OE.block_bound(*ref["dw_gate_up"]))
        close(self.dwd, ref["dw_down"][0], OE.block_bound(*ref["dw_down"]))
        gone = self.off.cpu().numpy()
        assert (f64(self.y)[gone] == 0).all() and (f64(self.dx)[gone] == 0).all()
        assert (f64(self.dweight)[index < 0] == 0).all()
        for e in range(self.e):
            if not (index == e).any():
                assert (f64(self.dwgu[e]) == 0).all() and (f64(self.dwd[e]) == 0).all()


def f64(t):
    return t.detach().double().cpu().numpy()


def close(got, ref, bound):
    got = f64(got)
    assert np.isfinite(got).all()
    worst = float((np.abs(got - ref) / bound).max()) if got.size else 0.0
    assert worst <= 1.0, worst


@pytest.mark.parametrize("case", CASES)
def test_both_directions(zopt, case):
    b = Block(*case)
    b.forward(zopt)
    b.backward(zopt)
    b.check(zopt)
    first = b.results()
    b.forward(zopt)
    b.backward(zopt)
    assert all(torch.equal(x, y) for x, y in zip(first, b.results()))
    b.keep = "none"  # what is kept changes nothing of y
    b.forward(zopt)
    assert torch.equal(first[0], b.y)


@pytest.mark.parametrize("case,extra", [(CASES[3], 8), (CASES[3], 3), (CASES[4], 5), (CASES[5], 16), (CASES[6], 1), (CASES[9], 24)])
def test_row_distances_and_strides(zopt, case, extra):
    """Rows that the TMA can and cannot read in place, results inside wider rows, matrices with room between."""
    b = Block(*case, extra=extra, seed=1)
    b.forward(zopt)
    b.backward(zopt)
    b.check(zopt)


@pytest.mark.parametrize("case", [CASES[2], CASES[4], CASES[8], CASES[12]])
def test_x_as_a_checkpoint(zopt, case):
    b = Block(*case, x8=True, seed=2)
    b.forward(zopt)
    b.backward(zopt)
    b.check(zopt)


def test_an_expert_twice_and_experts_left_out(zopt):
    b = Block(50, 48, 64, 9, 3, "silu", "bf16", 0, seed=3)
    b.index[:] = torch.tensor([4, 7, 4], dtype=torch.int32, device="cuda")
    b.weight[:] = torch.rand(50, 3, device="cuda")
    b.x[:], b.dy[:] = torch.randn(50, 48, device="cuda"), torch.randn(50, 48, device="cuda")
    b.off[:] = False
    b.forward(zopt)
    b.backward(zopt)
    b.check(zopt)


@pytest.mark.parametrize("tokens", [4, 40])
def test_nobody_chose(zopt, tokens):
    b = Block(tokens, 48, 64, 4, 2, "silu", "e4m3", tokens, seed=4)
    b.forward(zopt)
    b.backward(zopt)
    b.check(zopt)


def test_no_tokens(zopt):
    x, index, weight = torch.empty(0, 16, dtype=torch.bfloat16, device="cuda"), torch.empty(0, 2, dtype=torch.int32, device="cuda"), torch.empty(0, 2, device="cuda")
    wgu, wd = torch.randn(3, 16, 24, device="cuda").bfloat16(), torch.randn(3, 12, 16, device="cuda").bfloat16()
    ws = zopt.new_experts_workspace(x, index, wgu, wd)
    zopt.experts_forward(x, index, weight, wgu, wd, torch.empty_like(x), ws)
    (whole_a, a), (whole_b, b) = frame((3, 16, 24), 5), frame((3, 12, 16), 5)
    zopt.experts_backward(x, x, index, weight, torch.empty(0, 24, dtype=torch.bfloat16, device="cuda"), wgu, wd, x.clone(), weight.clone(), a, b, ws)
    torch.cuda.synchronize()
    assert bool((a == 0).all()) and bool((b == 0).all()) and untouched(whole_a, a) and untouched(whole_b, b)


@pytest.mark.parametrize("tokens", [3, 60])
def test_an_index_out_of_range_poisons_its_token(zopt, tokens):
    b = Block(tokens, 40, 48, 4, 2, "silu", "bf16", 0, seed=5)
    b.forward(zopt)
    b.backward(zopt)
    good = b.results()
    b.index[2, 0], b.index[0, 1] = 4, -2
    b.forward(zopt)
    b.backward(zopt)
    torch.cuda.synchronize()
    for t in (0, 2):
        assert bool(torch.isnan(b.y[t]).all()) and bool(torch.isnan(b.dx[t]).all())
    assert torch.isnan(b.dweight[2, 0]) and torch.isnan(b.dweight[0, 1]) and torch.isfinite(b.dweight[2, 1])
    rest = [t for t in range(tokens) if t not in (0, 2)]
    assert torch.equal(b.y[rest], good[0][rest]) and torch.equal(b.dx[rest], good[1][rest])
    assert bool(torch.isfinite(b.dwgu.float()).all())


def test_one_experts_infinity_stays_its_own(zopt):
    """Weights of inf and NaN touch the tokens that chose their expert, and no neighbour's tile."""
    for d, f in ((72, 40), (40, 72), (33, 47)):
        b = Block(200, d, f, 3, 1, "silu", "bf16", 0, seed=6)
        b.forward(zopt)
        b.backward(zopt)
        good = b.results()
        b.wgu[1], b.wd[1] = float("nan"), float("inf")
        b.forward(zopt)
        b.backward(zopt)
        torch.cuda.synchronize()
        others = (b.index[:, 0] != 1).nonzero()[:, 0]
        for got, want in zip((b.y, b.dx, b.dweight), good):
            assert torch.equal(got[others], want[others])
        for e in (0, 2):
            assert torch.equal(b.dwgu[e], good[3][e]) and torch.equal(b.dwd[e], good[4][e])
        assert bool(torch.isnan(b.dx[b.index[:, 0] == 1].float()).all())


def test_captured_and_replayed_with_other_choices(zopt):
    b = Block(150, 64, 96, 6, 2, "silu", "e4m3", 0, seed=7)
    ws = zopt.new_experts_workspace(b.x, b.index, b.wgu, b.wd)
    b.forward(zopt, ws)
    b.backward(zopt, ws)
    outs = (b.y, b.dx, b.dweight, b.dwgu, b.dwd)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        zopt.experts_forward(b.x, b.index, b.weight, b.wgu, b.wd, b.y, ws, kept=b.kept, act=b.act)
        zopt.experts_backward(b.dy, b.x, b.index, b.weight, b.kept, b.wgu, b.wd, b.dx, b.dweight, b.dwgu, b.dwd, ws, act=b.act)
    for skew in (0.0, 3.0):  # evenly, and nearly all to one expert
        liking = torch.rand(150, 6, device="cuda")
        liking[:, 2] += skew
        b.index.copy_(liking.topk(2, dim=1).indices.int())
        b.weight.copy_(torch.rand(150, 2, device="cuda"))
        b.off[:] = False
        g.replay()
        torch.cuda.synchronize()
        got = [a.clone() for a in outs]
        b.whole_y.fill_(SENTINEL)
        b.forward(zopt)
        b.backward(zopt)
        b.check(zopt)
        assert all(torch.equal(x, y) for x, y in zip(got, b.results()))


def test_two_streams_at_once(zopt):
    blocks = [Block(120, 64, 96, 6, 2, "silu", "bf16", 0, seed=8 + i) for i in range(2)]
    want = []
    for b in blocks:
        b.forward(zopt)
        torch.cuda.synchronize()
        want.append(b.y.clone())
    streams = [torch.cuda.Stream() for _ in blocks]
    ws = [zopt.new_experts_workspace(b.x, b.index, b.wgu, b.wd) for b in blocks]
    torch.cuda.synchronize()
    for _ in range(3):
        for b, s, w in zip(blocks, streams, ws):
            zopt.experts_forward(b.x, b.index, b.weight, b.wgu, b.wd, b.y, w, kept=b.kept, act=b.act, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(b.y, w) for b, w in zip(blocks, want))


def test_gradients_against_differences(zopt):
    """dweight and dx of sum(y dy) by central differences through the forward itself, in bf16: directions of
    many entries, whose differences stand far above the roundings."""
    b = Block(60, 64, 96, 4, 2, "silu", "bf16", 0, seed=10)
    b.index[:] = torch.rand(60, 4, device="cuda").topk(2, dim=1).indices.int()
    b.weight[:] = torch.rand(60, 2, device="cuda") + 0.5
    b.x[:], b.dy[:] = torch.randn(60, 64, device="cuda"), torch.randn(60, 64, device="cuda")
    b.off[:] = False
    b.forward(zopt)
    b.backward(zopt)
    torch.cuda.synchronize()
    dx, dweight = f64(b.dx), f64(b.dweight)

    def loss():
        b.forward(zopt)
        torch.cuda.synchronize()
        return float((f64(b.y) * f64(b.dy)).sum())

    step, w0 = 0.25, b.weight.clone()
    to = torch.sign(b.dweight)
    b.weight.copy_(w0 + step * to)
    up = loss()
    b.weight.copy_(w0 - step * to)
    down = loss()
    b.weight.copy_(w0)
    want = np.abs(dweight).sum()  # (the loss is linear in the weights)
    assert abs((up - down) / (2 * step) - want) <= 0.01 * want
    step, x0 = 2.0 ** -4, b.x.clone()
    to = torch.sign(b.dx)
    b.x.copy_((x0.float() + step * to.float()).bfloat16())
    xu, up = f64(b.x), loss()
    b.x.copy_((x0.float() - step * to.float()).bfloat16())
    xd, down = f64(b.x), loss()
    want = (dx * (xu - xd)).sum()
    assert abs(up - down - want) <= 0.03 * abs(want)


@pytest.mark.parametrize("keep", ["bf16", "e4m3"])
def test_many_tiles(zopt, keep):
    """Several row tiles for most experts and several units for every pair of CTAs, in norm against fp32 products
    (3.2e-3 for two roundings to bf16 beside the result's own, as the dense block's)."""
    t, d, f, e, k = 3000, 512, 640, 11, 3
    b = Block(t, d, f, e, k, "silu", keep, 100, seed=11)
    b.forward(zopt)
    b.backward(zopt)
    torch.cuda.synchronize()
    assert zopt.take_device_error() == 0
    kept = b.kept
    if keep == "e4m3":
        kept = torch.empty(t * k, 2 * f, dtype=torch.bfloat16, device="cuda")
        zopt.act_unpack(b.kept, kept)
    y, dx = torch.zeros(t, d, device="cuda", dtype=torch.float64), torch.zeros(t, d, device="cuda", dtype=torch.float64)
    flat = b.index.reshape(-1)

    def near(got, ref, limit=3.2e-3):
        err = float((got.double() - ref).norm() / ref.norm())
        assert err <= limit, err

    silu = torch.nn.functional.silu
    for i in range(e):
        slots = (flat == i).nonzero()[:, 0]
        rows, w = slots // k, b.weight.reshape(-1)[slots][:, None].double()
        xi, dyi, up, down = b.x[rows].double(), b.dy[rows].double(), b.wgu[i].double(), b.wd[i].double()
        z = xi @ up
        y.index_add_(0, rows, w * ((silu(z[:, :f]) * z[:, f:]) @ down))
        q = kept[slots].double()
        near(q, z, 1.7e-3 * 1.2 if keep == "bf16" else 0.03)
        g, u = q[:, :f].requires_grad_(), q[:, f:]
        a = silu(g)
        da, = torch.autograd.grad(a.sum(), g)
        a = a.detach()
        dh = dyi @ down.t()
        assert torch.allclose(b.dweight.reshape(-1)[slots].double(), (dh * a * u).sum(1), rtol=1e-4, atol=1e-3)
        dgu = w * torch.cat((dh * u * da, dh * a), 1)
        dx.index_add_(0, rows, dgu @ up.t())
        near(b.dwgu[i], xi.t() @ dgu)
        near(b.dwd[i], (w * a * u).t() @ dyi)
    near(b.y, y)
    near(b.dx, dx)


def test_routed_step(zopt):
    """Routing, the experts forward and backward and the routing's backward in a row, as a training step runs them."""
    t, d, f, e, k = 200, 64, 96, 8, 2
    b = Block(t, d, f, e, k, "silu", "e4m3", 0, seed=12)
    b.x[:], b.dy[:] = torch.randn(t, d, device="cuda"), torch.randn(t, d, device="cuda")
    b.off[:] = False
    logits = torch.randn(t, e, device="cuda")
    live = torch.arange(t, device="cuda") < t - 9
    counts = torch.empty(e, dtype=torch.int32, device="cuda")
    zopt.route_forward(logits, b.index, b.weight, counts, live=live)
    b.off = ~live
    b.forward(zopt)
    b.backward(zopt)
    b.check(zopt)
    dl = torch.empty_like(logits)
    zopt.route_backward(logits, b.index, b.weight, b.dweight, dl)
    index, weight, n = OE.route_forward(f64(logits), k, live=live.cpu().numpy())
    assert np.array_equal(index, b.index.cpu().numpy()) and np.array_equal(n, counts.cpu().numpy())
    ref = OE.route_backward(f64(logits), index, f64(b.dweight))
    assert np.allclose(f64(dl), ref, rtol=1e-4, atol=1e-4 * np.abs(ref).max())


def test_refusals(zopt):
    b = Block(20, 16, 24, 4, 2, "silu", "bf16", 0)
    b.forward(zopt)
    ws = zopt.new_experts_workspace(b.x, b.index, b.wgu, b.wd)
    args = lambda **kw: {**dict(x=b.x, index=b.index, weight=b.weight, w_gate_up=b.wgu, w_down=b.wd, y=b.y, ws=ws), **kw}  # noqa: E731
    with pytest.raises(ValueError, match="index"):
        zopt.experts_forward(**args(index=b.index.long()))
    with pytest.raises(ValueError, match="weight"):
        zopt.experts_forward(**args(weight=b.weight.bfloat16()))
    with pytest.raises(ValueError, match="kept"):
        zopt.experts_forward(**args(kept=b.kept[1:]))
    with pytest.raises(ValueError, match="kept"):
        zopt.experts_forward(**args(kept=b.kept.float()))
    with pytest.raises(zopt.ZoptError, match="dtype"):
        zopt.experts_forward(**args(w_down=b.wd.float()))
    with pytest.raises(zopt.ZoptError, match="dtype"):
        zopt.experts_forward(**args(y=b.y.half()))
    with pytest.raises(zopt.ZoptError, match="act"):
        zopt.experts_forward(**args(act="relu"))
    with pytest.raises(zopt.ZoptError, match="workspace"):
        zopt.experts_forward(**args(ws=ws[:1024]))
    with pytest.raises(zopt.ZoptError, match="kept"):
        zopt.experts_backward(b.dy, b.x, b.index, b.weight, None, b.wgu, b.wd, b.x.clone(), b.weight.clone(), b.wgu.clone(), b.wd.clone(), ws)


@pytest.mark.parametrize("case", [(1, 264, 300, 6, 6, "silu", "e4m3", 0), (2, 2056, 40, 5, 3, "gelu", "bf16", 0), (5, 33, 129, 7, 3, "silu", "e4m3", 1),
                                  (8, 100, 47, 3, 2, "gelu", "bf16", 2), (16, 72, 264, 4, 1, "silu", "bf16", 3), (4, 520, 128, 9, 4, "silu", "e4m3", 0)])
@pytest.mark.parametrize("extra", [0, 3])
def test_a_few_slots(zopt, case, extra):
    """At most 16 slots: sums of weight rows, one slot's after another's."""
    b = Block(*case, extra=extra, seed=13)
    b.forward(zopt)
    b.backward(zopt)
    b.check(zopt)
    y = b.y.clone()
    b.forward(zopt)
    assert torch.equal(y, b.y)


@pytest.mark.parametrize("case", [(70, 64, 40, 3, 2, "silu", "e4m3", 4), (70, 64, 44, 3, 2, "gelu", "bf16", 4), (300, 33, 171, 5, 3, "silu", "e4m3", 9),
                                  (200, 96, 266, 1, 1, "silu", "bf16", 0), (333, 40, 24, 2, 2, "gelu", "e4m3", 0)])
def test_kept_rows_that_start_anywhere(zopt, case):
    """Widths whose kept rows, or their ups, do not start on 16 bytes, and tiles of 128 rows with tails of few."""
    b = Block(*case, seed=14)
    b.forward(zopt)
    b.backward(zopt)
    b.check(zopt)


@pytest.mark.parametrize("case", [(100, 16, 8, 1024, 4, "silu", "bf16", 0), (70, 24, 16, 40, 32, "gelu", "e4m3", 6), (9, 8, 16, 33, 32, "silu", "bf16", 0),
                                  (2100, 8, 8, 2, 1, "silu", "bf16", 0)])
def test_many_experts_and_many_slots(zopt, case):
    b = Block(*case, seed=15)
    b.forward(zopt)
    b.backward(zopt)
    b.check(zopt)


def test_one_expert_is_the_dense_block(zopt):
    """Every token to the one expert with weight 1: the dense block's bits but for its y (whose part carries 12 bits)."""
    b = Block(300, 72, 136, 1, 1, "silu", "bf16", 0, seed=16)
    b.weight.fill_(1.0)
    b.forward(zopt)
    b.backward(zopt)
    y, kept, dx = torch.empty_like(b.y), torch.empty_like(b.kept), torch.empty_like(b.dx)
    dwgu, dwd = torch.empty_like(b.wgu[0]), torch.empty_like(b.wd[0])
    ws = zopt.new_ffn_workspace(b.x, b.wgu[0], b.wd[0])
    zopt.ffn_forward(b.x, b.wgu[0], b.wd[0], y, ws, kept=kept)
    zopt.ffn_backward(b.dy, b.x, kept, b.wgu[0], b.wd[0], dx, dwgu, dwd, ws)
    torch.cuda.synchronize()
    assert torch.equal(kept, b.kept) and torch.equal(dwgu, b.dwgu[0]) and torch.equal(dwd, b.dwd[0])
    for got, want in ((b.y, y), (b.dx, dx)):
        assert bool(((got.float() - want.float()).abs() <= 2.0 ** -7 * want.float().abs() + 1e-6).all())


def test_rows_past_two_to_the_31(zopt):
    """Kept gate and up of 2.3e9 bytes, slots and rows in the hundred thousands: tokens from both ends against the
    formula."""
    t, d, f, e, k = 270000, 16, 2144, 3, 2
    g = torch.Generator(device="cuda").manual_seed(17)
    new = lambda *s, sigma=1.0: (torch.randn(*s, generator=g, device="cuda") * sigma).bfloat16()  # noqa: E731
    x, dy, wgu, wd = new(t, d), new(t, d), new(e, d, 2 * f, sigma=0.25), new(e, f, d, sigma=0.02)
    index = torch.rand(t, e, generator=g, device="cuda").topk(k, dim=1).indices.int()
    weight = torch.rand(t, k, generator=g, device="cuda")
    kept = zopt.new_act8(t * k, 2 * f, parts=2)
    assert kept.q.numel() > 1 << 31
    ws = zopt.new_experts_workspace(x, index, wgu, wd)
    y, dx, dweight, dwgu, dwd = torch.empty_like(x), torch.empty_like(x), torch.empty_like(weight), torch.empty_like(wgu), torch.empty_like(wd)
    zopt.experts_forward(x, index, weight, wgu, wd, y, ws, kept=kept)
    zopt.experts_backward(dy, x, index, weight, kept, wgu, wd, dx, dweight, dwgu, dwd, ws)
    torch.cuda.synchronize()
    assert zopt.take_device_error() == 0
    pick = torch.cat((torch.arange(40), torch.arange(t - 40, t))).cuda()
    n = lambda a: a[pick].cpu()  # noqa: E731
    W, D = f64(wgu), f64(wd)
    want, gu, size = OE.experts_forward(f64(n(x)), n(index).numpy(), f64(n(weight)), W, D, "silu")
    close(n(y), want, OE.block_bound(want, size))
    rows = (pick[:, None] * k + torch.arange(k, device="cuda")).flatten()
    nb = lm.BLOCK
    scale = kept.scale.view(t * k, -1)[rows].cpu().numpy()
    values = lm.act8_unpack(kept.q[rows].cpu().numpy(), scale, 2)
    top = np.abs(gu).max(axis=1, keepdims=True)
    terms = np.abs(f64(n(x))).sum(1).repeat(k)[:, None] * np.abs(W).max()
    assert (np.abs(values - gu) <= 2.0 ** -4 * np.abs(gu) + 2.0 ** -17 * top + 2.0 ** -13 * terms).all() and nb == 128
    ref = OE.experts_backward(f64(n(dy)), f64(n(x)), n(index).numpy(), f64(n(weight)), values, W, D, "silu")
    close(n(dx), ref["dx"][0], OE.block_bound(*ref["dx"]))
    close(n(dweight), ref["dweight"][0], OE.dweight_bound(ref["dweight"][1], d, f))
    # the gradients of the weights, in norm, from sums over pieces of the tokens
    dgu_ref, dwd_ref = torch.zeros(e, d, 2 * f, dtype=torch.float64, device="cuda"), torch.zeros(e, f, d, dtype=torch.float64, device="cuda")
    for c in range(0, t, 27000):
        s = slice(c * k, (c + 27000) * k)
        piece = zopt.Act8(kept.q[s], kept.scale.view(t * k, -1)[s].reshape(-1), 2)
        v = torch.empty(27000 * k, 2 * f, dtype=torch.bfloat16, device="cuda")
        zopt.act_unpack(piece, v)
        flat = index[c:c + 27000].reshape(-1)
        for i in range(e):
            slots = (flat == i).nonzero()[:, 0]
            r, w = c + slots // k, weight.reshape(-1)[c * k + slots][:, None]
            gg, u = v[slots, :f].float(), v[slots, f:].float()
            sg = torch.sigmoid(gg)
            a, da = gg * sg, sg * (1 + gg * (1 - sg))
            dh = dy[r].float() @ wd[i].float().t()
            dgu_ref[i] += (x[r].float().t() @ (w * torch.cat((dh * u * da, dh * a), 1))).double()
            dwd_ref[i] += ((w * a * u).t() @ dy[r].float()).double()
    for got, want in ((dwgu, dgu_ref), (dwd, dwd_ref)):
        assert float((got.double() - want).norm()) <= 3.2e-3 * float(want.norm())


@pytest.mark.parametrize("tokens", [1, 3, 17])
@pytest.mark.parametrize("extra", [0, 8, 5])
def test_wide_gradients_of_experts_without_rows(zopt, tokens, extra):
    """Parts of a gradient that are whole, end inside the matrix's rows or columns, or start anywhere."""
    b = Block(tokens, 300, 200, 12, 2, "silu", "bf16", 0, extra=extra, seed=19)
    b.index[:, 1] = b.index[:, 0]  # (half the experts or more have no rows)
    b.forward(zopt)
    b.backward(zopt)
    b.check(zopt)
    assert len(set(b.index.flatten().tolist())) < 12


@pytest.mark.parametrize("case", [(60, 40, 24, 4, 2, "silu", "bf16", 3), (4, 40, 24, 4, 2, "gelu", "e4m3", 0)])
@pytest.mark.parametrize("gap", [8, 3])
def test_matrices_any_distance_apart(zopt, case, gap):
    """Strides that are no multiple of the rows' distance, of the weights and of their gradients."""
    b = Block(*case, seed=18)

    def apart(a):
        n, r, c = a.shape
        flat = torch.full((n * (r * c + gap) + 8,), SENTINEL, dtype=a.dtype, device="cuda")
        v = flat.as_strided((n, r, c), (r * c + gap, c, 1))
        v.copy_(a)
        return flat, v

    b.wgu, b.wd = apart(b.wgu)[1], apart(b.wd)[1]
    b.forward(zopt)
    b.backward(zopt)
    b.check(zopt)
    (flat_a, a), (flat_b, c) = apart(torch.zeros_like(b.dwgu)), apart(torch.zeros_like(b.dwd))
    ws = zopt.new_experts_workspace(b.x, b.index, b.wgu, b.wd)
    zopt.experts_backward(b.dy, b.x, b.index, b.weight, b.kept, b.wgu, b.wd, b.dx, b.dweight, a, c, ws, act=b.act)
    torch.cuda.synchronize()
    assert torch.equal(a, b.dwgu) and torch.equal(c, b.dwd)
    for flat, v in ((flat_a, a), (flat_b, c)):
        keep = torch.ones_like(flat, dtype=torch.bool)
        keep.as_strided(v.shape, v.stride()).fill_(False)
        assert bool((flat[keep] == SENTINEL).all())
