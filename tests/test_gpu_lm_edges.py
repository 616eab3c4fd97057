"""The training operators at the narrowest widths, and on matrices whose rows lie further than 2^31 elements
from the first one's. Tolerances: those of test_gpu_lm.py; results of far rows are those of near ones bit
for bit."""
import pytest
import torch

from tests.test_gpu_lm import ce_case, check_ce, check_ffn, ffn_case, run_ce, run_ffn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t,d,v", [(5, 1, 3), (300, 1, 1), (3, 2, 1), (257, 3, 2), (4, 7, 129), (1, 1, 1)])
def test_cross_entropy_narrow(zopt, t, d, v):
    x, w, target, dloss = ce_case(t + d + v, t, d, v)
    check_ce(x, w, target, dloss, run_ce(zopt, x, w, target, dloss))


@pytest.mark.parametrize("keep", ["bf16", "e4m3"])
@pytest.mark.parametrize("t,d,f", [(5, 1, 1), (300, 1, 3), (7, 2, 1), (257, 9, 1), (6, 1, 129), (1, 1, 1)])
def test_block_narrow(zopt, t, d, f, keep):
    args = ffn_case(t + d + f, t, d, f)
    got, kept, x8 = run_ffn(zopt, *args, "silu", keep)
    check_ffn(*args, "silu", got, kept, x8)


def far(a):
    """a's rows at distances that put the last beyond 2^31 elements (4 GiB of bf16) from the first."""
    ld = ((1 << 31) // (a.shape[0] - 1) // 8 + 1) * 8
    v = torch.empty(((a.shape[0] - 1) * ld + a.shape[1],), dtype=a.dtype, device="cuda").as_strided(a.shape, (ld, 1))
    assert v.stride(0) * (a.shape[0] - 1) >= 1 << 31
    return v.copy_(a)


@pytest.mark.parametrize("t", [2, 40])
def test_cross_entropy_of_far_rows(zopt, t):
    x, w, target, dloss = ce_case(3, t, 72, 300, ignored=0.1)
    near = run_ce(zopt, x, w, target, dloss)
    loss, lse = torch.empty(t, device="cuda"), torch.empty(t, device="cuda")
    fx, fw = far(x), far(w)
    dx, dw = far(torch.zeros_like(x)), far(torch.zeros_like(w))
    ws = zopt.new_linear_ce_workspace(fx, fw)
    zopt.linear_ce_forward(fx, fw, target, loss, lse, ws)
    zopt.linear_ce_backward(fx, fw, target, lse, dloss, dx, dw, ws)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(near, (loss, lse, dx, dw)))


@pytest.mark.parametrize("t", [2, 40])
def test_block_of_far_rows(zopt, t):
    x, dy, wgu, wd = ffn_case(5, t, 72, 200)
    near, kept, _ = run_ffn(zopt, x, dy, wgu, wd, "gelu", "bf16")
    for which in ("x dy", "wgu wd", "kept y", "dx dwgu dwd"):
        a = dict(x=x, dy=dy, wgu=wgu, wd=wd, kept=torch.zeros_like(kept), y=torch.zeros_like(x), dx=torch.zeros_like(x),
                 dwgu=torch.zeros_like(wgu), dwd=torch.zeros_like(wd))
        a.update({n: far(a[n]) for n in which.split()})
        ws = zopt.new_ffn_workspace(a["x"], a["wgu"], a["wd"], dy=a["dy"])
        zopt.ffn_forward(a["x"], a["wgu"], a["wd"], a["y"], ws, kept=a["kept"], act="gelu")
        zopt.ffn_backward(a["dy"], a["x"], a["kept"], a["wgu"], a["wd"], a["dx"], a["dwgu"], a["dwd"], ws, act="gelu")
        torch.cuda.synchronize()
        for n, ref in (("kept", kept), ("y", near["y"]), ("dx", near["dx"]), ("dwgu", near["dw_gate_up"]), ("dwd", near["dw_down"])):
            assert torch.equal(a[n], ref), (which, n)
        del a


@pytest.mark.parametrize("cols,parts", [(40, 1), (46, 2)])
def test_checkpoint_of_far_rows(zopt, cols, parts):
    gen = torch.Generator(device="cuda").manual_seed(cols)
    x = torch.randn(33, cols, generator=gen, device="cuda").bfloat16()
    near, c = zopt.new_act8(33, cols, parts), zopt.new_act8(33, cols, parts)
    zopt.act_pack(x, near)
    zopt.act_pack(far(x), c)
    assert torch.equal(c.q, near.q) and torch.equal(c.scale, near.scale)
    out, fout = torch.empty_like(x), far(torch.zeros_like(x))
    zopt.act_unpack(near, out)
    zopt.act_unpack(c, fout)
    torch.cuda.synchronize()
    assert torch.equal(out, fout)


def test_checkpoint_of_more_than_2_31_entries(zopt):
    """Bytes past 2^31 of a contiguous checkpoint: the last rows are those of a checkpoint of their own."""
    rows, cols = (1 << 31) // 4096 + 5, 4096
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    x.fill_(1.0)
    gen = torch.Generator(device="cuda").manual_seed(8)
    x[-6:] = torch.randn(6, cols, generator=gen, device="cuda").bfloat16()
    c, tail = zopt.new_act8(rows, cols), zopt.new_act8(6, cols)
    zopt.act_pack(x, c)
    zopt.act_pack(x[-6:].contiguous(), tail)
    assert torch.equal(c.q[-6:], tail.q) and torch.equal(c.scale[-6 * 32:], tail.scale)
    out = torch.empty_like(x)
    zopt.act_unpack(c, out)
    want = torch.empty_like(x[-6:])
    zopt.act_unpack(tail, want)
    torch.cuda.synchronize()
    assert torch.equal(out[-6:], want) and torch.equal(out[:8], x[:8])
