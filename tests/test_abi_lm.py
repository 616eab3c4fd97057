"""CPU checks of the training operators' C entry points: struct sizes as the header states them,
workspace sizes, and refusals before any launch (the pointers are fake)."""
import ctypes

import pytest

from zero_sharded_optimizer_flat_gb300 import build_lib

build_lib.build()
import zero_sharded_optimizer_flat_gb300 as Z  # noqa: E402

P, BIG = 1 << 20, 1 << 50


def ce(**kw):
    j = Z._LinearCeJob()
    j.tokens, j.dim, j.vocab, j.ignore_index = 64, 32, 1000, -100
    j.x = j.w = j.target = j.loss = j.lse = j.dloss = j.dx = j.dw = P
    j.ld_x = j.ld_w = j.ld_dx = j.ld_dw = 32
    j.dtype = Z.BF16
    for k, v in kw.items():
        setattr(j, k, v)
    return j


def ffn(**kw):
    j = Z._FfnJob()
    j.tokens, j.dim, j.hidden, j.dtype = 64, 32, 48, Z.BF16
    for n, ld in (("w_gate_up", 96), ("w_down", 32), ("x", 32), ("kept", 96), ("y", 32), ("dy", 32), ("dx", 32),
                  ("dw_gate_up", 96), ("dw_down", 32)):
        setattr(j, n, P)
        setattr(j, "ld_" + {"w_gate_up": "gate_up", "w_down": "down"}.get(n, n), ld)
    for k, v in kw.items():
        setattr(j, k, v)
    return j


def act8(rows=64, cols=32, parts=1, q=P, scale=P):
    return Z._Act8(q, scale, rows, cols, parts, 0)


def test_struct_sizes():
    assert (ctypes.sizeof(Z._Act8), ctypes.sizeof(Z._FfnJob), ctypes.sizeof(Z._LinearCeJob)) == (40, 192, 136)


@pytest.mark.parametrize("kw,status,frag", [
    ({"dtype": Z.F32}, 2, b"dtype"), ({"dtype": -1}, 2, b"dtype"),
    ({"tokens": -1}, 1, b"tokens"), ({"dim": 0}, 1, b"dim"), ({"vocab": 0}, 1, b"vocab"),
    ({"tokens": (1 << 30) + 1}, 1, b"2^30"), ({"vocab": 1 << 31}, 1, b"2^30"),
    ({"ld_x": 31}, 1, b"row distance"), ({"ld_w": (1 << 32) + 8}, 1, b"row distance"),
    ({"x": None}, 1, b"NULL"), ({"w": None}, 1, b"NULL"), ({"target": None}, 1, b"NULL"), ({"lse": None}, 1, b"NULL"),
    ({"x": P + 8}, 1, b"aligned"), ({"w": P + 2}, 1, b"aligned"), ({"target": P + 4}, 1, b"aligned"),
    ({"lse": P + 2}, 1, b"aligned"),
])
def test_linear_ce_refusals(kw, status, frag):
    L = Z.lib()
    for call in (L.zopt_linear_ce_forward, L.zopt_linear_ce_backward):
        assert call(ce(**kw), P, BIG, None) == status and frag in L.zopt_last_error()


def test_linear_ce_refusals_of_one_direction():
    L = Z.lib()
    f, b = L.zopt_linear_ce_forward, L.zopt_linear_ce_backward
    assert f(None, P, BIG, None) == 1 and b(None, P, BIG, None) == 1
    assert f(ce(loss=None), P, BIG, None) == 1 and b(ce(dloss=None), P, BIG, None) == 1
    assert b(ce(dx=None, dw=None), P, BIG, None) == 1 and b"neither" in L.zopt_last_error()
    assert b(ce(dx=P + 8), P, BIG, None) == 1 and b(ce(dw=P + 8), P, BIG, None) == 1
    assert b(ce(ld_dx=31), P, BIG, None) == 1 and b(ce(ld_dw=31), P, BIG, None) == 1
    for call, back in ((f, 0), (b, 1)):
        need = L.zopt_linear_ce_workspace(ce(), back)
        assert need > 0
        assert call(ce(), P, need - 1, None) == 1 and b"workspace" in L.zopt_last_error()
        assert call(ce(), None, need, None) == 1 and call(ce(), P + 8, need, None) == 1


def test_linear_ce_workspace_keeps_no_logits():
    size = lambda back=1, **kw: Z.lib().zopt_linear_ce_workspace(ce(**kw), back)  # noqa: E731
    assert size(tokens=-1) == 0 and size(dim=0) == 0 and size(ld_x=8) == 0 and Z.lib().zopt_linear_ce_workspace(None, 1) == 0
    assert size(tokens=0) > 0
    big = dict(tokens=65536, dim=2048, vocab=131072, ld_x=2048, ld_w=2048)
    assert size(**big) >= size(0, **big)
    assert size(**big) < 65536 * 131072 * 2 / 4  # well under the bf16 logits alone
    assert size(tokens=1 << 25, vocab=1 << 20) == 0  # logits above 2^44
    odd = dict(dim=33, ld_x=33, ld_w=33)  # staged copies of x and w
    assert size(**odd) - size(dim=33, ld_x=40, ld_w=40) >= 2 * 40 * (64 + 1000)


@pytest.mark.parametrize("kw,status,frag", [
    ({"dtype": Z.F32}, 2, b"dtype"), ({"act": 2}, 1, b"act"), ({"act": -1}, 1, b"act"),
    ({"tokens": -1}, 1, b"tokens"), ({"dim": 0}, 1, b"dim"), ({"hidden": 0}, 1, b"hidden"),
    ({"hidden": 1 << 30}, 1, b"2^29"), ({"ld_gate_up": 95}, 1, b"row distance"), ({"ld_down": 31}, 1, b"row distance"),
    ({"w_gate_up": None}, 1, b"NULL"), ({"w_down": P + 8}, 1, b"aligned"), ({"x": P + 2}, 1, b"x:"),
    ({"x": None}, 1, b"x8"), ({"ld_x": 31}, 1, b"x:"), ({"kept": P + 8}, 1, b"kept"), ({"ld_kept": 95}, 1, b"kept"),
])
def test_ffn_refusals(kw, status, frag):
    L = Z.lib()
    for call in (L.zopt_ffn_forward, L.zopt_ffn_backward):
        assert call(ffn(**kw), P, BIG, None) == status and frag in L.zopt_last_error()


def test_ffn_refusals_of_one_direction():
    L = Z.lib()
    f, b = L.zopt_ffn_forward, L.zopt_ffn_backward
    ptr = lambda c: ctypes.pointer(c)  # noqa: E731
    assert f(None, P, BIG, None) == 1 and b(None, P, BIG, None) == 1
    assert f(ffn(y=None), P, BIG, None) == 1 and f(ffn(ld_y=31), P, BIG, None) == 1
    for k in ("dy", "dx", "dw_gate_up", "dw_down"):
        assert b(ffn(**{k: None}), P, BIG, None) == 1
        assert b(ffn(**{k: P + 8}), P, BIG, None) == 1
        assert b(ffn(**{"ld_" + k: 31}), P, BIG, None) == 1
    assert b(ffn(kept=None), P, BIG, None) == 1 and b"kept" in L.zopt_last_error()
    both = ffn(kept8=ptr(act8(64, 96, 2)))
    assert f(both, P, BIG, None) == 1 and b(both, P, BIG, None) == 1 and b"both" in L.zopt_last_error()
    for bad in (act8(64, 96, 1), act8(63, 96, 2), act8(64, 98, 2), act8(64, 96, 2, q=P + 8), act8(64, 96, 2, scale=None)):
        j = ffn(kept=None, kept8=ptr(bad))
        assert f(j, P, BIG, None) == 1 and b(j, P, BIG, None) == 1
    assert f(ffn(x8=ptr(act8())), P, BIG, None) == 1
    assert b(ffn(x8=ptr(act8())), P, BIG, None) == 1 and b"exactly one" in L.zopt_last_error()
    assert b(ffn(x=None, x8=ptr(act8(64, 33))), P, BIG, None) == 1
    for call, back in ((f, 0), (b, 1)):
        need = L.zopt_ffn_workspace(ffn(), back)
        assert need > 0
        assert call(ffn(), P, need - 1, None) == 1 and b"workspace" in L.zopt_last_error()
        assert call(ffn(), P + 8, need, None) == 1


def test_ffn_workspace_covers_both_directions():
    L = Z.lib()
    for kw in ({}, {"tokens": 1}, {"tokens": 8192, "dim": 2048, "hidden": 5632, "ld_gate_up": 11264, "ld_down": 2048,
                                  "ld_x": 2048, "ld_dy": 2048}, {"hidden": 47}):
        assert L.zopt_ffn_workspace(ffn(**kw), 1) >= L.zopt_ffn_workspace(ffn(**kw), 0) > 0
    assert L.zopt_ffn_workspace(ffn(tokens=1 << 30, dim=1 << 15, ld_down=1 << 15, ld_x=1 << 15, ld_dy=1 << 15), 1) == 0
    assert L.zopt_ffn_workspace(None, 1) == 0 and L.zopt_ffn_workspace(ffn(dim=0), 1) == 0


def test_act8_refusals():
    L = Z.lib()
    assert Z.act8_scale_bytes(10, 300) == 30 and Z.act8_scale_bytes(10, 300, 2) == 40
    assert Z.act8_scale_bytes(10, 301, 2) == 0 and Z.act8_scale_bytes(-1, 8) == 0 and Z.act8_scale_bytes(1, 0) == 0
    good = act8()
    pack = lambda x=P, ld=32, c=good: L.zopt_act_pack(x, ld, c, None)  # noqa: E731
    unpack = lambda x=P, ld=32, c=good: L.zopt_act_unpack(c, x, ld, None)  # noqa: E731
    for call in (pack, unpack):
        assert call(x=None) == 1 and call(x=P + 8) == 1 and b"aligned" in L.zopt_last_error()
        assert call(ld=31) == 1 and call(ld=1 << 33) == 1 and call(c=None) == 1
        for bad in (act8(rows=-1), act8(cols=0), act8(parts=0), act8(parts=3), act8(cols=33, parts=2),
                    act8(rows=1 << 31), act8(q=None), act8(scale=None), act8(q=P + 4)):
            assert call(ld=64, c=bad) == 1
        assert call(c=act8(rows=0)) == 0  # nothing to do


def test_python_refusals():
    torch = pytest.importorskip("torch")
    x, w = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(6, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        Z.linear_ce_workspace(x, w)
    with pytest.raises(ValueError, match="matrix"):
        Z.ffn_workspace(x, torch.zeros(8, 10, dtype=torch.bfloat16), w)
    with pytest.raises(ValueError, match="GPU"):
        Z.new_act8(4, 8, device="cpu")
    with pytest.raises(ValueError, match="bytes"):
        Z.Act8(torch.zeros(4, 8, dtype=torch.uint8), torch.zeros(3, dtype=torch.uint8))
