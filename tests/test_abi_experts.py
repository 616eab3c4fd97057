"""CPU checks of the routing's and the experts' C entry points: struct sizes as the header states them,
workspace sizes, and refusals before any launch (the pointers are fake)."""
import ctypes

import pytest

from zero_sharded_optimizer_flat_gb300 import build_lib

build_lib.build()
import zero_sharded_optimizer_flat_gb300 as Z  # noqa: E402

P, BIG = 1 << 20, 1 << 50


def route(**kw):
    j = Z._RouteJob()
    j.tokens, j.experts, j.top_k, j.groups, j.top_groups, j.renormalise, j.scale = 64, 16, 4, 1, 1, 1, 1.0
    j.dtype = Z.F32
    j.logits = j.index = j.weight = j.counts = j.bias = j.live = j.dweight = j.dlogits = P
    j.ld_logits = j.ld_dlogits = 16
    for k, v in kw.items():
        setattr(j, k, v)
    return j


def experts(**kw):
    j = Z._ExpertsJob()
    j.tokens, j.dim, j.hidden, j.experts, j.top_k, j.dtype = 64, 32, 48, 8, 2, Z.BF16
    j.index = j.weight = j.dweight = P
    for n, ld in (("w_gate_up", 96), ("w_down", 32), ("x", 32), ("kept", 96), ("y", 32), ("dy", 32), ("dx", 32),
                  ("dw_gate_up", 96), ("dw_down", 32)):
        setattr(j, n, P)
        setattr(j, "ld_" + {"w_gate_up": "gate_up", "w_down": "down"}.get(n, n), ld)
    j.stride_gate_up = j.stride_dw_gate_up = 32 * 96
    j.stride_down = j.stride_dw_down = 48 * 32
    for k, v in kw.items():
        setattr(j, k, v)
    return j


def act8(rows=128, cols=96, parts=2, q=P, scale=P):
    return Z._Act8(q, scale, rows, cols, parts, 0)


def test_struct_sizes():
    assert (ctypes.sizeof(Z._RouteJob), ctypes.sizeof(Z._ExpertsJob)) == (128, 256)


@pytest.mark.parametrize("kw,status,frag", [
    ({"dtype": 2}, 2, b"dtype"), ({"dtype": -1}, 2, b"dtype"), ({"score": 2}, 1, b"score"), ({"score": -1}, 1, b"score"),
    ({"tokens": -1}, 1, b"tokens"), ({"tokens": (1 << 30) + 1}, 1, b"2^30"),
    ({"experts": 0}, 1, b"experts"), ({"experts": 1025}, 1, b"experts"),
    ({"top_k": 0}, 1, b"top_k"), ({"top_k": 17}, 1, b"top_k"), ({"experts": 64, "top_k": 33, "ld_logits": 64}, 1, b"top_k"),
    ({"groups": 0}, 1, b"groups"), ({"groups": 3}, 1, b"groups"), ({"experts": 64, "groups": 64}, 1, b"groups"),
    ({"groups": 4, "top_groups": 0}, 1, b"top_groups"), ({"groups": 4, "top_groups": 5}, 1, b"top_groups"),
    ({"groups": 8, "top_groups": 1}, 1, b"top_k"), ({"renormalise": 2}, 1, b"renormalise"),
    ({"scale": 0.0}, 1, b"scale"), ({"scale": -1.0}, 1, b"scale"), ({"scale": float("inf")}, 1, b"scale"),
    ({"scale": float("nan")}, 1, b"scale"), ({"ld_logits": 15}, 1, b"row distance"), ({"ld_logits": (1 << 32) + 1}, 1, b"row distance"),
    ({"logits": None}, 1, b"NULL"), ({"index": None}, 1, b"NULL"), ({"weight": None}, 1, b"NULL"),
    ({"logits": P + 2}, 1, b"aligned"), ({"index": P + 2}, 1, b"aligned"), ({"weight": P + 1}, 1, b"aligned"),
    ({"bias": P + 2}, 1, b"aligned"), ({"counts": P + 2}, 1, b"aligned"), ({"reserved": (1, 0)}, 1, b"reserved"),
])
def test_route_refusals(kw, status, frag):
    if "reserved" in kw:
        kw = {"reserved": (ctypes.c_int32 * 2)(*kw["reserved"])}
    L = Z.lib()
    for call in (L.zopt_route_forward, L.zopt_route_backward):
        assert call(route(**kw), None) == status and frag in L.zopt_last_error()
        assert call(None, None) == 1


def test_route_refusals_of_the_backward():
    L = Z.lib()
    for kw in ({"dweight": None}, {"dlogits": None}, {"ld_dlogits": 15}, {"dlogits": P + 2}, {"dweight": P + 2}):
        assert L.zopt_route_backward(route(**kw), None) == 1
    assert L.zopt_route_backward(route(tokens=0), None) == 0  # nothing to do


@pytest.mark.parametrize("kw,status,frag", [
    ({"dtype": Z.F32}, 2, b"dtype"), ({"act": 2}, 1, b"act"), ({"act": -1}, 1, b"act"),
    ({"tokens": -1}, 1, b"tokens"), ({"dim": 0}, 1, b"dim"), ({"hidden": 0}, 1, b"hidden"),
    ({"experts": 0}, 1, b"experts"), ({"experts": 1025}, 1, b"experts"), ({"top_k": 0}, 1, b"top_k"), ({"top_k": 33}, 1, b"top_k"),
    ({"tokens": 1 << 26}, 1, b"2^26"), ({"hidden": 1 << 26}, 1, b"2^25"), ({"dim": 1 << 27}, 1, b"2^26"),
    ({"ld_gate_up": 95}, 1, b"row distance"), ({"ld_down": 31}, 1, b"row distance"), ({"ld_down": (1 << 32) + 8}, 1, b"row distance"),
    ({"stride_gate_up": 32 * 96 - 1}, 1, b"stride"), ({"stride_down": 0}, 1, b"stride"), ({"stride_down": 1 << 39}, 1, b"stride"),
    ({"w_gate_up": None}, 1, b"NULL"), ({"w_down": P + 8}, 1, b"aligned"),
    ({"index": None}, 1, b"NULL"), ({"weight": None}, 1, b"NULL"), ({"index": P + 2}, 1, b"aligned"), ({"weight": P + 2}, 1, b"aligned"),
    ({"x": P + 2}, 1, b"x:"), ({"x": None}, 1, b"x8"), ({"ld_x": 31}, 1, b"x:"),
    ({"kept": P + 8}, 1, b"kept"), ({"ld_kept": 95}, 1, b"kept"),
])
def test_experts_refusals(kw, status, frag):
    L = Z.lib()
    for call in (L.zopt_experts_forward, L.zopt_experts_backward):
        assert call(experts(**kw), P, BIG, None) == status and frag in L.zopt_last_error()


def test_experts_refusals_of_one_direction():
    L = Z.lib()
    f, b = L.zopt_experts_forward, L.zopt_experts_backward
    ptr = lambda c: ctypes.pointer(c)  # noqa: E731
    assert f(None, P, BIG, None) == 1 and b(None, P, BIG, None) == 1
    assert f(experts(y=None), P, BIG, None) == 1 and f(experts(ld_y=31), P, BIG, None) == 1 and f(experts(y=P + 2), P, BIG, None) == 1
    for k in ("dy", "dx", "dw_gate_up", "dw_down"):
        assert b(experts(**{k: None}), P, BIG, None) == 1
        assert b(experts(**{k: P + 8}), P, BIG, None) == 1
        assert b(experts(**{"ld_" + k: 31}), P, BIG, None) == 1
    for k in ("stride_dw_gate_up", "stride_dw_down"):
        assert b(experts(**{k: 100}), P, BIG, None) == 1 and b"stride" in L.zopt_last_error()
    assert b(experts(dweight=None), P, BIG, None) == 1 and b(experts(dweight=P + 2), P, BIG, None) == 1
    assert b(experts(kept=None), P, BIG, None) == 1 and b"kept" in L.zopt_last_error()
    both = experts(kept8=ptr(act8()))
    assert f(both, P, BIG, None) == 1 and b(both, P, BIG, None) == 1 and b"both" in L.zopt_last_error()
    for bad in (act8(parts=1), act8(rows=64), act8(cols=98), act8(q=P + 8), act8(scale=None)):
        j = experts(kept=None, kept8=ptr(bad))
        assert f(j, P, BIG, None) == 1 and b(j, P, BIG, None) == 1
    x8 = ptr(act8(64, 32, 1))
    assert f(experts(x8=x8), P, BIG, None) == 1 and f(experts(x=None, x8=x8), P, BIG, None) == 1
    assert b(experts(x8=x8), P, BIG, None) == 1 and b"exactly one" in L.zopt_last_error()
    assert b(experts(x=None, x8=ptr(act8(64, 33, 1))), P, BIG, None) == 1
    for call, back in ((f, 0), (b, 1)):
        need = L.zopt_experts_workspace(experts(), back)
        assert need > 0
        assert call(experts(), P, need - 1, None) == 1 and b"workspace" in L.zopt_last_error()
        assert call(experts(), P + 8, need, None) == 1 and call(experts(), None, need, None) == 1
    assert f(experts(tokens=0), None, 0, None) == 0  # nothing to do


def test_experts_workspace():
    size = lambda back=1, **kw: Z.lib().zopt_experts_workspace(experts(**kw), back)  # noqa: E731
    assert Z.lib().zopt_experts_workspace(None, 1) == 0 and size(dim=0) == 0 and size(ld_down=8) == 0 and size(stride_down=1) == 0
    assert size(experts=1, stride_gate_up=0, stride_down=0) > 0  # no distance between one expert's matrices
    for kw in ({}, {"tokens": 1}, {"tokens": 4096}, {"hidden": 47}, {"dim": 31}, {"experts": 1024, "tokens": 3}):
        assert size(**kw) >= size(0, **kw) > 0
    # the forward keeps the rows, and h, of every slot and at most 63 more for each expert in use
    rows = 4096 * 2 + 8 * 63 + 64
    assert size(0, tokens=4096) < rows * (32 + 48) * 2 + 64 * 1024 * 4
    assert size(0, ld_down=33, stride_down=48 * 33) - size(0) >= 8 * 48 * 32 * 2  # a copy that the TMA can read


def test_python_refusals():
    torch = pytest.importorskip("torch")
    x, wd = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(3, 6, 8, dtype=torch.bfloat16)
    index = torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        Z.experts_workspace(x, index, torch.zeros(3, 8, 12, dtype=torch.bfloat16), wd)
    with pytest.raises(ValueError, match="matrices"):
        Z.experts_workspace(x, index, torch.zeros(3, 8, 10, dtype=torch.bfloat16), wd)
    with pytest.raises(ValueError, match="GPU"):
        Z.route_forward(torch.zeros(4, 3), index, torch.zeros(4, 2))


@pytest.mark.parametrize("packer,job", [(Z._ROUTE_JOB, Z._RouteJob), (Z._EXPERTS_JOB, Z._ExpertsJob)])
def test_packed_jobs_have_the_structs_layout(packer, job):
    """The calls pack a job's fields in their order: each value lands in its field."""
    n = len(packer.unpack(bytes(packer.size)))
    j = job.from_buffer_copy(packer.pack(*range(1, n + 1)))
    names = [name for name, _ in job._fields_ if name != "reserved"]
    assert len(names) == n and packer.size == ctypes.sizeof(job)
    for k, name in enumerate(names, 1):
        v = getattr(j, name)
        assert (ctypes.cast(v, ctypes.c_void_p).value if isinstance(v, ctypes._Pointer) else v) == k, name
