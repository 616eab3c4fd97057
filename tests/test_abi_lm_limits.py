"""CPU checks: sizes whose products could outlast the kernels' bounded waits are refused, and those just
within are not refused for their size (the pointers are fake; a short workspace ends the call)."""
import pytest

from tests.test_abi_lm import BIG, P, Z, ce, ffn

M26 = 1 << 26


def ffn_of(tokens, dim, hidden):
    return ffn(tokens=tokens, dim=dim, hidden=hidden, ld_gate_up=2 * hidden, ld_down=dim, ld_x=dim, ld_kept=2 * hidden,
               ld_y=dim, ld_dy=dim, ld_dx=dim, ld_dw_gate_up=2 * hidden, ld_dw_down=dim)


def ce_of(tokens, dim, vocab):
    return ce(tokens=tokens, dim=dim, vocab=vocab, ld_x=dim, ld_w=dim, ld_dx=dim, ld_dw=dim)


@pytest.mark.parametrize("shape,refused", [  # in the forward, in the backward
    ((4, M26, 8), (0, 0)), ((4, M26 + 1, 8), (1, 1)), ((4, 8, M26 // 2), (0, 0)), ((4, 8, M26 // 2 + 1), (1, 1)),
    ((4, 8, 1 << 29), (1, 1)), ((M26, 8, 8), (0, 0)), ((M26 + 1, 8, 8), (0, 1)), ((1 << 30, 8, 8), (0, 1)),
    ((4, 1 << 30, 8), (1, 1)),
])
def test_block_limits(shape, refused):
    L = Z.lib()
    for back, call in enumerate((L.zopt_ffn_forward, L.zopt_ffn_backward)):
        j = ffn_of(*shape)
        assert (L.zopt_ffn_workspace(j, back) == 0) == bool(refused[back])
        assert call(j, P, 16 if not refused[back] else BIG, None) == 1
        assert (b"2^2" if refused[back] else b"workspace") in L.zopt_last_error()


@pytest.mark.parametrize("shape,refused", [
    ((4, M26, 8), (0, 0)), ((4, M26 + 1, 8), (1, 1)), ((M26, 8, 8), (0, 0)), ((M26 + 1, 8, 8), (0, 1)),
    ((1 << 30, 8, 8), (0, 1)), ((4, 1 << 30, 8), (1, 1)), ((4, 8, 1 << 30), (0, 0)),
])
def test_cross_entropy_limits(shape, refused):
    L = Z.lib()
    for back, call in enumerate((L.zopt_linear_ce_forward, L.zopt_linear_ce_backward)):
        j = ce_of(*shape)
        assert (L.zopt_linear_ce_workspace(j, back) == 0) == bool(refused[back])
        assert call(j, P, 16 if not refused[back] else BIG, None) == 1
        assert (b"2^26" if refused[back] else b"workspace") in L.zopt_last_error()
