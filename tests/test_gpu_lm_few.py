"""The block for one to four tokens, every count with both activations and both kept formats, against the
fp64 oracle with the tolerances of test_gpu_lm.py."""
import pytest
import torch

from tests.test_gpu_lm import check_ffn, ffn_case, run_ffn

pytestmark = pytest.mark.gpu

SHAPES = [  # dim, hidden, row distances beyond the rows (None: contiguous)
    (8, 8, None), (64, 128, None), (100, 130, None), (33, 97, 3), (264, 520, 8), (700, 300, None),
]


@pytest.mark.parametrize("keep", ["bf16", "e4m3"])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("d,f,pad", SHAPES)
@pytest.mark.parametrize("t", [1, 2, 3, 4])
def test_block_of_few_tokens(zopt, t, d, f, pad, act, keep):
    args = ffn_case(100 * t + d + f, t, d, f, pad)
    got, kept, x8 = run_ffn(zopt, *args, act, keep, pad)
    check_ffn(*args, act, got, kept, x8)
    again, _, _ = run_ffn(zopt, *args, act, keep, pad)
    assert all(torch.equal(got[n], again[n]) for n in got)


@pytest.mark.parametrize("t", [1, 2, 3, 4])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_block_of_few_tokens_keeps_nothing(zopt, t, act):
    x, dy, wgu, wd = ffn_case(t, t, 264, 520)
    kept = run_ffn(zopt, x, dy, wgu, wd, act, "bf16")[0]["y"]
    y = torch.empty_like(x)
    zopt.ffn_forward(x, wgu, wd, y, zopt.new_ffn_workspace(x, wgu, wd, backward=False), act=act)
    torch.cuda.synchronize()
    assert torch.equal(y, kept)


@pytest.mark.parametrize("t", [3, 4])
def test_few_tokens_of_large_weights_run_as_more_do(zopt, t):
    """Weights past the few-token path's size: a token's result is that of a larger batch, bit for bit."""
    x, _, wgu, wd = ffn_case(9, 5, 1536, 4096)
    y5, y = torch.empty_like(x), torch.empty_like(x[:t])
    zopt.ffn_forward(x, wgu, wd, y5, zopt.new_ffn_workspace(x, wgu, wd, backward=False))
    zopt.ffn_forward(x[:t], wgu, wd, y, zopt.new_ffn_workspace(x[:t], wgu, wd, backward=False))
    torch.cuda.synchronize()
    assert torch.equal(y, y5[:t])
