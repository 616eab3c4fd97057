"""CPU checks of which few-token calls keep partial sums for the CUDA cores: by the weights' size and by
whether their rows can be read in place. The workspace tells (a row of partial sums for every 128 hidden
columns there, none on the tensor cores' path)."""
import pytest

from tests.test_abi_lm import Z
from tests.test_abi_lm_limits import ffn_of


def workspace(tokens, dim, hidden):
    return Z.lib().zopt_ffn_workspace(ffn_of(tokens, dim, hidden), 0)


@pytest.mark.parametrize("dim,hidden", [(256, 768), (1000, 2732), (1024, 4096), (4096, 2048)])
def test_small_weights_take_the_cuda_cores(dim, hidden):
    for t in (1, 2, 3, 4):
        assert workspace(t, dim, hidden) >= 4 * t * dim * -(-hidden // 128)


@pytest.mark.parametrize("dim,hidden", [(1536, 4096), (2048, 5632), (4096, 4096), (8192, 4096)])
def test_large_weights_of_three_and_four_tokens_do_not(dim, hidden):
    for t in (1, 2):
        assert workspace(t, dim, hidden) >= 4 * t * dim * -(-hidden // 128)
    for t in (3, 4):
        assert workspace(t, dim, hidden) <= workspace(5, dim, hidden)


@pytest.mark.parametrize("dim,hidden", [(1999, 4001), (2047, 5632), (2048, 5636)])
def test_weights_that_would_be_copied_first_take_the_cuda_cores(dim, hidden):
    assert workspace(4, dim, hidden) - workspace(5, dim, hidden) >= 2 * dim * -(-hidden // 128)
