"""CPU checks of the binding's argument checks for the training operators, with stand-ins for GPU tensors."""
import pytest

torch = pytest.importorskip("torch")
import zero_sharded_optimizer_flat_gb300 as Z  # noqa: E402


class OnGpu:
    """What the checks look at of a contiguous vector on the GPU."""
    is_cuda = True

    def __init__(self, dtype, n=4):
        self.t = torch.zeros(n, dtype=dtype)
        self.shape, self.dtype = self.t.shape, dtype

    def __getattr__(self, name):
        return getattr(self.t, name)


@pytest.mark.parametrize("dtype", [torch.complex64, torch.float64, torch.int32, torch.float32])
def test_targets_are_int64(dtype):
    assert Z._vector(OnGpu(torch.int64), 4, Z.I64, "target")
    with pytest.raises(ValueError, match="int64"):
        Z._vector(OnGpu(dtype), 4, Z.I64, "target")


@pytest.mark.parametrize("dtype", [torch.complex64, torch.float64, torch.int64, torch.bfloat16])
def test_losses_are_fp32(dtype):
    assert Z._vector(OnGpu(torch.float32), 4, Z.F32, "loss")
    with pytest.raises(ValueError, match="fp32"):
        Z._vector(OnGpu(dtype), 4, Z.F32, "loss")
