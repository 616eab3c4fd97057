"""CPU checks of what the binding takes for a workspace, with stand-ins for GPU tensors."""
import pytest

torch = pytest.importorskip("torch")
import zero_sharded_optimizer_flat_gb300 as Z  # noqa: E402


class OnGpu:
    is_cuda = True

    def __init__(self, t):
        self.t = t

    def __getattr__(self, name):
        return getattr(self.t, name)


def test_its_bytes():
    t = torch.empty(64, dtype=torch.uint8)
    assert Z._workspace(OnGpu(t)) == (t.data_ptr(), 64)
    assert Z._workspace(OnGpu(t.view(torch.float32)))[1] == 64
    assert Z._workspace(OnGpu(t[16:]))[1] == 48


@pytest.mark.parametrize("ws", [torch.empty(1, dtype=torch.uint8).expand(1 << 40), torch.empty(64, dtype=torch.uint8)[::2]])
def test_memory_that_is_not_there(ws):
    """An expanded byte names a terabyte of which there is one."""
    with pytest.raises(ValueError, match="contiguous"):
        Z._workspace(OnGpu(ws))


def test_on_the_gpu():
    with pytest.raises(ValueError, match="GPU"):
        Z._workspace(torch.empty(64, dtype=torch.uint8))


CALLS = {
    "ffn_forward": (3, 5), "ffn_backward": (4, 9), "linear_ce_forward": (2, 6), "linear_ce_backward": (2, 8),
    "experts_forward": (5, 7), "experts_backward": (7, 12),
}


@pytest.mark.parametrize("name", CALLS)
def test_every_call_looks(name, monkeypatch):
    """Each operator passes on what _workspace gives, and a refusal before anything is launched."""
    args = CALLS[name][1] - 1
    for job in ("_ffn_job", "_linear_ce_job", "_experts_job"):
        monkeypatch.setattr(Z, job, lambda *a, **k: None)
    monkeypatch.setattr(Z, "_one_device", lambda *a: None)

    class Lib:
        def __getattr__(self, entry):
            return lambda *a: pytest.fail(f"{entry} was called")

    monkeypatch.setattr(Z, "lib", Lib)
    with pytest.raises(ValueError, match="contiguous"):
        getattr(Z, name)(*[None] * args, OnGpu(torch.empty(1, dtype=torch.uint8).expand(1 << 40)))
