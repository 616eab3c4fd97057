"""Experts' weights at widths that the TMA does not read in place: what is copied first are the matrices of
experts that some token chose, and of no others."""
import pytest
import torch

pytestmark = pytest.mark.gpu

EXPERTS, DIM, HIDDEN = 64, 255, 129
STAGED = EXPERTS * (DIM * 264 + HIDDEN * 256) * 2  # bytes of all experts' copies in the backward


def block(tokens, top_k, chosen, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    new = lambda *s: (torch.randn(*s, generator=g, device="cuda") / 16).bfloat16()  # noqa: E731
    index = chosen[torch.rand(tokens, len(chosen), generator=g, device="cuda").argsort(dim=1)[:, :top_k]].int()
    return dict(x=new(tokens, DIM), dy=new(tokens, DIM), index=index, weight=torch.rand(tokens, top_k, generator=g, device="cuda"),
                wgu=new(EXPERTS, DIM, 2 * HIDDEN), wd=new(EXPERTS, HIDDEN, DIM), kept=new(tokens * top_k, 2 * HIDDEN))


def framed(w):
    """The same matrices in rows that start on 16 bytes."""
    cols = (w.shape[2] + 7) // 8 * 8
    whole = torch.zeros(*w.shape[:2], cols, dtype=w.dtype, device="cuda")
    whole[:, :, :w.shape[2]] = w
    return whole[:, :, :w.shape[2]]


def backward(Z, b, wgu, wd):
    ws = Z.new_experts_workspace(b["x"], b["index"], wgu, wd)
    ws.fill_(0xA5)
    out = [torch.empty_like(t) for t in (b["x"], b["weight"], b["wgu"], b["wd"])]
    Z.experts_backward(b["dy"], b["x"], b["index"], b["weight"], b["kept"], wgu, wd, *out, ws)
    torch.cuda.synchronize()
    return out, int((ws != 0xA5).sum())


def forward(Z, b, wgu, wd):
    ws = Z.new_experts_workspace(b["x"], b["index"], wgu, wd, backward=False)
    ws.fill_(0xA5)
    y, kept = torch.empty_like(b["x"]), torch.empty_like(b["kept"])
    Z.experts_forward(b["x"], b["index"], b["weight"], wgu, wd, y, ws, kept=kept)
    torch.cuda.synchronize()
    return [y, kept], int((ws != 0xA5).sum())


@pytest.mark.parametrize("tokens,top_k,chosen", [(1, 2, (0, 63)), (3, 1, (17,)), (40, 2, (5, 31, 32, 62)), (200, 3, tuple(range(1, 64, 2)))])
def test_only_what_some_token_chose(zopt, tokens, top_k, chosen):
    b = block(tokens, top_k, torch.tensor(chosen, device="cuda"))
    for run in (backward, forward):
        if run is forward and tokens * top_k <= 64:
            continue  # (the CUDA cores' path copies nothing)
        got, touched = run(zopt, b, b["wgu"], b["wd"])
        want, rest = run(zopt, b, framed(b["wgu"]), framed(b["wd"]))
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        # beside the copies the two calls leave the same; the forward copies up's columns by themselves in either
        used = len(b["index"].unique())
        assert touched - rest <= STAGED * used / EXPERTS


def test_no_expert_at_all(zopt):
    b = block(70, 2, torch.tensor([1, 2], device="cuda"))
    b["index"].fill_(-1)
    (y, _), touched = forward(zopt, b, b["wgu"], b["wd"])
    assert bool((y == 0).all()) and touched < STAGED // 64
    (dx, dweight, dwgu, dwd), touched = backward(zopt, b, b["wgu"], b["wd"])
    assert all(bool((t == 0).all()) for t in (dx, dweight, dwgu, dwd)) and touched < STAGED // 64
