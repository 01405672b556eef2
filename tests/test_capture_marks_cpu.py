"""A captured backward beside a living eager loss of the same leaves (no GPU: streams and kernels are stood in for)."""
import pytest

torch = pytest.importorskip("torch")

from linear_cross_entropy_ce_gb300 import flce  # noqa: E402


class Double(torch.autograd.Function):
    """An operator that marks and checks its leaves as the framework's do."""

    @staticmethod
    def forward(ctx, x):
        flce._mark_leaves(ctx, x.device)
        return 2 * x

    @staticmethod
    def backward(ctx, g):
        flce._check_capture(ctx)
        return 2 * g


@pytest.fixture
def now(monkeypatch):
    now = {"stream": 0, "capturing": False}
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: now["stream"], raising=False)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: now["capturing"])
    monkeypatch.setattr(flce, "fwd_bwd", lambda h, w, *a: {
        "loss": h.sum().reshape(1), "n_valid": None, "grad_hidden": torch.ones_like(h), "grad_weight": torch.ones_like(w)})
    monkeypatch.setattr(flce, "scale_grads", lambda gh, gw, s: None)
    return now


@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("captured_loss", [False, True])
def test_refused_while_the_loss_lives(now, which, captured_loss):
    leaves = [torch.ones(2, 8, requires_grad=True), torch.ones(3, 8, requires_grad=True)]
    leaf = leaves[which]
    t = torch.zeros(2, dtype=torch.int32)

    def captured():
        now.update(stream=9, capturing=True)
        y = flce.linear_cross_entropy(*leaves, t) if captured_loss else Double.apply(leaf).sum()
        return torch.autograd.grad(y, leaf)[0]

    loss = flce.linear_cross_entropy(*leaves, t)   # eager, on the default stream
    assert torch.equal(torch.autograd.grad(loss, leaf, retain_graph=True)[0], torch.ones_like(leaf))
    with pytest.raises(RuntimeError, match="alive"):
        captured()
    del loss
    assert captured().shape == leaf.shape


def test_not_refused_on_another_stream(now):
    leaf, w, t = torch.ones(2, 8, requires_grad=True), torch.ones(3, 8), torch.zeros(2, dtype=torch.int32)
    now.update(stream=7)
    loss = flce.linear_cross_entropy(leaf, w, t)
    now.update(stream=9, capturing=True)
    assert torch.autograd.grad(Double.apply(leaf).sum(), leaf)[0].sum() == 32
    del loss
