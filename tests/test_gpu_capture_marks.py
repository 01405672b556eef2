"""A backward captured while an eager loss of the same leaf lives on the default stream is refused, before autograd
orders that stream behind the capture (which would end the process)."""
import pytest

from tests.test_gpu_logprobs import env, problem, to_gpu  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("captured", ["logprobs", "loss"])
def test_capture_beside_a_living_loss(env, captured):  # noqa: F811
    flce, torch, dev = env
    h, w, t = to_gpu(torch, dev, *problem(200, 64, 500, seed=4, ignored=0.1))
    w.requires_grad_(True)

    def forward():
        return flce.linear_logprobs(h, w, t)[0].sum() if captured == "logprobs" else flce.linear_cross_entropy(h, w, t)

    want = torch.autograd.grad(forward(), w)[0]
    loss = flce.linear_cross_entropy(h, w, t)   # eager, alive
    torch.cuda.synchronize()
    with pytest.raises(RuntimeError, match="alive"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            torch.autograd.grad(forward(), w)
    del loss
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = torch.autograd.grad(forward(), w)[0]
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)
