"""A distillation call behind what its caller put on the stream: a copy, a wait for another stream, eagerly and in a
captured graph (its first kernel is launched before any of its own stands in front of it)."""
import pytest

from tests.test_gpu_distill import env, problem, to_gpu  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu

KEYS = ("kl", "lse", "rest_logp", "student_logp")


@pytest.mark.parametrize("N", [20, 300])
@pytest.mark.parametrize("before", ["copy", "event", "kernel"])
def test_sees_what_stands_before_it(env, N, before):  # noqa: F811
    flce, torch, dev = env
    sets = [to_gpu(torch, dev, *problem(N, 64, 2000, 30, seed)) for seed in (1, 2)]
    want = [flce.topk_distill(*a) for a in sets]
    feed = [x.clone() for x in sets[0]]
    live = [torch.zeros_like(x) for x in feed]
    big = torch.zeros(1 << 27, device=dev)   # something that takes a while
    other = torch.cuda.Stream()

    def step():
        here = torch.cuda.current_stream()
        if before == "event":
            other.wait_stream(here)
            with torch.cuda.stream(other):
                big.add_(1.0)
                for x, y in zip(live, feed):
                    x.copy_(y)
            here.wait_stream(other)
        else:
            big.add_(1.0)
            for x, y in zip(live, feed):
                if before == "copy":
                    x.copy_(y)          # a copy on the device
                else:
                    torch.add(y, 0, out=x)
        return flce.topk_distill(*live)

    o = step()
    torch.cuda.synchronize()
    for k in KEYS:
        assert torch.equal(o[k], want[0][k]), k
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = step()
    for s in (1, 0, 1):
        for x, y in zip(feed, sets[s]):
            x.copy_(y)
        for x in live:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for k in KEYS:
            assert torch.equal(o[k], want[s][k]), (k, s)
