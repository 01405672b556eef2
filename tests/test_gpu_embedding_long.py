"""The embedding gradient of millions of tokens: right, repeatable, and in time proportional to their number."""
import pytest

from tests.test_gpu_logprobs import env  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu


def case(torch, dev, N, H, V, seed):
    r = torch.Generator(device=dev).manual_seed(seed)
    ids = (torch.rand(N, generator=r, device=dev) ** 3 * V).to(torch.int32).clamp_(max=V - 1)
    # whole numbers of at most 8: sums of up to 2^21 of them are exact in fp32 in any order
    return ids, torch.randint(-8, 9, (N, H), generator=r, device=dev).to(torch.bfloat16)


@pytest.mark.parametrize("N,H,V", [(1_048_577, 8, 1000), (1_500_003, 16, 200_003), (5_000_001, 8, 40_000),
                                   (17_000_001, 8, 3_000_000)])
def test_sums_of_many_tokens(env, N, H, V):  # noqa: F811
    """Sums are exact up to 2^24: |x| <= 8 and no id has 2^21 tokens (the most frequent of V^(1/3) N / V of them)."""
    flce, torch, dev = env
    ids, g = case(torch, dev, N, H, V, 1)
    ids[::997] = -1          # outside the table
    ids[5::1009] = V
    inside = (ids >= 0) & (ids < V) & (ids != 2)
    assert int(torch.bincount(ids[inside].long()).max()) < 1 << 21
    d = flce.embedding_bwd(g, ids, V, 0.5, 2)
    assert flce.query_status(d["workspace"]) == flce.FLCE_EBADTARGET
    want = torch.zeros(V, H, device=dev, dtype=torch.float64)
    want.index_add_(0, ids[inside].long(), g[inside].double())
    assert torch.equal(d["grad_weight"].double(), want * 0.5)
    again = flce.embedding_bwd(g, ids, V, 0.5, 2, workspace=torch.full_like(d["workspace"], 255))
    assert torch.equal(d["grad_weight"], again["grad_weight"])


def test_time_grows_with_the_tokens(env):  # noqa: F811
    """Four times the tokens take about four times as long; work that grows with their square would take up to sixteen
    (with every block of the sort reading the counts of all tiles: 7.6)."""
    flce, torch, dev = env
    V, H = 1000, 8

    def ms(N):
        ids, g = case(torch, dev, N, H, V, 2)
        ws = flce.embedding_bwd(g, ids, V)["workspace"]
        best = float("inf")
        for _ in range(3):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            flce.embedding_bwd(g, ids, V, workspace=ws)
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        return best

    assert ms(1 << 26) < 5.6 * ms(1 << 24)
