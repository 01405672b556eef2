"""Calls whose pipeline timed out: what the outputs hold, and that the next call is right.

The time-out is made by withholding one pipeline signal (a wait then runs into
its limit, the kernel returns and the status says so)."""
import pytest

from tests.test_gpu_logprobs import env, problem, to_gpu  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu

KEYS = ("logp", "lse", "entropy", "top_ids", "top_logp")


@pytest.mark.parametrize("N,H,V", [(1, 64, 100003), (40, 320, 40000), (128, 128, 100003), (300, 64, 30000),
                                   (300, 512, 30000)])
def test_next_call_is_right(env, N, H, V):  # noqa: F811
    """Fewer K blocks than ring stages: the loads of the last tile are all issued when another role gives up."""
    flce, torch, dev = env
    h, w, t = to_gpu(torch, dev, *problem(N, H, V, seed=2))
    want = flce.token_logprobs(h, w, t, top_k=4)
    up = torch.ones(N, device=dev)
    grads = flce.token_logprobs_bwd(h, w, t, want["lse"], None, up)
    for _ in range(2):
        flce.debug_arm_stall(50_000_000)
        bad = flce.token_logprobs(h, w, t, top_k=4)
        assert flce.query_status(bad["workspace"]) == flce.FLCE_ETIMEOUT
        assert torch.isnan(bad["logp"]).all()
        good = flce.token_logprobs(h, w, t, top_k=4, workspace=bad["workspace"])
        assert flce.query_status(good["workspace"]) == flce.FLCE_OK
        for k in KEYS:
            assert torch.equal(good[k], want[k]), k
        flce.debug_arm_stall(50_000_000)
        bad = flce.token_logprobs_bwd(h, w, t, want["lse"], None, up)
        assert flce.query_status(bad["workspace"]) == flce.FLCE_ETIMEOUT
        good = flce.token_logprobs_bwd(h, w, t, want["lse"], None, up, workspace=bad["workspace"])
        assert flce.query_status(good["workspace"]) == flce.FLCE_OK
        for k in ("grad_hidden", "grad_weight"):
            assert torch.equal(good[k], grads[k]), k
