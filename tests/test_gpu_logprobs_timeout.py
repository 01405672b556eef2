"""Calls whose pipeline timed out: what the outputs hold, and that the next call is right.

The time-out is made by withholding one pipeline signal (a wait then runs into
its limit, the kernel returns and the status says so)."""
import pytest

from tests.test_gpu_logprobs import env, problem, to_gpu  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu

KEYS = ("logp", "lse", "entropy", "top_ids", "top_logp")


@pytest.mark.parametrize("N,H,V", [(1, 64, 100003), (40, 320, 40000), (128, 128, 100003), (300, 64, 30000),
                                   (300, 512, 30000), (300, 1024, 9000), (20, 1024, 60000)])
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


@pytest.mark.parametrize("chunk", [0, 1, 3])
@pytest.mark.parametrize("K", [0, 5])
def test_every_scored_row_is_nan(env, chunk, K):  # noqa: F811
    """A time-out in any chunk of a call marks the rows of all of them; ignored tokens and bad targets stay as they are."""
    flce, torch, dev = env
    N, H, V = 500, 64, 3000   # four chunks of 128 tokens
    X, W, t = problem(N, H, V, seed=3)
    t[[7, 130, 499]] = -100
    t[300] = V
    h, w, tt = to_gpu(torch, dev, X, W, t)
    lo, hi = 0, flce.library().flce_logprobs_workspace_bytes(N, H, V, K)
    while hi - lo > 256:   # the smallest workspace that is accepted: chunks of 128
        mid = (lo + hi) // 2
        try:
            flce.token_logprobs(h, w, tt, top_k=K, workspace=flce.new_workspace(mid, dev))
            hi = mid
        except flce.FlceError:
            lo = mid
    ws = flce.new_workspace(hi, dev)
    good = flce.token_logprobs(h, w, tt, top_k=K, workspace=ws)
    assert flce.query_status(ws) == flce.FLCE_EBADTARGET
    scored = tt >= 0
    assert torch.isfinite(good["logp"][scored & (tt < V)]).all()
    flce.debug_arm_stall(50_000_000, after=chunk)
    bad = flce.token_logprobs(h, w, tt, top_k=K, workspace=ws)
    assert flce.query_status(ws) == flce.FLCE_ETIMEOUT
    for k in ("logp", "lse", "entropy") + (("top_logp",) if K else ()):
        assert torch.isnan(bad[k][scored]).all(), k
        assert not bad[k][~scored].any(), k
    if K:
        assert (bad["top_ids"] == -1).all()
