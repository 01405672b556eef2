"""Time-outs in any chunk of a constrained or a distillation call: no row of any chunk is left to be trusted.

The time-out is made by withholding one pipeline signal (a wait then runs into its limit, the kernel returns and the
status says so)."""
import numpy as np
import pytest

from tests.test_gpu_constrained import env, head, rules, to_kw  # noqa: F401 (fixture)
from tests.test_gpu_distill import problem, to_gpu

pytestmark = pytest.mark.gpu


def smallest(flce, dev, call, hi):
    lo = 0
    while hi - lo > 256:
        mid = (lo + hi) // 2
        try:
            call(flce.new_workspace(mid, dev))
            hi = mid
        except flce.FlceError as e:
            assert e.status == flce.FLCE_EWORKSPACE
            lo = mid
    return flce.new_workspace(hi, dev)


@pytest.mark.parametrize("chunk", [0, 1, 3])
@pytest.mark.parametrize("K,scored", [(0, True), (5, True), (4, False)])
def test_constrained(env, chunk, K, scored):  # noqa: F811
    flce, torch, dev = env
    N, H, V = 500, 64, 3000   # four chunks of 128 tokens
    X, W = head(N, H, V, 3)
    h, w = (torch.from_numpy(a).to(torch.bfloat16).to(dev) for a in (X, W))
    kw = to_kw(torch, dev, rules(N, V, 30, 3, True, 7))
    t = None
    if scored:
        t = np.arange(N, dtype=np.int32)
        t[[7, 130, 499]] = -100
        t[300] = V
        t = torch.from_numpy(t).to(dev)
    call = lambda ws: flce.constrained_logprobs(h, w, t, top_k=K, workspace=ws, **kw)  # noqa: E731
    ws = smallest(flce, dev, call, flce.library().flce_constrained_workspace_bytes(N, H, V, K, 30, 3))
    good = call(ws)
    assert flce.query_status(ws) == (flce.FLCE_EBADTARGET if scored else flce.FLCE_OK)
    rows = t != -100 if scored else torch.ones(N, dtype=torch.bool, device=dev)
    flce.debug_arm_stall(50_000_000, after=chunk)
    bad = call(ws)
    assert flce.query_status(ws) == flce.FLCE_ETIMEOUT
    for k in ("lse", "entropy") + (("logp",) if scored else ()) + (("top_logp",) if K else ()):
        assert torch.isnan(bad[k][rows]).all(), k
        assert not bad[k][~rows].any(), k
    if K:
        assert (bad["top_ids"] == -1).all()
    again = call(ws)
    for k in ("lse", "entropy") + (("logp",) if scored else ()) + (("top_ids", "top_logp") if K else ()):
        assert torch.equal(again[k].nan_to_num(7.0), good[k].nan_to_num(7.0)), k


@pytest.mark.parametrize("chunk", [0, 1, 3])
@pytest.mark.parametrize("K", [6, 70])
def test_distillation(env, chunk, K):  # noqa: F811
    flce, torch, dev = env
    N, H, V = 500, 64, 3000
    X, W, ids, t = problem(N, H, V, K, 7)
    ids[(ids >= 0).sum(1) == 0] = -1
    ids[10:14] = np.arange(K)   # rows with a teacher in the first chunk, whatever was drawn
    h, w, i, tt = a = to_gpu(torch, dev, X, W, ids, t)
    full = np.arange(N) < 490
    i[:490] = torch.where(i[:490] < 0, 3, i[:490])   # four chunks of rows with a teacher
    rows = torch.from_numpy(full).to(dev) | (i >= 0).any(1)
    i[495] = -1
    rows[495] = False
    i[300, 2] = V
    call = lambda ws: flce.topk_distill(*a, workspace=ws)  # noqa: E731
    ws = smallest(flce, dev, call, flce.library().flce_topk_distill_workspace_bytes(N, H, V, K))
    good = call(ws)
    assert flce.query_status(ws) == flce.FLCE_EBADTARGET
    flce.debug_arm_stall(50_000_000, after=chunk)
    bad = call(ws)
    assert flce.query_status(ws) == flce.FLCE_ETIMEOUT
    for k in ("kl", "lse", "rest_logp", "student_logp"):
        assert torch.isnan(bad[k][rows]).all(), k
        assert not bad[k][~rows].any(), k
    again = call(ws)
    for k in ("kl", "lse", "rest_logp", "student_logp"):
        assert torch.equal(again[k].nan_to_num(7.0), good[k].nan_to_num(7.0)), k


@pytest.mark.parametrize("launch", [0, 1, 4, 5])
def test_distillation_gradient(env, launch):  # noqa: F811
    """Two tcgen05 launches a chunk."""
    flce, torch, dev = env
    N, H, V, K = 500, 64, 3000, 6
    X, W, ids, t = problem(N, H, V, K, 7)
    a = to_gpu(torch, dev, X, W, ids, t)
    o = flce.topk_distill(*a)
    one = torch.ones(N, device=dev)
    call = lambda ws: flce.topk_distill_bwd(*a, o["lse"], o["rest_logp"], o["student_logp"], one, workspace=ws)  # noqa: E731
    ws = smallest(flce, dev, call, flce.library().flce_topk_distill_bwd_workspace_bytes(N, H, V, K, 0))
    good = call(ws)
    flce.debug_arm_stall(50_000_000, after=launch)
    bad = call(ws)
    assert flce.query_status(ws) == flce.FLCE_ETIMEOUT
    assert torch.isnan(bad["grad_hidden"].view(-1)[0]) and torch.isnan(bad["grad_weight"].view(-1)[0])
    again = call(ws)
    assert flce.query_status(ws) == flce.FLCE_OK
    assert torch.equal(again["grad_hidden"], good["grad_hidden"]) and torch.equal(again["grad_weight"], good["grad_weight"])
