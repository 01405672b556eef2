"""The caller's output dict over calls that ask for different outputs."""
import pytest

from tests.test_gpu_logprobs import env, problem, to_gpu  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N", [5, 200])
def test_entries_not_asked_for_are_left_alone(env, N):  # noqa: F811
    flce, torch, dev = env
    h, w, t = to_gpu(torch, dev, *problem(N, 64, 500, seed=1))
    full = flce.token_logprobs(h, w, t, top_k=3)
    out = {k: torch.full_like(full[k], -7) for k in ("logp", "lse", "entropy", "top_ids", "top_logp")}
    mine = dict(out)
    got = flce.token_logprobs(h, w, t, entropy=False, out=out)
    assert got is out and all(out[k] is mine[k] for k in mine)
    assert torch.equal(out["logp"], full["logp"]) and torch.equal(out["lse"], full["lse"])
    assert all((out[k] == -7).all() for k in ("entropy", "top_ids", "top_logp"))
    again = flce.token_logprobs(h, w, t, top_k=3, out=out)
    assert all(again[k] is mine[k] and torch.equal(mine[k], full[k]) for k in mine)
    up = torch.ones(N, device=dev)
    both = flce.token_logprobs_bwd(h, w, t, full["lse"], None, up)
    grads = {k: torch.full_like(both[k], -7) for k in ("grad_hidden", "grad_weight")}
    one = flce.token_logprobs_bwd(h, w, t, full["lse"], None, up, need_weight=False, out=grads)
    assert (one["grad_weight"] == -7).all() and torch.equal(one["grad_hidden"], both["grad_hidden"])
