"""A logit that is not a number and that a rule changes: its row says so."""
import numpy as np
import pytest

from tests.test_gpu_constrained import env, head  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("others", ["none", "banned", "said"])
@pytest.mark.parametrize("N", [5, 200])
def test_nan_of_a_listed_token(env, N, others):  # noqa: F811
    """The token is a row's only listed one, or the others' logits are -inf, or there are other ones."""
    flce, torch, dev = env
    V, bad = 900, 137
    X, W = head(N, 64, V, 5)
    h, w = (torch.from_numpy(a).to(torch.bfloat16).to(dev) for a in (X, W))
    w[bad] = float("nan")
    hist = torch.full((N, 40), -1, dtype=torch.int32, device=dev)
    hist[:, 3] = bad
    kw = {}
    if others == "said":
        hist[:, 5:35] = torch.arange(30, device=dev, dtype=torch.int32) * 11
    if others == "banned":
        kw = {"bias_ids": torch.arange(30, device=dev, dtype=torch.int32).expand(N, -1).contiguous(),
              "bias": torch.full((N, 30), -float("inf"), device=dev)}
    o = flce.constrained_logprobs(h, w, torch.arange(N, device=dev, dtype=torch.int32), history=hist,
                                  repetition_penalty=torch.full((N,), 1.25, device=dev), top_k=3, **kw)
    for k in ("logp", "lse", "entropy", "top_logp"):
        if k == "logp" and others == "banned":   # a forbidden target in a row that is not a number: that too
            continue
        assert torch.isnan(o[k]).all(), k
    assert not (o["top_ids"] == bad).any()
    # behind the mask it has no effect
    words = np.full((N, (V + 31) // 32), -1, np.int32)
    words[:, bad // 32] = ~(1 << (bad % 32))
    o = flce.constrained_logprobs(h, w, history=hist, repetition_penalty=torch.full((N,), 1.25, device=dev), top_k=3,
                                  mask=torch.from_numpy(words).to(dev), **kw)
    for k in ("lse", "entropy", "top_logp"):
        assert torch.isfinite(o[k]).all(), k
