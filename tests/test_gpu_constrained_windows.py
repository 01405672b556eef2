"""Masks, histories and biases on both sides of a bitmap window's edge (131072 tokens where a call has more than 128
rows, 262144 otherwise), against the fp64 oracle."""
import numpy as np
import pytest

from oracle.next_token_fp64 import constrained_oracle, rules_oracle
from tests.test_gpu_constrained import check, env, head, pack, to_kw  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("L", [200, 1500])
@pytest.mark.parametrize("N,V,edge", [(130, 140003, 131072), (130, 262177, 131072), (2, 270001, 262144), (128, 270001, 262144)])
def test_both_sides_of_a_window(env, N, V, edge, L):  # noqa: F811
    flce, torch, dev = env
    X, W = head(N, 8, V, 12)
    r = np.random.default_rng(N + L)
    near = np.concatenate([np.arange(edge - 40, min(edge + 40, V)), np.arange(V - 5, V), [0, 31, 32]])
    hist = np.where(r.random((N, L)) < 0.5, r.choice(near, (N, L)), r.integers(0, V, (N, L))).astype(np.int32)
    allowed = r.random((N, V)) < r.choice([0.02, 0.5, 1.0], N)[:, None]
    allowed[:, near] = r.random((N, len(near))) < 0.5
    bias_ids = np.tile(np.array([edge - 1, edge, V - 1, 5], np.int32), (N, 1))
    bias = (8 + r.standard_normal((N, 4))).astype(np.float32)
    k = dict(history=hist, history_lens=r.integers(L // 2, L + 1, N).astype(np.int32),
             prompt_lens=r.integers(0, L // 2, N).astype(np.int32), repetition=np.full(N, 1.25, np.float32),
             frequency=np.full(N, 0.125, np.float32), presence=np.full(N, 0.25, np.float32), bias_ids=bias_ids, bias=bias,
             allowed=allowed)
    rows = [0, 1, N // 2, N - 1]
    t = np.full(N, edge, np.int32)
    t[rows[1]] = edge - 1
    f = lambda a: torch.from_numpy(a).to(torch.bfloat16).to(dev)  # noqa: E731
    o = flce.constrained_logprobs(f(X), f(W), torch.from_numpy(t).to(dev), top_k=6, **to_kw(torch, dev, k))
    assert flce.query_status(o["workspace"]) == flce.FLCE_OK
    kk = {n: a[rows] for n, a in k.items()}
    ref = constrained_oracle(rules_oracle(X[rows] @ W.T, **kk), t[rows], top_k=6)
    # 2110 parts at most: (128 + 2110 / 32) 2^-24 of merges in sequence, and as many 2^-22 of their factors: 6e-5
    check({n: o[n][rows] for n in ("logp", "lse", "entropy", "top_ids", "top_logp")}, ref, 6, True, 8e-5)
