"""A list taken as the whole distribution may be logits: what they share takes no part.

The entries and what is added to all of them are multiples of 1/64 below 2^13, so that every one of them, and every
difference of two, is exact in fp32: the same masses, and so the same results bit for bit."""
import numpy as np
import pytest

from oracle.next_token_fp64 import distill_grad_oracle, distill_oracle
from tests.test_gpu_distill import check, check_gradients, env, np64, problem, to_gpu  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shift", [37.0, -512.0, 4096.0])
@pytest.mark.parametrize("N,V,K,T", [(40, 900, 20, 1.0), (300, 900, 20, 0.5), (100, 60, 60, 1.0), (300, 300, 150, 1.0)])
def test_shifted_logits(env, N, V, K, T, shift):  # noqa: F811
    flce, torch, dev = env
    X, W, ids, t = problem(N, 64, V, K, N + K, T=T)
    t = np.where(np.isinf(t), t, np.round(t * 64) / 64).astype(np.float32)
    g = np.random.default_rng(1).standard_normal(N).astype(np.float32)
    outs = []
    for s in (0.0, shift):
        a = to_gpu(torch, dev, X, W, ids, (t + np.float32(s)).astype(np.float32))
        o = flce.topk_distill(*a, temperature=T, tail=False)
        d = flce.topk_distill_bwd(*a, o["lse"], o["rest_logp"], o["student_logp"], torch.from_numpy(g).to(dev), temperature=T,
                                  tail=False)
        outs.append((o, d))
        check(o, distill_oracle(X, W, ids, t, T, False))
        check_gradients(d, distill_grad_oracle(X, W, ids, t, g, T, False), False)
    (o, d), (p, e) = outs
    for k in ("kl", "lse", "rest_logp", "student_logp"):
        assert torch.equal(o[k], p[k]), k
    for k in ("grad_hidden", "grad_weight"):
        assert torch.equal(d[k], e[k]), k


@pytest.mark.parametrize("N", [60, 300])
def test_unlikely_tokens_only(env, N):  # noqa: F811
    """A list without a teacher's likeliest tokens: log probabilities far below 0, which the masses are normalised from."""
    flce, torch, dev = env
    X, W, ids, t = problem(N, 64, 40, 40, 3, T=0.25, ignored=0.0)
    t = (t - 100).astype(np.float32)
    o = flce.topk_distill(*to_gpu(torch, dev, X, W, ids, t), temperature=0.25, tail=False)
    ref = distill_oracle(X, W, ids, t, 0.25, False)
    # the bound of test_gpu_distill.py's check, without its 4e-5 of the mass: every token is listed, so the sum of
    # exponentials is expf's (2^-22) and K / 32 + 6 additions
    tol = ref["mass"] * (2.0 ** -22 + 8 * 2.0 ** -24) + 2.0 ** -21 * (ref["size"] + 1)
    err = np.abs(np64(o["kl"]) - ref["kl"])
    assert np.all(err <= tol), (err / tol).max()
