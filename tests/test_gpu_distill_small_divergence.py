"""Divergences far below the terms that they are what is left of keep their digits.

Tolerance (derived, before the first run), on logits that are exact and temperatures
that are powers of two, so that x = (z - max) / T is exact too.  To the first order
kl changes with the masses w by p (log p - log q) + 1 each where they add up to 1, with
the listed part of the sum of exponentials by itself, with every logarithm by its
weight, and with the mass s behind the list by A s - r.  Exponentials and logarithms
are held to 2.2e-9 (2^-28.8; an fp32 value and its remainder), sums to far less, r to
that and 2^-28 (the largest mass near 1), s to 4e-5 (as in test_gpu_distill.py):
  2.2e-9 (sum p |log p - log q| + P (2 + |log r - log s|) + A + 2 r) + 2^-28 + 4e-5 |A s - r|
and kl is rounded to fp32 once, 2^-24 of it.
"""
import numpy as np
import pytest

from oracle.next_token_fp64 import distill_oracle
from tests.test_gpu_distill import env, np64, to_gpu  # noqa: F401 (fixture)
from tests.test_gpu_distill_near_agreement import agreeing

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1.0, 2.0])
@pytest.mark.parametrize("far", [0.05, 0.0])
@pytest.mark.parametrize("N,V,K,tail", [(40, 4000, 2, True), (300, 4000, 2, True), (40, 4000, 20, True), (300, 4000, 20, True),
                                        (100, 700, 200, True), (300, 700, 200, True), (40, 60, 60, False),
                                        (300, 150, 150, False), (300, 60, 60, True)])
def test_small_divergence(env, N, V, K, tail, far, T):  # noqa: F811
    flce, torch, dev = env
    for shift in (0.0, 2048.0):
        X, W, ids, t = agreeing(N, V, K, far, shift, N + K)
        if T != 1.0:   # the teacher at that temperature
            move = far * np.random.default_rng(3).standard_normal(X.shape)
            move[:, 0] = 0
            z = (X + move) @ W.T / T
            top = z.max(1, keepdims=True)
            lp = z - top - np.log(np.exp(z - top).sum(1, keepdims=True))
            ids = np.argsort(-z, 1)[:, :K].astype(np.int32)
            t = np.take_along_axis(lp, ids, 1).astype(np.float32)
        ref = distill_oracle(X, W, ids, t, T, tail)
        p, r, s, A = ref["p"], ref["r"], np.exp(ref["rest_logp"]), ref["mass"]
        with np.errstate(divide="ignore", invalid="ignore"):
            own = np.where(p > 0, p * np.abs(np.log(p) - ref["lq"]), 0.0).sum(1)
            gap = np.where(r > 0, np.abs(np.log(r) - ref["rest_logp"]), 0.0)
        tol = 2.2e-9 * (own + p.sum(1) * (2 + gap) + A + 2 * r) + 2.0 ** -28 + 4e-5 * np.abs(A * s - r) * (r > 0)
        tol += 2.0 ** -24 * np.abs(ref["kl"])
        o = flce.topk_distill(*to_gpu(torch, dev, X, W, ids, t), temperature=T, tail=tail)
        err = np.abs(np64(o["kl"]) - ref["kl"])
        print(tail, far, T, shift, "median kl", np.median(ref["kl"]), "error", np.median(err), err.max(), "tolerance",
              np.median(tol), "worst", (err / tol).max())
        assert np.all(err <= tol), (shift, (err / tol).max())
