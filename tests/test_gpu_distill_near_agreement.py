"""The divergence where student and teacher nearly agree: what is left of terms that cancel.

Tolerance (derived, before the first run), on logits that are exact, with x = (z -
max) / T, P = sum p, s the mass behind the list and ls = ln sum exp x:
  the terms p (t - x): each is rounded to 2^-24 of itself three times (the difference,
    the product, p: the same p weighs ls, so that p's own error, 2^-22, counts for
    p |log p - log q| only), and is added up in K / 32 + 5 steps, each off by 2^-24
    of the sum of their magnitudes;
  ls: the listed part of the sum by expf (2^-22) and K / 32 + 6 additions, its
    logarithm by 2^-23 of |ln f| < 0.7; P, which it is weighed with, is added up in
    K / 32 + 5 steps;
  the mass behind the list, off by 4e-5 of itself (see test_gpu_distill.py), moves kl
    by A s - r times that, which is nothing where the two agree;
  r: 1 - p_max - the others, off by 2^-22 + (K / 32 + 5) 2^-24, times |log r - log s| + 1,
    and its term, rounded twice;
  and kl itself once.
What all log probabilities share must not be rounded: with logits of 2048 an fp32
log-sum-exp is off by up to 2^-13, which the tolerance does not leave room for.
"""
import numpy as np
import pytest

from oracle.next_token_fp64 import distill_oracle
from tests.test_gpu_distill import env, np64, to_gpu  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu


def agreeing(N, V, K, far, shift, seed):
    """A teacher that is the student with its hidden states moved by `far`; all logits moved by `shift`."""
    H = 64
    r = np.random.default_rng(seed)
    std = 1.28 / np.sqrt(H)
    X, W = r.standard_normal((N, H)), std * r.standard_normal((V, H))
    X += W[r.integers(0, V, N)] * (10 * r.random((N, 1)) / (H * std * std))
    step = 2.0 ** np.round(np.log2(std / 10))
    X, W = np.clip(np.round(X * 16), -64, 64) / 16, np.clip(np.round(W / step), -63, 63) * step
    X[:, 0], W[:, 0] = 64.0, shift / 64.0
    move = far * r.standard_normal((N, H))
    move[:, 0] = 0
    z = (X + move) @ W.T
    ids = np.argsort(-z, 1)[:, :K].astype(np.int32)
    top = z.max(1, keepdims=True)
    lp = z - top - np.log(np.exp(z - top).sum(1, keepdims=True))
    return X, W, ids, np.take_along_axis(lp, ids, 1).astype(np.float32)


def tolerance(X, W, ids, t, tail, ref):
    K, u = ids.shape[1], 2.0 ** -24
    z = X @ W.T
    x = np.take_along_axis(z - z.max(1, keepdims=True), ids, 1)
    p, lq = np.take_along_axis(ref["p"], ids, 1), np.take_along_axis(ref["lq"], ids, 1)
    with np.errstate(divide="ignore"):
        lp = np.where(p > 0, np.log(p), 0.0)
    add = K / 32 + 5
    terms = ((add + 3) * u * p * np.abs(lp - x) + 4 * u * p * np.abs(lp - lq)).sum(1)
    if not tail:   # p renormalised: its shift is rounded, and off by what its sum is
        terms += p.sum(1) * (u * np.abs(np.where(p > 0, t, 0)).max(1) + (4 + add) * u)
    ls = ref["mass"] * ((4 + add + 1) * u + 2 * u) + p.sum(1) * add * u * np.abs(ref["lse"] - z.max(1))
    s = np.exp(ref["rest_logp"])
    behind = np.abs(ref["mass"] * s - ref["r"]) * 4e-5 if tail else p.sum(1) * s * 4e-5
    with np.errstate(divide="ignore", invalid="ignore"):
        gap = np.where(ref["r"] > 0, np.abs(np.log(ref["r"]) - ref["rest_logp"]), 0.0)
        far = np.where(ref["r"] > 0, np.abs(ref["rest_logp"]) + np.log(X.shape[0] + 1e9), 0.0)
    r = (4 + add) * u * (gap + 1) + 4 * u * ref["r"] * (gap + far) if tail else 0.0
    return terms + ls + behind + r + 2 * u * np.abs(ref["kl"])


def plain32(X, W, ids, t, tail):
    f = np.float32
    z = (X @ W.T).astype(f)
    m = z.max(1, keepdims=True)
    lse = (m + np.log(np.exp(z - m, dtype=f).sum(1, keepdims=True, dtype=f))).astype(f)
    lq = (np.take_along_axis(z, ids, 1) - lse).astype(f)
    if not tail:
        e = np.exp(t - t.max(1, keepdims=True), dtype=f)
        p = e / e.sum(1, keepdims=True, dtype=f)
        return (p * (np.log(p) - lq)).sum(1, dtype=f).astype(float)
    p = np.exp(t, dtype=f)
    r, s = (np.maximum(f(1e-30), f(1) - q.sum(1, dtype=f)) for q in (p, np.exp(lq, dtype=f)))
    return ((p * (t - lq)).sum(1, dtype=f) + r * (np.log(r) - np.log(s))).astype(float)


@pytest.mark.parametrize("tail", [True, False])
@pytest.mark.parametrize("far", [0.1, 0.02, 0.0])
@pytest.mark.parametrize("N,V,K", [(40, 4000, 20), (300, 4000, 20), (100, 700, 200), (300, 700, 200)])
def test_near_agreement(env, N, V, K, far, tail):  # noqa: F811
    flce, torch, dev = env
    for shift in (0.0, 2048.0):
        X, W, ids, t = agreeing(N, V, K, far, shift, N + K)
        ref = distill_oracle(X, W, ids, t, 1.0, tail)
        tol = tolerance(X, W, ids, t, tail, ref)
        o = flce.topk_distill(*to_gpu(torch, dev, X, W, ids, t), tail=tail)
        err = np.abs(np64(o["kl"]) - ref["kl"])
        print(far, tail, shift, "median kl", np.median(ref["kl"]), "error", np.median(err), err.max(), "tolerance", np.median(tol))
        assert np.all(err <= tol), (shift, (err / tol).max())
        if shift and not tail:   # a log-sum-exp of 2048 in fp32 is not enough (with a tail its error nearly cancels)
            assert np.mean(np.abs(plain32(X, W, ids, t, tail) - ref["kl"]) > tol) > 0.3
        if far == 0.1:
            assert np.median(tol) < 0.05 * np.median(ref["kl"])
