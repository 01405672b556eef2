"""fp64 CPU oracles of the constrained log probabilities and of the distillation
from a teacher's list, with its gradient.  TEST INFRASTRUCTURE ONLY.

Plain definitions with numpy, no code shared with the CUDA path:

  z = X W^T, then per row: repetition, frequency and presence penalties, biases
  and mask (each step rounded to fp32, as the operator defines it), and the
  log probabilities of z / T
  kl = sum_I p (log p - log q) + r (log r - log s), q = softmax(X W^T / T)
  dz = g (A q - p - [v not in I] r q / s) / T, A = sum p + r
"""
from __future__ import annotations

import numpy as np


def rules_oracle(z, history=None, history_lens=None, prompt_lens=None, repetition=None, frequency=None, presence=None,
                 bias_ids=None, bias=None, allowed=None):
    """The logits [N, V] (exact in fp32) under the rules, in fp32 steps."""
    z = np.asarray(z).astype(np.float32)
    assert np.array_equal(z, np.asarray(z, np.float32))
    N, V = z.shape
    out = z.copy()
    f32 = np.float32
    for n in range(N):
        if history is not None:
            L = history.shape[1]
            length = L if history_lens is None else min(max(int(history_lens[n]), 0), L)
            prompt = 0 if prompt_lens is None else int(prompt_lens[n])
            count = {}
            for i in range(length):
                v = int(history[n, i])
                if 0 <= v < V:
                    count[v] = count.get(v, 0) + (1 if i >= prompt else 0)
            for v, c in count.items():
                x = out[n, v]
                if repetition is not None:
                    x = f32(x / f32(repetition[n])) if x > 0 else f32(x * f32(repetition[n]))
                if c > 0:
                    if frequency is not None:
                        x = f32(x - f32(f32(frequency[n]) * f32(c)))
                    if presence is not None:
                        x = f32(x - f32(presence[n]))
                out[n, v] = x
        if bias_ids is not None:
            named = {int(v): j for j, v in enumerate(bias_ids[n])}   # the last entry holds
            for v, j in named.items():
                if 0 <= v < V:
                    out[n, v] = f32(out[n, v] + f32(bias[n, j]))
        if allowed is not None:
            out[n, ~allowed[n]] = -np.inf
    return out


def constrained_oracle(z, t=None, ignore_index=-100, temperature=1.0, top_k=0):
    """Outputs of logits z [N, V] that are already under the rules."""
    zz = np.asarray(z, np.float64) / temperature
    N, V = zz.shape
    valid = np.ones(N, bool) if t is None else np.asarray(t) != ignore_index
    m = zz.max(1, keepdims=True)
    some = np.isfinite(m)
    with np.errstate(divide="ignore", invalid="ignore"):
        lse = np.where(some, m + np.log(np.exp(zz - np.where(some, m, 0.0)).sum(1, keepdims=True)), -np.inf)
        lp = np.where(np.isneginf(zz), -np.inf, zz - np.where(some, lse, 0.0))
        p = np.exp(lp)
        ent = -np.where(p > 0, p * lp, 0.0).sum(1)
    r = {"lse": np.where(valid, lse[:, 0], 0.0), "entropy": np.where(valid, ent, 0.0), "all_logp": lp, "valid": valid}
    if t is not None:
        r["logp"] = np.where(valid, lp[np.arange(N), np.where(valid, t, 0)], 0.0)
    if top_k:
        order = np.argsort(-np.asarray(z, np.float64), axis=1, kind="stable")[:, :top_k]
        best = np.take_along_axis(lp, order, 1)
        order = np.where(np.isneginf(best), -1, order)
        r["top_ids"] = np.where(valid[:, None], order, -1)
        r["top_logp"] = np.where(valid[:, None], best, 0.0)
    return r


def teacher_oracle(ids, logp, V, tail):
    """Dense masses [N, V], the mass behind the list [N], and which tokens are listed."""
    N, K = ids.shape
    p = np.zeros((N, V))
    listed = np.zeros((N, V), bool)
    r = np.zeros(N)
    for n in range(N):
        there = ids[n] >= 0
        if not there.any():
            continue
        t = np.asarray(logp[n], np.float64)[there]
        if tail:
            w = np.exp(t)
        else:
            top = t.max()
            e = np.exp(t - top) if np.isfinite(top) else np.zeros_like(t)
            w = e / e.sum() if e.sum() > 0 else e
        np.add.at(p[n], ids[n][there], w)
        listed[n, ids[n][there]] = True
        if tail and not listed[n].all():
            r[n] = max(0.0, 1.0 - w.sum())
    return p, r, listed


def distill_oracle(X, W, ids, logp, temperature=1.0, tail=True):
    X, W = np.asarray(X, np.float64), np.asarray(W, np.float64)
    N, V = X.shape[0], W.shape[0]
    valid = (ids >= 0).any(1)
    z = X @ W.T / temperature
    m = z.max(1, keepdims=True)
    lse = m + np.log(np.exp(z - m).sum(1, keepdims=True))
    lq = z - lse
    p, r, listed = teacher_oracle(ids, logp, V, tail)
    with np.errstate(divide="ignore", invalid="ignore"):
        behind = np.where(listed, -np.inf, z)
        bm = behind.max(1, keepdims=True)
        some = np.isfinite(bm)
        rest = np.where(some, bm + np.log(np.exp(behind - np.where(some, bm, 0)).sum(1, keepdims=True)) - lse, -np.inf)[:, 0]
        terms = np.where(p > 0, p * (np.log(p) - lq), 0.0)
        last = np.where(r > 0, r * (np.log(r) - np.where(r > 0, rest, 0.0)), 0.0)
    return {"kl": np.where(valid, terms.sum(1) + last, 0.0), "lse": np.where(valid, lse[:, 0], 0.0),
            "rest_logp": np.where(valid, rest, 0.0),
            "student_logp": np.where(ids >= 0, np.take_along_axis(lq, np.maximum(ids, 0), 1), 0.0),
            "size": np.where(valid, np.abs(terms).sum(1) + np.abs(last), 0.0), "mass": p.sum(1) + r, "p": p, "r": r,
            "listed": listed, "lq": lq, "valid": valid}


def distill_grad_oracle(X, W, ids, logp, g, temperature=1.0, tail=True):
    """Gradients, and elementwise sums of magnitudes that rounding bounds scale with."""
    X, W = np.asarray(X, np.float64), np.asarray(W, np.float64)
    f = distill_oracle(X, W, ids, logp, temperature, tail)
    q = np.exp(f["lq"])
    g = np.where(f["valid"], np.asarray(g, np.float64), 0.0)[:, None]
    s = np.where(f["listed"], 0.0, q).sum(1, keepdims=True)
    with np.errstate(divide="ignore", invalid="ignore"):
        behind = np.where(f["listed"], 0.0, np.where(s > 0, f["r"][:, None] * q / s, 0.0))
    A = f["mass"][:, None]
    dz = g * (A * q - f["p"] - behind) / temperature
    mag = np.abs(g) * (A * q + f["p"] + behind) / temperature
    return {"grad_hidden": dz @ W, "grad_weight": dz.T @ X, "dz": dz, "mag_hidden": mag @ np.abs(W),
            "mag_weight": mag.T @ np.abs(X)}
