"""fp64 CPU oracle of the token log probabilities, their gradient, and the
scaled embedding with its gradient.  TEST INFRASTRUCTURE ONLY, as flce_fp64.

Plain definitions with numpy, no code shared with the CUDA path:

  z = X W^T / T, m_n = max_v z_nv, lse_n = m_n + log sum_v exp(z_nv - m_n)
  logp_n = z_{n,t_n} - lse_n,  entropy_n = -sum_v p_nv log p_nv, p = exp(z - lse)
  top: the K largest z_nv - lse_n, equal ones by the lower id
  dz_nv = (g_n ([v = t_n] - p_nv) - e_n p_nv (log p_nv + entropy_n)) / T
  grad_hidden = dz W, grad_weight = dz^T X
Rows whose target is the ignore index hold zeros (ids -1).
"""
from __future__ import annotations

import numpy as np


def logprobs_oracle(X, W, t, ignore_index=-100, temperature=1.0, top_k=0):
    X, W = np.asarray(X, np.float64), np.asarray(W, np.float64)
    N = X.shape[0]
    valid = np.asarray(t) != ignore_index
    z = X @ W.T / temperature
    m = z.max(axis=1, keepdims=True)
    lse = m + np.log(np.exp(z - m).sum(axis=1, keepdims=True))
    lp = z - lse
    p = np.exp(lp)
    ent = -(p * lp).sum(axis=1)
    at = np.where(valid, t, 0)
    r = {"logp": np.where(valid, lp[np.arange(N), at], 0.0), "lse": np.where(valid, lse[:, 0], 0.0),
         "entropy": np.where(valid, ent, 0.0), "all_logp": lp, "valid": valid}
    if top_k:
        order = np.argsort(-z, axis=1, kind="stable")[:, :top_k]
        r["top_ids"] = np.where(valid[:, None], order, -1)
        r["top_logp"] = np.where(valid[:, None], np.take_along_axis(lp, order, 1), 0.0)
    return r


def logprobs_grad_oracle(X, W, t, g, e, ignore_index=-100, temperature=1.0):
    """Gradients, and elementwise sums of magnitudes that rounding bounds scale with."""
    X, W = np.asarray(X, np.float64), np.asarray(W, np.float64)
    f = logprobs_oracle(X, W, t, ignore_index, temperature)
    lp, valid = f["all_logp"], f["valid"]
    p = np.exp(lp)
    g = np.where(valid, np.zeros(len(t)) if g is None else np.asarray(g, np.float64), 0.0)[:, None]
    e = np.where(valid, np.zeros(len(t)) if e is None else np.asarray(e, np.float64), 0.0)[:, None]
    H = f["entropy"][:, None]
    onehot = np.zeros_like(lp)
    onehot[np.arange(len(t))[valid], np.asarray(t)[valid]] = 1.0
    dz = (g * (onehot - p) - e * p * (lp + H)) / temperature
    mag = (np.abs(g) * (onehot + p) + np.abs(e) * p * (np.abs(lp) + H)) / temperature
    return {"grad_hidden": dz @ W, "grad_weight": dz.T @ X, "mag_hidden": mag @ np.abs(W),
            "mag_weight": mag.T @ np.abs(X)}


def embedding_oracle(W, ids, scale=1.0):
    return np.asarray(W, np.float64)[np.asarray(ids)] * scale


def embedding_grad_oracle(dout, ids, V, scale=1.0, padding_idx=None):
    """Gradient and, per element, the sum of the magnitudes added."""
    dout = np.asarray(dout, np.float64)
    g = np.zeros((V, dout.shape[1]))
    mag = np.zeros_like(g)
    for n, v in enumerate(np.asarray(ids)):
        if padding_idx is None or v != padding_idx:
            g[v] += scale * dout[n]
            mag[v] += abs(scale) * np.abs(dout[n])
    return g, mag
