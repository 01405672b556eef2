"""Pins of the oracles of the constrained log probabilities and the distillation
loss: torch fp64 autograd, hand-worked rows, central differences."""
import numpy as np
import pytest

from oracle.next_token_fp64 import constrained_oracle, distill_grad_oracle, distill_oracle, rules_oracle


def test_rules_by_hand():
    z = np.array([[2.0, -1.0, 4.0, 0.5, 3.0, 1.0]])
    hist = np.array([[0, 1, 2, 2, 9, -1, 2, 0]])
    r = rules_oracle(z, hist, np.array([7]), np.array([3]), [2.0], [0.25], [0.5], np.array([[4, 3, 4, 7]]),
                     np.array([[9.0, -np.inf, 1.0, 5.0]]), np.array([[True] * 5 + [False]]))
    # 0: prompt only; 1: negative, multiplied; 2: twice in the output (7 of 8 entries count); 4: the last bias holds
    np.testing.assert_array_equal(r, [[1.0, -2.0, 4.0 / 2 - 0.25 * 2 - 0.5, -np.inf, 4.0, -np.inf]])
    o = constrained_oracle(r, np.array([5]), top_k=6)
    assert o["logp"][0] == -np.inf
    assert o["top_ids"].tolist() == [[4, 0, 2, 1, -1, -1]]
    np.testing.assert_allclose(np.exp(o["all_logp"]).sum(), 1.0)


def test_a_row_with_nothing_left():
    o = constrained_oracle(np.full((1, 5), -np.inf), np.array([2]), top_k=2)
    assert o["lse"][0] == -np.inf and o["entropy"][0] == 0 and o["logp"][0] == -np.inf
    assert o["top_ids"].tolist() == [[-1, -1]] and np.isneginf(o["top_logp"]).all()


def problem(seed, N=6, H=5, V=17, K=4):
    r = np.random.default_rng(seed)
    X, W = r.standard_normal((N, H)), r.standard_normal((V, H))
    ids = np.array([r.permutation(V)[:K] for _ in range(N)])
    t = np.log(r.dirichlet(np.ones(K + 1), N)[:, :K])
    ids[1] = -1
    ids[2, 2] = -1
    ids[3, 1] = ids[3, 0]     # named twice
    t[4, 3] = -np.inf
    return X, W, ids, t


@pytest.mark.parametrize("tail", [True, False])
@pytest.mark.parametrize("T", [1.0, 1.7])
def test_distill_against_autograd(tail, T):
    import torch
    X, W, ids, t = problem(1)
    N, V = X.shape[0], W.shape[0]
    x, w = torch.tensor(X, requires_grad=True), torch.tensor(W, requires_grad=True)
    lq = torch.log_softmax(x @ w.T / T, 1)
    g = np.random.default_rng(2).standard_normal(N)
    total, kls = 0, []
    for n in range(N):
        p, listed = torch.zeros(V, dtype=torch.float64), torch.zeros(V, dtype=torch.bool)
        there = ids[n] >= 0
        masses = np.exp(t[n])[there]
        if not tail and there.any():
            masses = masses / masses.sum()
        for v, m in zip(ids[n][there], masses):
            p[v] += m
            listed[v] = True
        kl = torch.nn.functional.kl_div(lq[n], p, reduction="sum")
        if tail and there.any():
            r = 1 - p.sum()
            kl = kl + r * (torch.log(r) - torch.log(torch.exp(lq[n])[~listed].sum()))
        kls.append(float(kl.detach()))
        total = total + g[n] * kl
    total.backward()
    o, d = distill_oracle(X, W, ids, t, T, tail), distill_grad_oracle(X, W, ids, t, g, T, tail)
    np.testing.assert_allclose(o["kl"], kls, atol=1e-12)
    np.testing.assert_allclose(d["grad_hidden"], x.grad.numpy(), atol=1e-12)
    np.testing.assert_allclose(d["grad_weight"], w.grad.numpy(), atol=1e-12)


@pytest.mark.parametrize("tail", [True, False])
def test_distill_against_differences(tail):
    X, W, ids, t = problem(3)
    g = np.linspace(-1, 2, X.shape[0])
    d = distill_grad_oracle(X, W, ids, t, g, 0.8, tail)
    f = lambda A, B: (g * distill_oracle(A, B, ids, t, 0.8, tail)["kl"]).sum()  # noqa: E731
    for (A, name), at in [((X, "grad_hidden"), (2, 3)), ((X, "grad_hidden"), (0, 0)), ((W, "grad_weight"), (5, 1)),
                          ((W, "grad_weight"), (int(ids[0, 0]), 4))]:
        e = np.zeros_like(A)
        e[at] = 1e-6
        hi, lo = (f(A + e, W), f(A - e, W)) if A is X else (f(X, A + e), f(X, A - e))
        assert abs((hi - lo) / 2e-6 - d[name][at]) <= 1e-7 * (1 + abs(d[name][at]))


def test_distill_of_itself_is_nothing():
    X, W, ids, t = problem(4)
    z = X @ W.T
    lq = z - np.log(np.exp(z).sum(1, keepdims=True))
    ids = np.argsort(-lq, 1)[:, :4]
    own = np.take_along_axis(lq, ids, 1)
    o = distill_oracle(X, W, ids, own)
    np.testing.assert_allclose(o["kl"], 0, atol=1e-14)
    np.testing.assert_allclose(distill_grad_oracle(X, W, ids, own, np.ones(6))["dz"], 0, atol=1e-15)


def test_a_list_of_every_token():
    X, W, ids, t = problem(5, V=4)
    ids = np.tile(np.arange(4), (6, 1))
    o = distill_oracle(X, W, ids, np.log(np.full((6, 4), 0.25 - 1e-9)))
    assert (o["r"] == 0).all() and np.isneginf(o["rest_logp"]).all() and np.isfinite(o["kl"]).all()
