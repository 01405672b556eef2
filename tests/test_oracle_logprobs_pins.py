"""Pins of the fp64 oracle of the token log probabilities and the embedding:
autograd in fp64 of the definitions, central differences, closed forms."""
import numpy as np
import pytest

from oracle.logprobs_fp64 import (embedding_grad_oracle, embedding_oracle, logprobs_grad_oracle, logprobs_oracle)

torch = pytest.importorskip("torch")


def problem(N, H, V, seed, ignored=0.2):
    r = np.random.default_rng(seed)
    t = r.integers(0, V, N)
    t[r.random(N) < ignored] = -100
    return r.standard_normal((N, H)), 0.3 * r.standard_normal((V, H)), t, r.standard_normal(N), r.standard_normal(N)


@pytest.mark.parametrize("N,H,V,T", [(7, 5, 11, 1.0), (4, 16, 3, 0.7), (1, 8, 1, 2.0)])
def test_against_autograd(N, H, V, T):
    X, W, t, g, e = problem(N, H, V, seed=N)
    x, w = torch.tensor(X, requires_grad=True), torch.tensor(W, requires_grad=True)
    q = torch.distributions.Categorical(logits=x @ w.T / T)
    keep = torch.tensor(t != -100)
    tt = torch.tensor(np.where(t == -100, 0, t))
    logp, ent = q.log_prob(tt) * keep, q.entropy() * keep
    (logp @ torch.tensor(g) + ent @ torch.tensor(e)).backward()
    o, d = logprobs_oracle(X, W, t, temperature=T), logprobs_grad_oracle(X, W, t, g, e, temperature=T)
    np.testing.assert_allclose(o["logp"], logp.detach(), atol=1e-12)
    np.testing.assert_allclose(o["entropy"], ent.detach(), atol=1e-12)
    np.testing.assert_allclose(d["grad_hidden"], x.grad, atol=1e-12)
    np.testing.assert_allclose(d["grad_weight"], w.grad, atol=1e-12)


def test_against_central_differences():
    X, W, t, g, e = problem(5, 6, 9, seed=3)

    def L(X, W):
        o = logprobs_oracle(X, W, t, temperature=0.8)
        return o["logp"] @ g + o["entropy"] @ e

    d = logprobs_grad_oracle(X, W, t, g, e, temperature=0.8)
    h = 1e-6
    for a, name in ((X, "grad_hidden"), (W, "grad_weight")):
        for i in np.ndindex(a.shape):
            keep = a[i]
            a[i] = keep + h
            up = L(X, W)
            a[i] = keep - h
            down = L(X, W)
            a[i] = keep
            assert abs((up - down) / (2 * h) - d[name][i]) < 1e-7


def test_closed_forms():
    X, t = np.random.default_rng(0).standard_normal((3, 4)), np.array([2, -100, 0])
    o = logprobs_oracle(X, np.zeros((8, 4)), t, top_k=3)
    np.testing.assert_allclose(o["logp"], [-np.log(8), 0, -np.log(8)], atol=1e-15)
    np.testing.assert_allclose(o["entropy"], [np.log(8), 0, np.log(8)], atol=1e-14)
    assert o["top_ids"].tolist() == [[0, 1, 2], [-1, -1, -1], [0, 1, 2]]   # equal logits: lowest ids first


def test_embedding_against_torch():
    r = np.random.default_rng(1)
    W, ids, dout = r.standard_normal((10, 4)), np.array([3, 3, 9, 0, 3, 2]), r.standard_normal((6, 4))
    w = torch.tensor(W, requires_grad=True)
    out = 2.5 * torch.nn.functional.embedding(torch.tensor(ids), w, padding_idx=2)
    out.backward(torch.tensor(dout))
    np.testing.assert_allclose(embedding_oracle(W, ids, 2.5), out.detach(), atol=1e-14)
    np.testing.assert_allclose(embedding_grad_oracle(dout, ids, 10, 2.5, padding_idx=2)[0], w.grad, atol=1e-13)
