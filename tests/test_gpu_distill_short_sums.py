"""Divergences of short sums over H are as exact as an fp32 product makes them.

The tensor core cuts off what an fp32 accumulator cannot hold, always to the same side, so the logits of one piece of
3 and 4 K blocks were off by more than those of an fp32 product, whose roundings average out.  Pieces of two blocks at
most are not: the error stays within half as much again of the fp32 product's, over several problems (the ratio of
the two scatters with a problem's few largest rows), and what both have of roundings behind the logits, 2^-24 of the
divergence."""
import numpy as np
import pytest

from oracle.next_token_fp64 import distill_oracle
from tests.test_gpu_distill import env, np64, problem, to_gpu  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,H,V,K,T", [(600, 192, 2250, 8, 1.0), (600, 192, 2250, 2, 2.0), (600, 248, 2250, 8, 1.0),
                                       (600, 248, 2250, 2, 2.0), (64, 248, 2250, 8, 1.0), (128, 248, 2250, 8, 1.0)])
def test_no_worse_than_an_fp32_product(env, N, H, V, K, T):  # noqa: F811
    flce, torch, dev = env
    assert not torch.backends.cuda.matmul.allow_tf32
    mine = plain = size = 0.0
    for seed in range(6):
        X, W, ids, t = problem(N, H, V, K, seed, grid=False, T=T)
        h, w, i, tt = to_gpu(torch, dev, X, W, ids, t)
        ref = distill_oracle(X, W, ids, t, T)
        z = np64(h.float() @ w.float().T) / T
        # the same divergence of the fp32 product's logits, everything behind them in 64 bits
        lse = np.log(np.exp(z - z.max(1, keepdims=True)).sum(1, keepdims=True)) + z.max(1, keepdims=True)
        lq = z - lse
        p, r = ref["p"], ref["r"]
        rest = np.log(np.where(ref["listed"], 0.0, np.exp(lq)).sum(1))
        with np.errstate(divide="ignore", invalid="ignore"):
            kl = np.where(p > 0, p * (np.log(p) - lq), 0.0).sum(1) + np.where(r > 0, r * (np.log(r) - rest), 0.0)
        kl = np.where(ref["valid"], kl, 0.0)
        got = np64(flce.topk_distill(h, w, i, tt, temperature=T)["kl"])
        mine += np.square(got - ref["kl"]).sum()
        plain += np.square(kl - ref["kl"]).sum()
        size += np.square(ref["kl"]).sum()
    print("error", np.sqrt(mine / size), "of an fp32 product", np.sqrt(plain / size))
    assert np.sqrt(mine) <= 1.5 * np.sqrt(plain) + 2.0 ** -24 * np.sqrt(size), (mine / plain) ** 0.5
