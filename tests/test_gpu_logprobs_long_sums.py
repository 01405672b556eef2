"""Log probabilities at large hidden sizes: a logit's sum over H is taken in segments.

The tensor core cuts off what its fp32 accumulator cannot hold at every 16-wide
step.  A step of a segment of L blocks of 64 cuts half a unit (2^-24 of the
partial sum) on average, always towards zero, and the partial sums are half of
the segment's on average: 4 L steps come to L 2^-24 of the logit.  The norm of a
row's errors in log probabilities and entropies is allowed twice that, with 3e-7
for the softmax, as in test_gpu_logprobs.py.  In one piece, L is H / 64 (4.8e-6
to 2.2e-5 of entropies at H = 4096 to 16384).
On grid inputs every partial sum is exact, so segments change nothing.
"""
import math

import numpy as np
import pytest

from oracle.logprobs_fp64 import logprobs_grad_oracle, logprobs_oracle
from tests.test_gpu_logprobs import check_forward, env, np64, problem, to_gpu  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu


def segment(H):
    """Blocks of a segment, as the library cuts them."""
    blocks = -(-H // 64)
    most = max(11, int(2 * math.sqrt(blocks)))
    return -(-blocks // -(-blocks // most))


def continuous(torch, dev, N, H, V, seed):
    """Inputs whose sums of products round: logits of deviation 1.28, some tokens likely."""
    r = torch.Generator(device=dev).manual_seed(seed)
    std = 1.28 / math.sqrt(H)
    w = torch.randn(V, H, generator=r, device=dev) * std
    t = torch.randint(0, V, (N,), generator=r, device=dev, dtype=torch.int32)
    lift = 14 * torch.rand(N, 1, generator=r, device=dev) / (H * std * std)
    x = torch.randn(N, H, generator=r, device=dev) + w[t.long()] * lift
    return x.to(torch.bfloat16), w.to(torch.bfloat16), t


@pytest.mark.parametrize("N", [16, 64, 128, 300])
@pytest.mark.parametrize("H,V", [(2048, 20011), (4096, 20011), (8192, 5003), (16384, 5003)])
def test_error_does_not_grow_with_the_sum(env, N, H, V):  # noqa: F811
    flce, torch, dev = env
    x, w, t = continuous(torch, dev, N, H, V, N + H)
    o = flce.token_logprobs(x, w, t)
    lp = torch.log_softmax(x.double() @ w.double().T, 1)
    want = {"logp": lp.gather(1, t.long()[:, None])[:, 0], "entropy": -(lp.exp() * lp).sum(1)}
    for k, v in want.items():
        err = float((o[k].double() - v).norm() / v.norm())
        assert err <= 2 * segment(H) * 2.0 ** -24 + 3e-7, (k, err)


SHAPES = [  # N, H, V, K: one segment of 11 blocks, two of 6, an odd last one, equal ones, many; K with and without a bound
    (1, 704, 3001, 5), (17, 712, 1000, 32), (33, 776, 40003, 4), (64, 1032, 2050, 7), (100, 2056, 515, 3),
    (128, 4104, 1200, 16), (128, 712, 20003, 8), (3, 16392, 300, 2), (300, 704, 515, 5), (300, 712, 1000, 0),
    (700, 1032, 4099, 12), (260, 4104, 300, 32), (200, 776, 40003, 4), (513, 2056, 3079, 8), (129, 16392, 190, 9),
    (1030, 1288, 130, 1), (300, 712, 64, 3), (300, 712, 65, 3), (300, 712, 1, 1)]


@pytest.mark.parametrize("N,H,V,K", SHAPES)
def test_exact_sums(env, N, H, V, K):  # noqa: F811
    flce, torch, dev = env
    X, W, t = problem(N, H, V, seed=N + H, ignored=0.1)
    o = flce.token_logprobs(*to_gpu(torch, dev, X, W, t), temperature=0.8, top_k=K)
    assert flce.query_status(o["workspace"]) == flce.FLCE_OK
    check_forward(o, logprobs_oracle(X, W, t, temperature=0.8, top_k=K), 0.8, K)


@pytest.mark.parametrize("N", [20, 200])
def test_extreme_rows(env, N):  # noqa: F811
    """Rows with NaN and inf, and logits of -inf beside ordinary ones, as with short sums."""
    flce, torch, dev = env
    X, W, t = problem(N, 1032, 600, seed=9)
    X[:, 7] = 1
    t[t == 5] = 6
    h, w, tt = to_gpu(torch, dev, X, W, t)
    w[5] = 0
    w[5, 7] = float("-inf")   # one logit of -inf in every row
    h[2, 1000] = float("nan")
    h[3, 5] = float("inf")
    o = flce.token_logprobs(h, w, tt, top_k=5)
    assert all(torch.isnan(o[k][2:4]).all() for k in ("logp", "lse", "entropy"))
    keep = np.array([i for i in range(N) if i not in (2, 3)])
    rest = np.delete(np.arange(600), 5)
    tk = t[keep] - (t[keep] > 5)
    ref = logprobs_oracle(X[keep], W[rest], tk, top_k=5)
    ref["top_ids"] = rest[ref["top_ids"]]
    got = {k: o[k][torch.from_numpy(keep).to(dev)] for k in ("logp", "lse", "entropy", "top_ids", "top_logp")}
    check_forward(got, ref, 1.0, 5)


@pytest.mark.parametrize("N,H,V", [(300, 776, 2049), (140, 4104, 513), (513, 2056, 1000), (20, 1032, 130)])
@pytest.mark.parametrize("grid", [True, False])
def test_gradients(env, N, H, V, grid):  # noqa: F811
    flce, torch, dev = env
    X, W, t = problem(N, H, V, seed=N, ignored=0.1, grid=grid)
    r = np.random.default_rng(1)
    g, e = (r.standard_normal(N).astype(np.float32) for _ in range(2))
    h, w, tt = to_gpu(torch, dev, X, W, t)
    o = flce.token_logprobs(h, w, tt, temperature=0.9)
    d = flce.token_logprobs_bwd(h, w, tt, o["lse"], o["entropy"], *(torch.from_numpy(a).to(dev) for a in (g, e)),
                                temperature=0.9, grad_weight_dtype=torch.bfloat16)
    assert flce.query_status(d["workspace"]) == flce.FLCE_OK
    ref = logprobs_grad_oracle(X, W, t, g, e, temperature=0.9)
    for k in ("hidden", "weight"):   # as in test_gpu_logprobs.py
        tol = ref["mag_" + k] * (2.0 ** -8 + 2e-4) * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref["grad_" + k])
        err = np.abs(np64(d["grad_" + k]) - ref["grad_" + k])
        assert np.all(err <= tol + 1e-30), (k, (err / (tol + 1e-30)).max())


@pytest.mark.parametrize("N", [100, 300])
def test_captured_and_on_two_streams(env, N):  # noqa: F811
    """Replays on new inputs, and two calls at once, are bitwise the eager calls."""
    flce, torch, dev = env
    H, V, K = 1032, 3000, 4
    probs = [continuous(torch, dev, N, H, V, s) for s in (1, 2)]
    g = torch.randn(N, device=dev)

    def both(h, w, t, stream=None):
        o = flce.token_logprobs(h, w, t, top_k=K, stream=stream)
        d = flce.token_logprobs_bwd(h, w, t, o["lse"], o["entropy"], g, g, stream=stream)
        return [o[k] for k in ("logp", "entropy", "lse", "top_ids", "top_logp")] + [d["grad_hidden"], d["grad_weight"]]

    want = [both(*p) for p in probs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = [both(*p, stream=s) for p, s in zip(probs, streams)]
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    h, w, t = (x.clone() for x in probs[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both(h, w, t)
    for p, a in ((probs[1], want[1]), (probs[0], want[0])):
        for x, y in zip((h, w, t), p):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, a))


@pytest.mark.parametrize("K", [0, 3, 32])
def test_chunks(env, K):  # noqa: F811
    """Chunks of 128 tokens give the values of one chunk, with and without a bound of the alternatives."""
    flce, torch, dev = env
    N, H, V = 500, 776, 20003
    h, w, t = continuous(torch, dev, N, H, V, 3)
    whole = flce.token_logprobs(h, w, t, top_k=K)
    # a chunk of 128: its fp32 logits where there are alternatives, the statistics, its rows
    nb = (128 * (V + 64) * 4 if K else 0) + 128 * 160 * 12 + 128 * H * 2 + (1 << 16)
    part = flce.token_logprobs(h, w, t, top_k=K, workspace=torch.full((nb,), 255, dtype=torch.uint8, device=dev))
    for k in ("logp", "lse", "entropy") + (("top_ids", "top_logp") if K else ()):
        assert torch.equal(whole[k], part[k]), k
