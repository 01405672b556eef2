"""Gradients of the distillation loss keep what an fp32 dz has: nothing of it is lost to 16 bits.

Tolerances (derived, before the first run).  dz in fp32 is off by less than 2e-4 of
the sum of its terms' magnitudes (see test_gpu_distill.py).  Held as two bf16 parts
it loses at most half a step of the second one, 2^-8 of what the first leaves, so
2^-16 of itself; the products are exact in fp32 and their sum of n terms, each
cut off rather than rounded, is off by n 2^-23 of the sum of the magnitudes (n: the
tokens for grad_weight, the vocabulary for grad_hidden, in 16-wide steps and twice
for the parts).  A bf16 output is rounded once: half a step, 2^-8 of itself.
Together 2^-16 + 2e-4 + n / 8 * 2^-23 of the magnitudes; one bf16 part alone is off
by up to 2^-8 of dz, 4e-3.
"""
import numpy as np
import pytest

from oracle.next_token_fp64 import distill_grad_oracle
from tests.test_gpu_distill import env, np64, problem, to_gpu  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu

CASES = [  # N, H, V, K, T, tail
    (2, 64, 500, 1, 1.0, True), (2, 512, 3001, 8, 1.0, True), (17, 136, 1000, 5, 1.0, False), (63, 264, 2049, 20, 2.0, True),
    (128, 64, 512, 64, 1.0, True), (129, 72, 4000, 3, 0.7, True), (300, 64, 512, 8, 2.0, False), (450, 520, 999, 1, 1.0, False),
    (453, 256, 3000, 32, 1.0, True), (900, 64, 2000, 256, 1.0, True), (16500, 8, 300, 5, 1.0, True)]


def gradients(flce, torch, dev, X, W, ids, t, g, T, tail, **kw):
    a = to_gpu(torch, dev, X, W, ids, t)
    o = flce.topk_distill(*a, temperature=T, tail=tail)
    d = flce.topk_distill_bwd(*a, o["lse"], o["rest_logp"], o["student_logp"], torch.from_numpy(g).to(dev), temperature=T,
                              tail=tail, **kw)
    assert flce.query_status(d["workspace"]) == flce.FLCE_OK
    return d


def near(d, ref, N, V, bf16):
    for k, n, rounds in (("hidden", V, 1), ("weight", N, int(bf16))):
        if d["grad_" + k] is None:
            continue
        tol = ref["mag_" + k] * (2.0 ** -16 + 2e-4 + n / 8 * 2.0 ** -23) + rounds * 2.0 ** -8 * np.abs(ref["grad_" + k])
        err = np.abs(np64(d["grad_" + k]) - ref["grad_" + k])
        assert np.all(err <= tol + 1e-30), (k, (err / (tol + 1e-30)).max())


@pytest.mark.parametrize("N,H,V,K,T,tail", CASES)
@pytest.mark.parametrize("bf16", [False, True])
def test_as_exact_as_dz_in_32_bits(env, N, H, V, K, T, tail, bf16):  # noqa: F811
    flce, torch, dev = env
    X, W, ids, t = problem(N, H, V, K, N + K, T=T)
    g = np.random.default_rng(2).standard_normal(N).astype(np.float32)
    d = gradients(flce, torch, dev, X, W, ids, t, g, T, tail, grad_weight_dtype=torch.bfloat16 if bf16 else torch.float32)
    near(d, distill_grad_oracle(X, W, ids, t, g, T, tail), N, V, bf16)


@pytest.mark.parametrize("side", ["hidden", "weight"])
@pytest.mark.parametrize("N", [40, 300])
def test_one_side_alone(env, N, side):  # noqa: F811
    flce, torch, dev = env
    X, W, ids, t = problem(N, 200, 1500, 12, 5)
    g = np.random.default_rng(3).standard_normal(N).astype(np.float32)
    d = gradients(flce, torch, dev, X, W, ids, t, g, 1.0, True, need_hidden=side == "hidden", need_weight=side == "weight")
    near(d, distill_grad_oracle(X, W, ids, t, g), N, 1500, False)


def test_in_chunks(env):  # noqa: F811
    """The smallest workspace that is taken, and one of a few chunks: as exact, and nothing behind it written."""
    flce, torch, dev = env
    N, H, V, K = 700, 136, 1000, 12
    X, W, ids, t = problem(N, H, V, K, 3)
    g = np.random.default_rng(1).standard_normal(N).astype(np.float32)
    a = to_gpu(torch, dev, X, W, ids, t)
    o = flce.topk_distill(*a)
    args = (*a, o["lse"], o["rest_logp"], o["student_logp"], torch.from_numpy(g).to(dev))
    ref = distill_grad_oracle(X, W, ids, t, g)
    for bf16 in (False, True):
        kw = {"grad_weight_dtype": torch.bfloat16 if bf16 else torch.float32}
        lo, hi = 0, flce.library().flce_topk_distill_bwd_workspace_bytes(N, H, V, K, 2 if bf16 else 0)
        top = hi
        near(flce.topk_distill_bwd(*args, **kw), ref, N, V, bf16)
        while hi - lo > 256:
            mid = (lo + hi) // 2
            try:
                flce.topk_distill_bwd(*args, workspace=flce.new_workspace(mid, dev), **kw)
                hi = mid
            except flce.FlceError as e:
                assert e.status == flce.FLCE_EWORKSPACE
                lo = mid
        assert hi < top
        for size in (hi, (hi + top) // 2):
            ws = torch.full((size + 512,), 171, dtype=torch.uint8, device=dev)
            d = flce.topk_distill_bwd(*args, workspace=ws[:size], **kw)
            assert (ws[size:] == 171).all()
            near(d, ref, N, V, bf16)
            assert not d["grad_hidden"][torch.from_numpy((ids < 0).all(1)).to(dev)].any()
