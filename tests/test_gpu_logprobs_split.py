"""Gradients whose grad_hidden units are split over the vocabulary and claimed
between grad_weight units: a warpgroup then writes its staging buffer for a
split part right after a grad_weight box has left from the same bytes.

The order of the two is fixed by a wait in the kernel, and no test can make the
copy late; these run the sizes where the two follow each other (as slabs, and
as an ordered chain) and compare every element, and every repeat bit for bit.

Tolerances as in test_gpu_logprobs.py: dz is rounded to bf16 once (2^-8) and its
fp32 value is off by less than 2e-4 of its terms' magnitudes on grid inputs
(1002 parts of 128 terms: (128 + 1002) 2^-24 = 6.8e-5 of the sum); a bf16 output
is rounded once more.
"""
import numpy as np
import pytest

from tests.test_gpu_logprobs import env, problem, to_gpu  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu


def reference(torch, h, w, t, g):
    """Gradients of sum(g logp) and the sums of magnitudes, in fp64 on the device."""
    x, u, g = h.double(), w.double(), g.double()
    p = torch.softmax(x @ u.T, 1)
    keep = (t != -100)
    g = torch.where(keep, g, 0.0)
    at = torch.where(keep, t, 0).long()[:, None]
    dz = (-p * g[:, None]).scatter_add_(1, at, g[:, None])
    ref = dz @ u, dz.T @ x
    mag = (p * g.abs()[:, None]).scatter_add_(1, at, g.abs()[:, None])
    return ref, (mag @ u.abs(), mag.T @ x.abs())


@pytest.mark.parametrize("N,H,V", [(256, 1280, 16000), (128, 4096, 128256), (200, 1288, 16001), (120, 2056, 70001)])
@pytest.mark.parametrize("bf16", [True, False])
def test_split_units_between_weight_units(env, N, H, V, bf16):  # noqa: F811
    flce, torch, dev = env
    X, W, t = problem(N, H, V, seed=N, ignored=0.05)
    h, w, tt = to_gpu(torch, dev, X, W, t)
    g = torch.from_numpy(np.random.default_rng(1).standard_normal(N).astype(np.float32)).to(dev)
    o = flce.token_logprobs(h, w, tt)
    dt = torch.bfloat16 if bf16 else torch.float32
    first = None
    for _ in range(4):
        d = flce.token_logprobs_bwd(h, w, tt, o["lse"], None, g, grad_weight_dtype=dt)
        if first is None:
            first = d
        for k in ("grad_hidden", "grad_weight"):
            assert torch.equal(first[k], d[k]), k
    assert flce.query_status(d["workspace"]) == flce.FLCE_OK
    ref, mag = reference(torch, h, w, tt, g)
    for k, r, m, rounds in zip(("grad_hidden", "grad_weight"), ref, mag, (1, int(bf16))):
        tol = m * (2.0 ** -8 + 2e-4) * (1 + 2.0 ** -8) + rounds * 2.0 ** -8 * r.abs()
        err = (d[k].double() - r).abs()
        assert bool((err <= tol + 1e-30).all()), (k, float((err / (tol + 1e-30)).max()))
