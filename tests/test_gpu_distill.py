"""Distillation from a teacher's list, and its gradients, against the fp64 oracle.

Tolerances (derived, not fitted).  On grid inputs every logit is exact in fp32.
The sums of 2^x are off by at most 4e-5 of themselves (rounded arguments, the
approximate 2^x, the merges of the parts: as for the log probabilities), so
every log probability by 4e-5 + 2^-22 of its size.  The masses p come from expf
(2 ulp: 2^-22 of them), their sum and r by as much of theirs.  So
  kl: A (4e-5 + ...) + 2^-21 of the sum of its terms' magnitudes, + the error of r
  times |log r - log s| + 1, below 2^-21 (1 + that) .
On other inputs a logit adds (H / 16 + 4) 2^-23 sum |x w|, twice (in z and lse).
Gradients: dz is rounded to bf16 once (2^-8 of it), its fp32 value is off by less
than 2e-4 of the sum of its terms' magnitudes (the errors above), and a bf16
output is rounded once more.
"""
import gc

import numpy as np
import pytest

from oracle.next_token_fp64 import distill_grad_oracle, distill_oracle

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from linear_cross_entropy_ce_gb300 import flce
    try:
        flce.library()
    except RuntimeError:
        import __graft_entry__
        __graft_entry__.build()
    return flce, torch, torch.device("cuda:0")


def problem(N, H, V, K, seed, grid=True, T=1.0, ignored=0.2):
    import torch
    r = np.random.default_rng(seed)
    std = 1.28 / np.sqrt(H)
    X, W = r.standard_normal((N, H)), std * r.standard_normal((V, H))
    X += W[r.integers(0, V, N)] * (10 * r.random((N, 1)) / (H * std * std))
    if grid:
        step = 2.0 ** np.round(np.log2(std / 10))
        X, W = np.clip(np.round(X * 16), -64, 64) / 16, np.clip(np.round(W / step), -63, 63) * step
    else:
        X, W = (torch.from_numpy(a).to(torch.bfloat16).double().numpy() for a in (X, W))
    z = (X + r.standard_normal((N, H))) @ W.T / T
    ids = np.argsort(-z, 1)[:, :K].astype(np.int32)
    top = z.max(1, keepdims=True)
    lp = z - top - np.log(np.exp(z - top).sum(1, keepdims=True))
    t = np.take_along_axis(lp, ids, 1).astype(np.float32)
    # in any order, some entries absent, some tokens named twice, some without mass, rows without a teacher
    order = r.permutation(K)
    ids, t = ids[:, order].copy(), t[:, order].copy()
    ids[r.random((N, K)) < 0.05] = -1
    if K > 1:
        twice = r.random(N) < 0.2
        ids[twice, 0] = ids[twice, K - 1]
        t[twice, 0] -= 3
    t[r.random((N, K)) < 0.03] = -np.inf
    ids[r.random(N) < ignored] = -1
    return X, W, ids, t


def to_gpu(torch, dev, X, W, ids, t):
    f = lambda a: torch.from_numpy(a).to(torch.bfloat16).to(dev)  # noqa: E731
    return f(X), f(W), torch.from_numpy(ids).to(dev), torch.from_numpy(t).to(dev)


def np64(a):
    return a.detach().double().cpu().numpy()


def check(o, ref, zerr=0.0):
    got = {k: np64(o[k]) for k in ("kl", "lse", "rest_logp", "student_logp")}
    for k in ("lse", "rest_logp", "student_logp"):
        inf = np.isneginf(ref[k])
        np.testing.assert_array_equal(np.isneginf(got[k]), inf)
        want = np.where(inf, 0, ref[k])
        ze = (zerr if np.ndim(zerr) == 0 or k != "student_logp" else zerr[:, None])
        err = np.abs(np.where(inf, 0, got[k]) - want)
        assert np.all(err <= 4e-5 + 2 * ze + 2.0 ** -22 * np.abs(want)), (k, err.max())
    gap = np.abs(np.log(np.maximum(ref["r"], 1e-38)) - np.where(np.isfinite(ref["rest_logp"]), ref["rest_logp"], 0)) + 1
    tol = ref["mass"] * (4e-5 + 2 * zerr) + 2.0 ** -21 * (ref["size"] + 1 + np.where(ref["r"] > 0, gap, 0))
    err = np.abs(got["kl"] - ref["kl"])
    assert np.all(err <= tol), (err / tol).max()


SHAPES = [  # N, H, V, K, T, tail
    (1, 64, 1, 1, 1.0, True), (1, 8, 2, 1, 1.0, True), (1, 8, 2, 2, 1.0, False), (1, 4096, 5003, 20, 1.0, True),
    (2, 72, 129, 32, 0.7, True), (5, 2048, 257, 1, 1.3, False), (16, 512, 16000, 64, 1.0, True),
    (17, 520, 1000, 100, 2.0, False), (33, 64, 31, 31, 1.0, True), (61, 136, 16007, 7, 0.5, True),
    (64, 1024, 4096, 256, 1.0, True), (100, 264, 3001, 3, 2.0, True), (128, 128, 300, 255, 1.0, True),
    (129, 64, 512, 9, 1.0, True), (257, 192, 1030, 40, 1.0, False), (300, 64, 512, 8, 0.9, True),
    (700, 520, 4099, 129, 1.0, True), (200, 8, 1, 1, 1.0, True), (200, 8, 300, 256, 1.0, True),
    (300, 1024, 9001, 33, 1.0, True), (140, 64, 64, 64, 1.0, True), (16500, 8, 300, 5, 1.0, True),
    (150, 512, 2000, 20, 1.0, True), (40, 384, 2000, 20, 1.0, False), (129, 704, 999, 70, 1.0, True)]


@pytest.mark.parametrize("N,H,V,K,T,tail", SHAPES)
def test_forward_grid(env, N, H, V, K, T, tail):
    flce, torch, dev = env
    X, W, ids, t = problem(N, H, V, K, N + V, T=T)
    o = flce.topk_distill(*to_gpu(torch, dev, X, W, ids, t), temperature=T, tail=tail)
    assert flce.query_status(o["workspace"]) == flce.FLCE_OK
    check(o, distill_oracle(X, W, ids, t, T, tail))


@pytest.mark.parametrize("N,H,V", [(1, 4096, 3000), (40, 1024, 5000), (300, 2048, 1111), (130, 8192, 300)])
def test_forward_continuous(env, N, H, V):
    flce, torch, dev = env
    X, W, ids, t = problem(N, H, V, 17, 5, grid=False)
    o = flce.topk_distill(*to_gpu(torch, dev, X, W, ids, t))
    zerr = (H / 16 + 4) * 2.0 ** -23 * (np.abs(X) @ np.abs(W).T).max(1)
    check(o, distill_oracle(X, W, ids, t), zerr)


GRADS = [  # N, H, V, K, T, tail, bf16
    (1, 64, 512, 8, 1.0, True, False), (3, 72, 130, 30, 0.7, False, True), (128, 64, 512, 64, 1.0, True, False),
    (300, 64, 512, 8, 2.0, False, True), (513, 136, 1000, 100, 1.3, True, False), (640, 520, 2049, 20, 1.0, True, True),
    (200, 8, 1, 1, 1.0, True, True), (140, 8, 77, 77, 1.0, True, False), (300, 256, 9000, 256, 1.0, True, True)]


@pytest.mark.parametrize("N,H,V,K,T,tail,bf16", GRADS)
@pytest.mark.parametrize("grid", [True, False])
def test_gradients(env, N, H, V, K, T, tail, bf16, grid):
    flce, torch, dev = env
    X, W, ids, t = problem(N, H, V, K, N, grid=grid, T=T)
    g = np.random.default_rng(1).standard_normal(N).astype(np.float32)
    a = to_gpu(torch, dev, X, W, ids, t)
    o = flce.topk_distill(*a, temperature=T, tail=tail)
    args = (*a, o["lse"], o["rest_logp"], o["student_logp"], torch.from_numpy(g).to(dev))
    kw = dict(temperature=T, tail=tail, grad_weight_dtype=torch.bfloat16 if bf16 else torch.float32)
    d = flce.topk_distill_bwd(*args, **kw)
    assert flce.query_status(d["workspace"]) == flce.FLCE_OK
    check_gradients(d, distill_grad_oracle(X, W, ids, t, g, T, tail), bf16)
    assert not d["grad_hidden"][torch.from_numpy((ids < 0).all(1)).to(dev)].any()
    one = flce.topk_distill_bwd(*args, need_weight=False, **kw)
    two = flce.topk_distill_bwd(*args, need_hidden=False, **kw)
    assert one["grad_weight"] is None and two["grad_hidden"] is None
    assert torch.equal(one["grad_hidden"], d["grad_hidden"]) and torch.equal(two["grad_weight"], d["grad_weight"])


def check_gradients(d, ref, bf16):
    for k, rounds in (("hidden", 1), ("weight", int(bf16))):
        tol = ref["mag_" + k] * (2.0 ** -8 + 2e-4) * (1 + 2.0 ** -8) + rounds * 2.0 ** -8 * np.abs(ref["grad_" + k])
        err = np.abs(np64(d["grad_" + k]) - ref["grad_" + k])
        assert np.all(err <= tol + 1e-30), (k, (err / (tol + 1e-30)).max())


@pytest.mark.parametrize("N", [30, 200])
def test_nearly_all_of_the_mass_is_listed(env, N):
    """Student masses behind the list from 1e-3 down to far below what fp32 can tell from 0, and teachers of no tail."""
    flce, torch, dev = env
    V, H, K = 400, 64, 3
    X, W = np.zeros((N, H)), np.zeros((V, H))
    X[:, 0] = 2.0 ** (np.arange(N) % 9)            # logits of the listed tokens: 1 to 256
    X[:, 1] = 1
    r = np.random.default_rng(0)
    W[:K, 0] = 1
    W[:, 1] = np.round(r.standard_normal(V) * 16) / 16
    ids = np.tile(np.arange(K, dtype=np.int32), (N, 1))
    t = np.log(np.tile(np.array([0.5, 0.25, 0.25 - 1e-4]), (N, 1))).astype(np.float32)
    t[::2, 2] = np.float32(np.log(0.25))           # sums to 1 but for rounding
    a = to_gpu(torch, dev, X, W, ids, t)
    o = flce.topk_distill(*a)
    ref = distill_oracle(X, W, ids, t)
    assert ref["rest_logp"].min() < -240
    check(o, ref)
    g = np.ones(N, np.float32)
    d = flce.topk_distill_bwd(*a, o["lse"], o["rest_logp"], o["student_logp"], torch.from_numpy(g).to(dev))
    back = distill_grad_oracle(X, W, ids, t, g)
    # r is the difference of 1 and a sum of about 1: off by 2^-22, which stands against the gradient's terms as a whole
    q = np.abs(back["mag_hidden"]).max() * 2.0 ** -20
    for k in ("hidden", "weight"):
        tol = back["mag_" + k] * (2.0 ** -8 + 2e-4) * 1.01 + (2.0 ** -8) * np.abs(back["grad_" + k]) + q
        assert np.all(np.abs(np64(d["grad_" + k]) - back["grad_" + k]) <= tol), k


@pytest.mark.parametrize("N", [6, 200])
def test_rows_of_their_own(env, N):
    """No entry, a token outside, no mass, NaN, infinite logits: each row by itself."""
    flce, torch, dev = env
    X, W, ids, t = problem(N, 64, 300, 5, 3, ignored=0.0)
    good = flce.topk_distill(*to_gpu(torch, dev, X, W, ids, t))
    ids, t = ids.copy(), t.copy()
    ids[0] = -1
    ids[1, 2] = 300
    t[2] = -np.inf
    t[3, 1] = np.nan
    ids[3, 1] = 7
    h, w, i, tt = to_gpu(torch, dev, X, W, ids, t)
    h[4, 2] = float("inf")
    for tail in (True, False):
        o = flce.topk_distill(h, w, i, tt, tail=tail)
        assert flce.query_status(o["workspace"]) == flce.FLCE_EBADTARGET
        for k in ("kl", "lse", "rest_logp", "student_logp"):
            assert not o[k][0].any() and torch.isnan(o[k][1]).all(), k
        assert torch.isnan(o["kl"][3]) and not torch.isnan(o["lse"][3]) and torch.isnan(o["kl"][4])
        ref = distill_oracle(X[2:3], W, ids[2:3], t[2:3], tail=tail)
        assert abs(o["kl"][2].item() - ref["kl"][0]) <= 1e-4 * (1 + ref["kl"][0])
        if tail:
            assert torch.equal(o["kl"][5:], good["kl"][5:]) and torch.equal(o["lse"][5:], good["lse"][5:])
    ids[1], ids[3] = -1, -1
    h, w, i, tt = to_gpu(torch, dev, X, W, ids, t)
    one = torch.ones(N, device=dev)
    for tail in (True, False):
        o = flce.topk_distill(h, w, i, tt, tail=tail)
        d = flce.topk_distill_bwd(h, w, i, tt, o["lse"], o["rest_logp"], o["student_logp"], one, tail=tail)
        check_gradients(d, distill_grad_oracle(X, W, ids, np.nan_to_num(t, nan=0.0, neginf=-np.inf), np.ones(N), tail=tail), False)
    none = torch.full_like(i, -3)
    o = flce.topk_distill(h, w, none, tt)
    d = flce.topk_distill_bwd(h, w, none, tt, o["lse"], o["rest_logp"], o["student_logp"], one)
    assert flce.query_status(o["workspace"]) == flce.FLCE_OK
    assert not o["kl"].any() and not d["grad_hidden"].any() and not d["grad_weight"].any()


@pytest.mark.parametrize("bf16", [False, True])
def test_in_chunks(env, bf16):
    """Workspaces for 128 rows at a time, and nothing behind the outputs written."""
    flce, torch, dev = env
    N, H, V, K = 700, 136, 1000, 12
    X, W, ids, t = problem(N, H, V, K, 3)
    a = to_gpu(torch, dev, X, W, ids, t)
    whole = flce.topk_distill(*a)
    lo, hi = 0, flce.library().flce_topk_distill_workspace_bytes(N, H, V, K)
    top = hi
    while hi - lo > 256:
        mid = (lo + hi) // 2
        try:
            flce.topk_distill(*a, workspace=flce.new_workspace(mid, dev))
            hi = mid
        except flce.FlceError as e:
            assert e.status == flce.FLCE_EWORKSPACE
            lo = mid
    assert hi < top
    ws = torch.full((hi + 512,), 171, dtype=torch.uint8, device=dev)
    big = torch.full((N * K + 8,), 7.0, device=dev)
    o = flce.topk_distill(*a, workspace=ws[:hi], out={"student_logp": big[:N * K].view(N, K)})
    assert (big[N * K:] == 7).all() and (ws[hi:] == 171).all()
    for k in ("kl", "lse", "rest_logp", "student_logp"):
        assert torch.equal(o[k], whole[k]), k
    g = np.random.default_rng(1).standard_normal(N).astype(np.float32)
    dt = torch.bfloat16 if bf16 else torch.float32
    need = flce.workspace_bytes(N, H, V, chunk_rows=128, grad_weight_dtype=dt) + 4096 + 3 * 3072 + N * K * 2 + 1024
    d = flce.topk_distill_bwd(*a, o["lse"], o["rest_logp"], o["student_logp"], torch.from_numpy(g).to(dev),
                              grad_weight_dtype=dt, workspace=flce.new_workspace(need, dev))
    check_gradients(d, distill_grad_oracle(X, W, ids, t, g), bf16)


@pytest.mark.parametrize("N", [20, 300])
def test_the_same_token_named_in_every_entry(env, N):
    flce, torch, dev = env
    X, W, ids, t = problem(N, 64, 500, 6, 3, ignored=0.0)
    ids[:] = ids[:, :1].clip(min=0)
    t[:] = np.log(np.float32(0.1))
    a = to_gpu(torch, dev, X, W, ids, t)
    for tail in (True, False):
        o = flce.topk_distill(*a, tail=tail)
        check(o, distill_oracle(X, W, ids, t, tail=tail))
        d = flce.topk_distill_bwd(*a, o["lse"], o["rest_logp"], o["student_logp"], torch.ones(N, device=dev), tail=tail)
        check_gradients(d, distill_grad_oracle(X, W, ids, t, np.ones(N), tail=tail), False)


def test_gradient_against_differences(env):
    """Steps of one weight and one hidden value, on logits that are exact."""
    flce, torch, dev = env
    N, H, V, K = 8, 64, 200, 10
    X, W, ids, t = problem(N, H, V, K, 11, ignored=0.0)
    a = to_gpu(torch, dev, X, W, ids, t)
    o = flce.topk_distill(*a)
    d = flce.topk_distill_bwd(*a, o["lse"], o["rest_logp"], o["student_logp"], torch.ones(N, device=dev))
    ref = distill_grad_oracle(X, W, ids, t, np.ones(N))
    e = 2.0 ** -4
    for which, at in [(0, (1, 3)), (1, (int(ids[2].max()), 7)), (1, (int((set(range(V)) - set(ids.ravel())).pop()), 2))]:
        sums = []
        for s in (e, -e):
            b = [x.clone() for x in a]
            old = b[which][at].item()
            b[which][at] = old + s
            assert b[which][at].item() == old + s   # exact in bf16
            sums.append(np64(flce.topk_distill(*b)["kl"]).sum())
        slope = (sums[0] - sums[1]) / (2 * e)
        got = d["grad_hidden" if which == 0 else "grad_weight"][at].item()
        # the central difference's own error is of the third derivative: at most (e max|x or w|)^2 of the magnitudes
        size = (W if which == 0 else X)
        mag = (ref["mag_hidden"] if which == 0 else ref["mag_weight"])[at]
        far = mag * ((e * np.abs(size).max()) ** 2 + 2.0 ** -7) + 2 * N * 1e-4 / (2 * e)
        assert abs(slope - got) <= far, (slope, got, far)


def test_module_step_and_capture(env):
    """Autograd through the module, eagerly and in a captured training step."""
    flce, torch, dev = env
    N, H, V, K = 200, 64, 900, 16
    X, W, ids, t = problem(N, H, V, K, 4)
    h, w, i, tt = to_gpu(torch, dev, X, W, ids, t)
    m = flce.LinearTopKDistill(w.clone(), temperature=1.5, tail=True)
    x = h.clone().requires_grad_(True)
    wt = torch.rand(N, device=dev, generator=torch.Generator(device=dev).manual_seed(0))
    (m(x, i, tt) * wt).sum().backward()
    ref = distill_grad_oracle(X, W, ids, t, np64(wt), 1.5, True)
    check_gradients({"grad_hidden": x.grad, "grad_weight": m.weight.grad}, ref, True)
    eager = x.grad.clone(), m.weight.grad.clone()
    # a frozen head, a frozen trunk
    y = h.clone().requires_grad_(True)
    flce.linear_topk_distill(y, w, i, tt, 1.5).backward(wt)
    assert torch.equal(y.grad, eager[0])
    # captured: warm up on a side stream, then replay on other weights of the tokens
    x.grad = m.weight.grad = None
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        (m(x, i, tt) * wt).sum().backward()
        x.grad = m.weight.grad = None
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            loss = (m(x, i, tt) * wt).sum()
            loss.backward()
    keep = wt.clone()
    wt.zero_()
    graph.replay()
    assert not x.grad.any()
    wt.copy_(keep)
    x.grad.zero_()
    m.weight.grad.zero_()
    graph.replay()
    torch.cuda.synchronize()
    got = x.grad.clone()
    assert torch.equal(got, eager[0]) or torch.allclose(got.float(), eager[0].float(), rtol=2 ** -7, atol=1e-6)


@pytest.mark.parametrize("N", [8, 300])
def test_time_out(env, N):
    flce, torch, dev = env
    X, W, ids, t = problem(N, 64, 900, 6, 7)
    a = to_gpu(torch, dev, X, W, ids, t)
    good = flce.topk_distill(*a)
    rows = torch.from_numpy((ids >= 0).any(1)).to(dev)
    flce.debug_arm_stall(20_000_000)
    o = flce.topk_distill(*a)
    assert flce.query_status(o["workspace"]) == flce.FLCE_ETIMEOUT
    assert torch.isnan(o["kl"][rows]).all() and not o["kl"][~rows].any()
    one = torch.ones(N, device=dev)
    args = (*a, good["lse"], good["rest_logp"], good["student_logp"], one)
    flce.debug_arm_stall(20_000_000)
    d = flce.topk_distill_bwd(*args)
    assert flce.query_status(d["workspace"]) == flce.FLCE_ETIMEOUT
    assert torch.isnan(d["grad_hidden"].view(-1)[0]) and torch.isnan(d["grad_weight"].view(-1)[0])
    again = flce.topk_distill(*a)
    assert flce.query_status(again["workspace"]) == flce.FLCE_OK and torch.equal(again["kl"], good["kl"])


def test_generate_under_rules_then_distill(env):
    """As they are used together: a teacher generates under penalties and a mask, its alternatives of those tokens
    teach a student whose embedding and head are tied."""
    flce, torch, dev = env
    V, H, steps, B = 500, 64, 12, 6
    gen = torch.Generator(device=dev).manual_seed(3)
    teacher = (torch.randn((V, H), generator=gen, device=dev) * 0.3).to(torch.bfloat16)
    trunk = torch.randn((H, H), generator=gen, device=dev) / 8
    state = lambda w, ids: torch.tanh(flce.embedding(ids, w).float() @ trunk).to(torch.bfloat16)  # noqa: E731
    history = torch.full((B, steps + 1), -1, dtype=torch.int32, device=dev)
    history[:, 0] = torch.arange(B, device=dev)
    allowed = np.ones((B, V), bool)
    allowed[:, 250:] = False
    words = np.zeros((B, 512), bool)
    words[:, :V] = allowed
    mask = torch.from_numpy(np.packbits(words, 1, bitorder="little").view(np.int32)).to(dev)
    ones = torch.ones(B, dtype=torch.int32, device=dev)
    for i in range(steps):
        o = flce.constrained_logprobs(state(teacher, history[:, i].contiguous()), teacher, history=history,
                                      history_lens=ones * (i + 1), prompt_lens=ones,
                                      presence_penalty=100.0 * ones.float(), mask=mask, top_k=1)
        history[:, i + 1] = o["top_ids"][:, 0]
    out = history[:, 1:].cpu().numpy()
    assert (out >= 0).all() and (out < 250).all()
    assert all(len(set(row)) == steps for row in out.tolist())   # no token of the output comes again
    ids = history[:, :-1].reshape(-1).contiguous()
    tops = flce.token_logprobs(state(teacher, ids), teacher, history[:, 1:].reshape(-1).contiguous(), top_k=10)
    student = torch.nn.Parameter((torch.randn((V, H), generator=gen, device=dev) * 0.3).to(torch.bfloat16))
    x = torch.tanh(flce.embedding(ids, student).float() @ trunk).to(torch.bfloat16)
    x.retain_grad()
    kl = flce.linear_topk_distill(x, student, tops["top_ids"], tops["top_logp"])
    kl.mean().backward()
    N = ids.numel()
    args = (np64(x), np64(student), tops["top_ids"].cpu().numpy(), tops["top_logp"].cpu().numpy())
    ref = distill_oracle(*args)
    zerr = (H / 16 + 4) * 2.0 ** -23 * (np.abs(args[0]) @ np.abs(args[1]).T).max(1)
    check({"kl": kl, **{k: torch.from_numpy(ref[k]) for k in ("lse", "rest_logp", "student_logp")}}, ref, zerr)
    g = distill_grad_oracle(*args, np.full(N, 1.0 / N))
    err = np.abs(np64(x.grad) - g["grad_hidden"])
    assert np.all(err <= g["mag_hidden"] * (2.0 ** -8 + 2e-4) * 1.01 + 2.0 ** -8 * np.abs(g["grad_hidden"]) + 1e-30)
    assert student.grad is not None and torch.isfinite(student.grad).all()


def test_repeated_calls_agree_bit_for_bit(env):
    flce, torch, dev = env
    for N in (20, 300):
        X, W, ids, t = problem(N, 128, 3000, 40, 6)
        a = to_gpu(torch, dev, X, W, ids, t)
        one = torch.ones(N, device=dev)
        first = None
        for _ in range(4):
            o = flce.topk_distill(*a)
            d = flce.topk_distill_bwd(*a, o["lse"], o["rest_logp"], o["student_logp"], one)
            got = [o["kl"], o["lse"], o["rest_logp"], o["student_logp"], d["grad_hidden"], d["grad_weight"]]
            first = first or got
            assert all(torch.equal(x, y) for x, y in zip(first, got))


def test_two_streams_at_once(env):
    flce, torch, dev = env
    sets = []
    for seed, N in ((1, 90), (2, 260)):
        a = to_gpu(torch, dev, *problem(N, 64, 2000, 30, seed))
        sets.append((a, flce.topk_distill(*a)))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [flce.topk_distill(*a, stream=st) for st, (a, _) in zip(streams, sets) for _ in range(3)]
    torch.cuda.synchronize()
    for i, o in enumerate(got):
        for k in ("kl", "rest_logp", "student_logp"):
            assert torch.equal(o[k], sets[i // 3][1][k]), k


def test_capture_beside_a_living_graph_is_refused(env):
    """Autograd would order the default stream behind the capture, which ends the process: refused before that."""
    flce, torch, dev = env
    h, w, i, tt = to_gpu(torch, dev, *problem(150, 64, 500, 6, 4))
    w.requires_grad_(True)
    step = lambda: flce.linear_topk_distill(h, w, i, tt).sum()  # noqa: E731
    want = torch.autograd.grad(step(), w)[0]
    alive = step()
    torch.cuda.synchronize()
    with pytest.raises(RuntimeError, match="alive"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            torch.autograd.grad(step(), w)
    del alive
    gc.collect()   # the refused step's graph hangs on its exception's traceback, a cycle, and keeps the leaf's accumulator
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = torch.autograd.grad(step(), w)[0]
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("N", [60, 300])
def test_two_captures_replayed_in_turn(env, N):
    """Two captured calls from one pool of memory, replayed one after the other on new lists."""
    flce, torch, dev = env
    sets = [to_gpu(torch, dev, *problem(N, 64, 2000, 30, seed)) for seed in (1, 2, 3)]
    want = [flce.topk_distill(*a) for a in sets]
    live = [[x.clone() for x in sets[0]], [x.clone() for x in sets[1]]]
    torch.cuda.synchronize()
    graphs, outs, pool = [], [], None
    for a in live:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=pool):
            outs.append({k: v for k, v in flce.topk_distill(*a).items() if k != "workspace"})
        pool = g.pool()
        graphs.append(g)
    for which in ((0, 1), (2, 0), (1, 2)):
        for a, s in zip(live, which):
            for x, y in zip(a, sets[s]):
                x.copy_(y)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for o, s in zip(outs, which):
            for k in ("kl", "lse", "rest_logp", "student_logp"):
                assert torch.equal(o[k], want[s][k]), (k, which)
