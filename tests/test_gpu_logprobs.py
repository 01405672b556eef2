"""Token log probabilities, entropies, top alternatives and their gradients
against the fp64 oracle.

Tolerances (derived, not fitted).  On grid inputs every sum of products is
exact in fp32, so only the softmax rounds: the argument of each 2^x is off by at
most |x| 2^-23 (x up to ~60: 5e-6 of the term), the approximate 2^x by 2^-22,
and the sums of P parts of 128 terms by (128 + P) 2^-24.  With P <= 200 that
is under 3e-5 of each sum, so logp and lse are off by at most 3e-5 plus
2^-22 of their size, the entropy by 3e-5 (1 + its size + the mean of |log p|).
On other inputs a logit adds (H / 16 + 4) 2^-23 sum |x w|: one rounding per
16-wide matrix instruction.
Gradients: dz is rounded to bf16 once (2^-8 of it), its fp32 value is off by
less than 2e-4 of the sum of its terms' magnitudes (the errors above), and a
bf16 output is rounded once more.
"""
import numpy as np
import pytest

from oracle.logprobs_fp64 import logprobs_grad_oracle, logprobs_oracle

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


def problem(N, H, V, seed, ignored=0.0, grid=True, std=None):
    """Inputs exactly representable in bf16; on a grid, sums of products are exact in fp32."""
    r = np.random.default_rng(seed)
    std = 1.28 / np.sqrt(H) if std is None else std
    X, W = r.standard_normal((N, H)), std * r.standard_normal((V, H))
    t = r.integers(0, V, N).astype(np.int32)
    X += W[t] * (10 * r.random((N, 1)) / (H * std * std))
    if grid:
        step = 2.0 ** np.round(np.log2(std / 10))
        X, W = np.clip(np.round(X * 16), -64, 64) / 16, np.clip(np.round(W / step), -63, 63) * step
    else:
        import torch
        X, W = (torch.from_numpy(a).to(torch.bfloat16).double().numpy() for a in (X, W))
    t[r.random(N) < ignored] = -100
    return X, W, t


def to_gpu(torch, dev, X, W, t):
    f = lambda a: torch.from_numpy(a).to(torch.bfloat16).to(dev)  # noqa: E731
    return f(X), f(W), torch.from_numpy(t).to(dev)


def np64(a):
    return a.detach().double().cpu().numpy()


def check_forward(o, ref, T, K, zerr=0.0):
    zerr = zerr / T
    for k in ("logp", "lse"):
        err = np.abs(np64(o[k]) - ref[k])
        assert np.all(err <= 3e-5 + 2 * zerr + 2.0 ** -22 * np.abs(ref[k])), (k, err.max())
    p = np.exp(ref["all_logp"])
    mean = -(p * ref["all_logp"]).sum(1)
    err = np.abs(np64(o["entropy"]) - ref["entropy"])
    assert np.all(err <= (3e-5 + 2 * zerr) * (1 + 2 * mean)), err.max()
    if K:
        if not np.any(zerr):
            np.testing.assert_array_equal(o["top_ids"].cpu().numpy(), ref["top_ids"])
        err = np.abs(np64(o["top_logp"]) - ref["top_logp"])
        assert np.all(err <= (3e-5 + 2 * zerr + 0 * ref["logp"])[:, None] + 2.0 ** -22 * np.abs(ref["top_logp"]))


SHAPES = [  # N, H, V, K, ignored, T
    (1, 64, 1, 1, 0.0, 1.0), (1, 8, 2, 2, 0.0, 1.0), (1, 4096, 5003, 8, 0.0, 1.0), (2, 72, 129, 32, 0.0, 0.7),
    (5, 2048, 257, 1, 0.3, 1.3), (16, 512, 16000, 5, 0.0, 1.0), (17, 520, 1000, 20, 0.2, 1.0),
    (33, 64, 31, 31, 0.0, 1.0), (61, 136, 16007, 7, 0.1, 0.5), (64, 1024, 4096, 0, 0.5, 1.0),
    (100, 264, 3001, 3, 0.05, 2.0), (127, 128, 2000, 16, 0.3, 1.0), (128, 128, 128, 32, 0.0, 1.0),
    (129, 64, 512, 9, 0.9, 1.0), (257, 192, 1030, 4, 0.1, 1.0), (300, 64, 512, 0, 0.1, 0.9),
    (700, 520, 4099, 12, 0.3, 1.0), (1000, 256, 16000, 0, 0.05, 1.0), (200, 8, 1, 1, 0.0, 1.0),
    (200, 8, 300, 32, 0.2, 1.0), (1, 8, 100003, 32, 0.0, 1.0)]


@pytest.mark.parametrize("N,H,V,K,ignored,T", SHAPES)
def test_forward_grid(env, N, H, V, K, ignored, T):
    flce, torch, dev = env
    X, W, t = problem(N, H, V, seed=N + V, ignored=ignored)
    o = flce.token_logprobs(*to_gpu(torch, dev, X, W, t), temperature=T, top_k=K)
    assert flce.query_status(o["workspace"]) == flce.FLCE_OK
    check_forward(o, logprobs_oracle(X, W, t, temperature=T, top_k=K), T, K)


@pytest.mark.parametrize("N,H,V", [(1, 4096, 3000), (40, 1024, 5000), (300, 2048, 1111), (3, 16384, 100),
                                   (130, 16384, 300)])
def test_forward_continuous(env, N, H, V):
    flce, torch, dev = env
    X, W, t = problem(N, H, V, seed=5, grid=False)
    o = flce.token_logprobs(*to_gpu(torch, dev, X, W, t), top_k=4)
    zerr = (H / 16 + 4) * 2.0 ** -23 * (np.abs(X) @ np.abs(W).T).max(1)
    check_forward(o, logprobs_oracle(X, W, t, top_k=4), 1.0, 4, zerr)


@pytest.mark.parametrize("N", [1, 30, 200])
def test_ties_go_to_the_lowest_id(env, N):
    """Every row of the weight occurs many times: whole blocks of logits are equal."""
    flce, torch, dev = env
    X, W, t = problem(N, 64, 7, seed=2)
    W = np.tile(W, (430, 1))[:3000]
    o = flce.token_logprobs(*to_gpu(torch, dev, X, W, t), top_k=32)
    ref = logprobs_oracle(X, W, t, top_k=32)
    np.testing.assert_array_equal(o["top_ids"].cpu().numpy(), ref["top_ids"])
    zero = flce.token_logprobs(*to_gpu(torch, dev, 0 * X, W, t), top_k=32)
    assert zero["top_ids"].tolist() == [list(range(32))] * N
    np.testing.assert_allclose(np64(zero["entropy"]), np.log(3000), rtol=2e-6)


@pytest.mark.parametrize("N,sign", [(3, 1), (3, -1), (200, 1), (200, -1)])
def test_sorted_logits(env, N, sign):
    """Logits that rise or fall along the vocabulary: every or no candidate replaces the list."""
    flce, torch, dev = env
    V = 4000
    X = np.zeros((N, 64))
    X[:, 0], X[:, 1] = 1, 1
    W = np.zeros((V, 64))
    v = np.arange(V) if sign > 0 else np.arange(V)[::-1]
    W[:, 0], W[:, 1] = v // 64, (v % 64) / 64   # both exact in bf16
    t = np.zeros(N, np.int32)
    o = flce.token_logprobs(*to_gpu(torch, dev, X, W, t), top_k=32)
    check_forward(o, logprobs_oracle(X, W, t, top_k=32), 1.0, 32)


@pytest.mark.parametrize("N,chunk", [(1, 0), (20, 0), (120, 0), (300, 0), (300, 128)])
@pytest.mark.parametrize("kind", ["random", "rising", "falling", "equal", "peaks"])
def test_alternatives_over_many_parts(env, N, chunk, kind):
    """Vocabularies of many more parts than alternatives, where only parts above a running bound are kept."""
    flce, torch, dev = env
    V, K = 20003, 8
    X, W, t = problem(N, 64, V, seed=7, ignored=0.1)
    if kind != "random":
        X = np.zeros((N, 64))
        X[:, 0], X[:, 1] = 1, 1
        v = np.arange(V)[::-1] if kind == "falling" else np.arange(V)
        W = np.zeros((V, 64))
        if kind in ("rising", "falling"):
            W[:, 0], W[:, 1] = v // 128, (v % 128) / 128   # both exact in bf16
        elif kind == "peaks":
            W[(v * 7919) % V < 12, 0] = 3   # a dozen equal peaks far apart
    T = 1.0 if kind in ("random", "peaks", "equal") else 16.0
    h, w, tt = to_gpu(torch, dev, X, W, t)
    kw = {}
    if chunk:   # the fp32 logits of `chunk` rows and the rest
        kw["workspace"] = flce.new_workspace((V + 64) * 4 * chunk + (1 << 20), dev)
    o = flce.token_logprobs(h, w, tt, temperature=T, top_k=K, **kw)
    check_forward(o, logprobs_oracle(X, W, t, temperature=T, top_k=K), T, K)


@pytest.mark.parametrize("N", [4, 150])
def test_extreme_rows(env, N):
    """A dominant logit, a row of large logits, rows with NaN and inf: only those rows are NaN."""
    flce, torch, dev = env
    X, W, t = problem(N, 64, 600, seed=9)
    X[0] *= 64
    ref = logprobs_oracle(X, W, t, top_k=5)
    h, w, tt = to_gpu(torch, dev, X, W, t)
    h[2, 3] = float("nan")
    h[3, 5] = float("inf")
    o = flce.token_logprobs(h, w, tt, top_k=5)
    keep = np.array([i for i in range(N) if i not in (2, 3)])
    assert torch.isnan(o["logp"][2:4]).all() and torch.isnan(o["lse"][2:4]).all() and torch.isnan(o["entropy"][2:4]).all()
    cut = {k: (v[keep] if isinstance(v, np.ndarray) else v) for k, v in ref.items()}
    got = {k: o[k][torch.from_numpy(keep).to(dev)] for k in ("logp", "lse", "entropy", "top_ids", "top_logp")}
    check_forward(got, cut, 1.0, 5, zerr=np.zeros(len(keep)))
    assert np64(o["logp"])[0] <= 0 and np64(o["entropy"])[0] >= -1e-6


@pytest.mark.parametrize("N", [6, 200])
def test_all_ignored_and_bad_targets(env, N):
    flce, torch, dev = env
    X, W, t = problem(N, 64, 300, seed=1)
    h, w, tt = to_gpu(torch, dev, X, W, t)
    o = flce.token_logprobs(h, w, torch.full_like(tt, -100), top_k=3)
    assert flce.query_status(o["workspace"]) == flce.FLCE_OK
    assert not o["logp"].any() and not o["entropy"].any() and (o["top_ids"] == -1).all() and not o["top_logp"].any()
    bad = tt.clone()
    bad[1], bad[4] = 300, -7
    b = flce.token_logprobs(h, w, bad, top_k=3)
    assert flce.query_status(b["workspace"]) == flce.FLCE_EBADTARGET
    assert torch.isnan(b["logp"][[1, 4]]).all() and (b["top_ids"][[1, 4]] == -1).all()
    good = flce.token_logprobs(h, w, tt, top_k=3)
    rest = [i for i in range(N) if i not in (1, 4)]
    for k in ("logp", "entropy", "lse", "top_ids", "top_logp"):
        assert torch.equal(b[k][rest], good[k][rest]), k
    g = flce.token_logprobs_bwd(h, w, torch.full_like(tt, -100), o["lse"], o["entropy"], torch.ones_like(o["lse"]))
    assert not g["grad_hidden"].any() and not g["grad_weight"].any()


@pytest.mark.parametrize("N", [3, 700])
def test_small_workspace_and_outputs_left_alone(env, N):
    """Smaller chunks give the same values; nothing behind the outputs is written."""
    flce, torch, dev = env
    X, W, t = problem(N, 128, 2000, seed=4, ignored=0.2)
    h, w, tt = to_gpu(torch, dev, X, W, t)
    a = flce.token_logprobs(h, w, tt, top_k=6)
    lo, hi = 0, flce.library().flce_logprobs_workspace_bytes(N, 128, 2000, 6)
    while hi - lo > 256:   # the smallest workspace that is accepted
        mid = (lo + hi) // 2
        try:
            flce.token_logprobs(h, w, tt, top_k=6, workspace=flce.new_workspace(mid, dev))
            hi = mid
        except flce.FlceError as e:
            assert e.status == flce.FLCE_EWORKSPACE
            lo = mid
    ws = torch.full((hi + 4096,), 171, dtype=torch.uint8, device=dev)
    big = torch.full((N + 8,), 7.0, device=dev)
    bid = torch.full((N * 6 + 8,), 7, dtype=torch.int32, device=dev)
    out = {"logp": big[:N], "top_ids": bid[:N * 6].view(N, 6)}
    b = flce.token_logprobs(h, w, tt, top_k=6, workspace=ws[:hi], out=out)
    assert (big[N:] == 7).all() and (bid[N * 6:] == 7).all() and (ws[hi:] == 171).all()
    for k in ("logp", "entropy", "lse", "top_ids", "top_logp"):
        assert torch.equal(a[k], b[k]), k


GRADS = [  # N, H, V, ignored, T, logp, entropy, bf16
    (1, 64, 512, 0.0, 1.0, True, True, False), (3, 72, 130, 0.3, 0.7, True, False, True),
    (128, 64, 512, 0.0, 1.0, False, True, False), (300, 64, 512, 0.1, 1.0, True, True, True),
    (513, 136, 1000, 0.5, 1.3, True, True, False), (640, 520, 2049, 0.05, 1.0, True, True, True),
    (200, 8, 1, 0.0, 1.0, True, True, True), (140, 8, 77, 0.1, 1.0, True, True, False),
    (300, 256, 9000, 0.2, 1.0, True, True, True)]


@pytest.mark.parametrize("N,H,V,ignored,T,gl,ge,bf16", GRADS)
@pytest.mark.parametrize("grid", [True, False])
def test_gradients(env, N, H, V, ignored, T, gl, ge, bf16, grid):
    flce, torch, dev = env
    X, W, t = problem(N, H, V, seed=N, ignored=ignored, grid=grid)
    r = np.random.default_rng(1)
    g = r.standard_normal(N).astype(np.float32) if gl else None
    e = r.standard_normal(N).astype(np.float32) if ge else None
    h, w, tt = to_gpu(torch, dev, X, W, t)
    up = lambda a: None if a is None else torch.from_numpy(a).to(dev)  # noqa: E731
    o = flce.token_logprobs(h, w, tt, temperature=T)
    kw = dict(temperature=T, grad_weight_dtype=torch.bfloat16 if bf16 else torch.float32)
    args = (h, w, tt, o["lse"], o["entropy"] if ge else None, up(g), up(e))
    d = flce.token_logprobs_bwd(*args, **kw)
    assert flce.query_status(d["workspace"]) == flce.FLCE_OK
    ref = logprobs_grad_oracle(X, W, t, g, e, temperature=T)
    for k, rounds in (("hidden", 1), ("weight", int(bf16))):
        tol = ref["mag_" + k] * (2.0 ** -8 + 2e-4) * (1 + 2.0 ** -8) + rounds * 2.0 ** -8 * np.abs(ref["grad_" + k])
        err = np.abs(np64(d["grad_" + k]) - ref["grad_" + k])
        assert np.all(err <= tol + 1e-30), (k, (err / (tol + 1e-30)).max())
    assert not d["grad_hidden"][tt == -100].any()
    # either gradient alone is the same, bit for bit
    one = flce.token_logprobs_bwd(*args, need_weight=False, **kw)
    two = flce.token_logprobs_bwd(*args, need_hidden=False, **kw)
    assert one["grad_weight"] is None and two["grad_hidden"] is None
    assert torch.equal(one["grad_hidden"], d["grad_hidden"]) and torch.equal(two["grad_weight"], d["grad_weight"])


@pytest.mark.parametrize("bf16", [False, True])
def test_gradients_in_chunks(env, bf16):
    """A workspace for 128 rows: grad_weight accumulates over chunks in fp32 and is rounded at the end."""
    flce, torch, dev = env
    N, H, V = 700, 136, 1000
    X, W, t = problem(N, H, V, seed=3, ignored=0.1)
    g = np.random.default_rng(1).standard_normal(N).astype(np.float32)
    h, w, tt = to_gpu(torch, dev, X, W, t)
    tg = torch.from_numpy(g).to(dev)
    dt = torch.bfloat16 if bf16 else torch.float32
    o = flce.token_logprobs(h, w, tt)
    nb = flce.workspace_bytes(N, H, V, chunk_rows=128, grad_weight_dtype=dt) + 4096   # and the rows' constants
    d = flce.token_logprobs_bwd(h, w, tt, o["lse"], None, tg, grad_weight_dtype=dt, workspace=flce.new_workspace(nb, dev))
    ref = logprobs_grad_oracle(X, W, t, g, None)
    for k, rounds in (("hidden", 1), ("weight", int(bf16))):
        tol = ref["mag_" + k] * (2.0 ** -8 + 2e-4) * (1 + 2.0 ** -8) + rounds * 2.0 ** -8 * np.abs(ref["grad_" + k])
        assert np.all(np.abs(np64(d["grad_" + k]) - ref["grad_" + k]) <= tol + 1e-30), k
    whole = flce.token_logprobs_bwd(h, w, tt, o["lse"], None, tg, grad_weight_dtype=dt)
    # complete per chunk, but the chunk size decides how the sum over the vocabulary is split: two fp32 sums of V terms
    # in other orders differ by at most 2 V 2^-24 of the sum of magnitudes, and each is rounded to bf16 (2^-8 of it)
    a, b = np64(whole["grad_hidden"]), np64(d["grad_hidden"])
    assert np.all(np.abs(a - b) <= 2 * V * 2.0 ** -24 * ref["mag_hidden"] * 1.01 + 2.0 ** -8 * (np.abs(a) + np.abs(b)))
    none = flce.token_logprobs_bwd(h, w, torch.full_like(tt, -100), o["lse"], None, tg, grad_weight_dtype=dt)
    assert not none["grad_hidden"].any() and not none["grad_weight"].any()


@pytest.mark.parametrize("N", [5, 200])
def test_ignore_index_inside_the_vocabulary(env, N):
    """Any int32 may be the ignore index, an id too."""
    flce, torch, dev = env
    X, W, t = problem(N, 64, 40, seed=3)
    h, w, tt = to_gpu(torch, dev, X, W, t)
    o = flce.token_logprobs(h, w, tt, ignore_index=int(t[0]), top_k=2)
    assert flce.query_status(o["workspace"]) == flce.FLCE_OK
    check_forward(o, logprobs_oracle(X, W, t, ignore_index=int(t[0]), top_k=2), 1.0, 2)
    d = flce.token_logprobs_bwd(h, w, tt, o["lse"], None, torch.ones(N, device=dev), ignore_index=int(t[0]))
    assert not d["grad_hidden"][tt == int(t[0])].any() and d["grad_hidden"].any()


def test_no_entropy_and_given_outputs(env):
    flce, torch, dev = env
    for N in (6, 260):
        X, W, t = problem(N, 64, 900, seed=3, ignored=0.2)
        h, w, tt = to_gpu(torch, dev, X, W, t)
        a = flce.token_logprobs(h, w, tt, entropy=False)
        b = flce.token_logprobs(h, w, tt)
        assert a["entropy"] is None and torch.equal(a["logp"], b["logp"]) and torch.equal(a["lse"], b["lse"])
        again = flce.token_logprobs(h, w, tt, out=b, workspace=b["workspace"])
        assert again is b and torch.equal(a["logp"], b["logp"])


def test_autograd_step(env):
    """A clipped policy-gradient loss through the module, against autograd in fp64."""
    flce, torch, dev = env
    N, H, V = 200, 128, 1500
    X, W, t = problem(N, H, V, seed=8, ignored=0.25)
    h, w, tt = to_gpu(torch, dev, X, W, t)
    adv = torch.randn(N, device=dev, generator=torch.Generator(device=dev).manual_seed(0))
    keep = tt != -100

    def loss(logp, ent, old, adv, keep):
        ratio = torch.exp(logp - old)
        obj = torch.minimum(ratio * adv, ratio.clamp(0.8, 1.2) * adv) + 0.01 * ent
        return -(obj * keep).sum() / keep.sum()

    m = flce.LinearLogProbs(w.clone())
    h.requires_grad_(True)
    logp, ent = m(h, tt)
    loss(logp, ent, logp.detach() - 0.05, adv, keep).backward()
    x, u = torch.from_numpy(X).requires_grad_(True), torch.from_numpy(W).requires_grad_(True)
    q = torch.log_softmax(x @ u.T, 1)
    at = torch.from_numpy(np.where(t < 0, 0, t)).long()[:, None]
    kc = keep.cpu()
    lp, en = q.gather(1, at)[:, 0] * kc, -(q.exp() * q).sum(1) * kc
    loss(lp, en, lp.detach() - 0.05, adv.double().cpu(), kc).backward()
    for a, b in ((h.grad, x.grad), (m.weight.grad, u.grad)):
        assert a.dtype == torch.bfloat16
        # dz and the output are each off by at most 2^-8 of themselves
        assert np.linalg.norm(np64(a) - b.numpy()) <= 2 * 2.0 ** -8 * np.linalg.norm(b.numpy())
    # a frozen head: only the hidden states' gradient
    h2 = h.detach().clone().requires_grad_(True)
    lp2, en2 = flce.linear_logprobs(h2, w, tt)
    loss(lp2, en2, lp2.detach() - 0.05, adv, keep).backward()
    assert torch.equal(h2.grad, h.grad)


def test_against_differences(env):
    """The gradient along a direction against differences of the forward (exact logits: a grid direction)."""
    flce, torch, dev = env
    N, H, V = 8, 64, 300
    X, W, t = problem(N, H, V, seed=6)
    h, w, tt = to_gpu(torch, dev, X, W, t)
    o = flce.token_logprobs(h, w, tt)
    one = torch.ones(N, device=dev)
    d = flce.token_logprobs_bwd(h, w, tt, o["lse"], o["entropy"], one, one)
    D = (np.arange(N * H).reshape(N, H) % 3 - 1) / 8.0
    f = [logprobs_oracle(X + s * D, W, t) for s in (1e-4, -1e-4)]
    want = sum(s * (q["logp"] + q["entropy"]).sum() for s, q in zip((1, -1), f)) / 2e-4
    ref = logprobs_grad_oracle(X, W, t, np.ones(N), np.ones(N))
    got = (np64(d["grad_hidden"]) * D).sum()
    assert abs(got - want) <= (ref["mag_hidden"] * np.abs(D)).sum() * 2 * 2.0 ** -8 + 1e-4


@pytest.mark.parametrize("N,K", [(5, 4), (300, 4)])
def test_captured_repeated_and_on_another_stream(env, N, K):
    """Replays on new inputs, two calls at once on two streams, and repeats are bitwise the eager call."""
    flce, torch, dev = env
    H, V = 128, 3000
    probs = [to_gpu(torch, dev, *problem(N, H, V, seed=s, ignored=0.2)) for s in (1, 2)]
    g = torch.randn(N, device=dev)

    def both(h, w, t, stream=None):
        o = flce.token_logprobs(h, w, t, top_k=K, stream=stream)
        d = flce.token_logprobs_bwd(h, w, t, o["lse"], o["entropy"], g, g, stream=stream)
        return [o[k] for k in ("logp", "entropy", "lse", "top_ids", "top_logp")] + [d["grad_hidden"], d["grad_weight"]]

    want = [both(*p) for p in probs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
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


@pytest.mark.parametrize("N", [3, 130])
def test_offsets_past_32_bits(env, N):
    """A weight of 2.3e9 elements (its gradient 9 GB), zero but for the last rows: logits in closed form."""
    flce, torch, dev = env
    V, H, m, K = 1_100_007, 2056, 40, 5
    X, tail, _ = problem(N, H, m, seed=N)
    w = torch.zeros(V, H, dtype=torch.bfloat16, device=dev)
    w[V - m:] = torch.from_numpy(tail).to(torch.bfloat16).to(dev)
    t = (V - 1 - np.arange(N) % (m + 5)).astype(np.int32)
    h = torch.from_numpy(X).to(torch.bfloat16).to(dev)
    o = flce.token_logprobs(h, w, torch.from_numpy(t).to(dev), top_k=K)
    z = X @ tail.T
    mx = np.maximum(z.max(1), 0)
    lse = mx + np.log((V - m) * np.exp(-mx) + np.exp(z - mx[:, None]).sum(1))
    at = t - (V - m)
    zt = np.where(at >= 0, z[np.arange(N), np.maximum(at, 0)], 0)
    # the sum of 8594 parts of equal terms is off by at most (128 + 8594) 2^-24 = 5.2e-4 of itself
    assert np.all(np.abs(np64(o["lse"]) - lse) <= 6e-4) and np.all(np.abs(np64(o["logp"]) - (zt - lse)) <= 6e-4)
    order = np.argsort(-z, axis=1, kind="stable")[:, :K]
    assert (np.take_along_axis(z, order, 1) > 0).all()
    np.testing.assert_array_equal(o["top_ids"].cpu().numpy(), order + V - m)
    g = np.random.default_rng(0).standard_normal(N).astype(np.float32)
    d = flce.token_logprobs_bwd(h, w, torch.from_numpy(t).to(dev), o["lse"], None, torch.from_numpy(g).to(dev))
    rows = np.r_[0, 1, V // 2, V - m - 1, V - m:V]
    zr = np.concatenate([np.zeros((N, 4)), z], 1)
    p = np.exp(zr - lse[:, None])
    hit = rows[None] == t[:, None]
    ref, mag = (g[:, None] * (hit - p)).T @ X, (np.abs(g)[:, None] * (hit + p)).T @ np.abs(X)
    got = np64(d["grad_weight"][torch.from_numpy(rows).to(dev)])
    assert np.all(np.abs(got - ref) <= mag * (2.0 ** -8 + 1e-3))
    ref_h = g[:, None] * (np.where(at >= 0, 1, 0)[:, None] * tail[np.maximum(at, 0)] - p[:, 4:] @ tail)
    mag_h = np.abs(g)[:, None] * (np.abs(tail[np.maximum(at, 0)]) + p[:, 4:] @ np.abs(tail))
    assert np.all(np.abs(np64(d["grad_hidden"]) - ref_h) <= mag_h * (2.0 ** -7 + 1e-3))


def test_python_refusals_on_gpu(env):
    flce, torch, dev = env
    X, W, t = problem(4, 64, 300, seed=1)
    h, w, tt = to_gpu(torch, dev, X, W, t)
    o = flce.token_logprobs(h, w, tt)
    one = torch.ones(4, device=dev)
    bad = [lambda: flce.token_logprobs(h.float(), w, tt), lambda: flce.token_logprobs(h, w, tt.long()),
           lambda: flce.token_logprobs(h.T.contiguous().T, w, tt), lambda: flce.token_logprobs(h, w, tt[:3]),
           lambda: flce.token_logprobs(h, w, tt, top_k=33), lambda: flce.token_logprobs(h, w, tt, top_k=-1),
           lambda: flce.token_logprobs(h, w, tt, temperature=0.0),
           lambda: flce.token_logprobs(h, w, tt, temperature=float("nan")),
           lambda: flce.token_logprobs(h, w, tt, out={"logp": torch.empty(5, device=dev)}),
           lambda: flce.token_logprobs(h, w, tt, out={"logp": torch.empty(4, device=dev, dtype=torch.float64)}),
           lambda: flce.token_logprobs(h, w, tt, workspace=flce.new_workspace(1024, dev)),
           lambda: flce.token_logprobs_bwd(h, w, tt, o["lse"], None, one, one),
           lambda: flce.token_logprobs_bwd(h, w, tt, o["lse"], o["entropy"], None, None),
           lambda: flce.token_logprobs_bwd(h, w, tt, o["lse"][:3], o["entropy"], one),
           lambda: flce.token_logprobs_bwd(h, w, tt, o["lse"], o["entropy"], one.half()),
           lambda: flce.token_logprobs_bwd(h, w, tt, o["lse"], o["entropy"], one, need_hidden=False, need_weight=False)]
    for f in bad:
        with pytest.raises((ValueError, TypeError, flce.FlceError)):
            f()


@pytest.mark.parametrize("N", [3, 128, 300])
def test_time_out_is_seen(env, N):
    """A withheld pipeline signal: the wait runs out, the status says so, and the outputs are NaN."""
    flce, torch, dev = env
    X, W, t = problem(N, 64, 2000, seed=1)
    h, w, tt = to_gpu(torch, dev, X, W, t)
    o = flce.token_logprobs(h, w, tt)
    flce.debug_arm_stall(50_000_000)
    b = flce.token_logprobs(h, w, tt)
    assert flce.query_status(b["workspace"]) == flce.FLCE_ETIMEOUT
    assert torch.isnan(b["logp"]).all() and torch.isnan(b["lse"]).all() and torch.isnan(b["entropy"]).all()
    flce.debug_arm_stall(50_000_000)
    d = flce.token_logprobs_bwd(h, w, tt, o["lse"], o["entropy"], o["logp"])
    assert flce.query_status(d["workspace"]) == flce.FLCE_ETIMEOUT
    assert torch.isnan(d["grad_hidden"][0, 0]) and torch.isnan(d["grad_weight"][0, 0])


@pytest.mark.parametrize("N,H,V,ignored", [(1, 64, 100, 1.0), (5, 72, 513, 0.5), (61, 256, 1000, 0.3), (128, 64, 2000, 1.0),
                                           (129, 64, 100, 0.97), (300, 64, 512, 0.3), (1030, 136, 5000, 0.3)])
def test_nothing_is_read_behind_ignored_targets(env, N, H, V, ignored):
    """NaN and inf in ignored tokens' rows and upstream gradients, and a workspace full of NaN, change no bit."""
    flce, torch, dev = env
    X, W, t = problem(N, H, V, seed=N, ignored=ignored)
    h, w, tt = to_gpu(torch, dev, X, W, t)
    off = tt == -100
    r = torch.Generator(device=dev).manual_seed(1)
    g, e = (torch.randn(N, generator=r, device=dev) for _ in range(2))

    def spoil(a, v):
        a = a.clone()
        a[off] = v
        return a

    bad = spoil(h, float("nan"))
    for K in (0, 5):
        a = flce.token_logprobs(h, w, tt, top_k=K)
        b = flce.token_logprobs(bad, w, tt, top_k=K, workspace=torch.full_like(a["workspace"], 255))
        for k in ("logp", "lse", "entropy") + (("top_ids", "top_logp") if K else ()):
            assert torch.equal(a[k], b[k]), (K, k)
    for dt in (torch.float32, torch.bfloat16):
        c = flce.token_logprobs_bwd(h, w, tt, a["lse"], a["entropy"], g, e, grad_weight_dtype=dt)
        d = flce.token_logprobs_bwd(bad, w, tt, spoil(a["lse"], float("nan")), spoil(a["entropy"], float("inf")),
                                    spoil(g, float("inf")), spoil(e, float("nan")), grad_weight_dtype=dt,
                                    workspace=torch.full_like(c["workspace"], 255))
        for k in ("grad_hidden", "grad_weight"):
            assert torch.isfinite(c[k]).all() and torch.equal(c[k], d[k]), (dt, k)


@pytest.mark.parametrize("N", [7, 300])
def test_gradient_of_bad_targets(env, N):
    """Targets outside the vocabulary add nothing to the gradients, as ignored ones, and set the status."""
    flce, torch, dev = env
    V = 300
    X, W, t = problem(N, 64, V, seed=2, ignored=0.2)
    h, w, tt = to_gpu(torch, dev, X, W, t)
    bad, left_out = tt.clone(), tt.clone()
    for i, v in ((1, V), (4, -7), (5, 2 ** 31 - 1), (6, -2 ** 31)):
        bad[i], left_out[i] = v, -100
    g = torch.randn(N, device=dev)
    o = flce.token_logprobs(h, w, bad)
    p = flce.token_logprobs(h, w, left_out)
    a = flce.token_logprobs_bwd(h, w, bad, o["lse"], o["entropy"], g, g)
    assert flce.query_status(a["workspace"]) == flce.FLCE_EBADTARGET
    b = flce.token_logprobs_bwd(h, w, left_out, p["lse"], p["entropy"], g, g)
    assert flce.query_status(b["workspace"]) == flce.FLCE_OK
    for k in ("grad_hidden", "grad_weight"):
        assert torch.equal(a[k], b[k]), k
