"""Constrained log probabilities against the fp64 oracle.

Tolerances (derived, not fitted).  On grid inputs every logit is exact in fp32,
and the rules are defined in fp32 steps, so the constrained logits are the same
bit for bit and the ids have to be equal.  Only the softmax rounds: the argument
of each 2^x is off by at most |x| 2^-23 (x up to ~60: 5e-6 of the term), the
approximate 2^x by 2^-22, and a sum of 128-term parts and of a list, P and L / 32
merges, by (128 + P + L / 32 + 5) 2^-24: with both under 200 below 3e-5 of each
sum (a merge's own factor adds 2^-22 of the smaller side each time, 200 of them
under 1e-5 once the sides are equal).  So logp and lse are off by at most 4e-5
plus 2^-22 of their size, the entropy by 4e-5 (1 + twice its size).
"""
import numpy as np
import pytest

from oracle.next_token_fp64 import constrained_oracle, rules_oracle

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


def head(N, H, V, seed):
    """Inputs on a grid: sums of products are exact in fp32."""
    r = np.random.default_rng(seed)
    std = 1.28 / np.sqrt(H)
    X, W = r.standard_normal((N, H)), std * r.standard_normal((V, H))
    X += W[r.integers(0, V, N)] * (10 * r.random((N, 1)) / (H * std * std))
    step = 2.0 ** np.round(np.log2(std / 10))
    return np.clip(np.round(X * 16), -64, 64) / 16, np.clip(np.round(W / step), -63, 63) * step


def pack(allowed):
    N, V = allowed.shape
    words = (V + 31) // 32
    bits = np.zeros((N, words * 32), bool)
    bits[:, :V] = allowed
    return np.packbits(bits, axis=1, bitorder="little").view(np.uint32).view(np.int32)


def rules(N, V, L, B, mask, seed):
    r = np.random.default_rng(seed + 1000)
    k = {}
    if L:
        h = np.minimum(r.zipf(1.3, (N, L)) - 1, V + 3).astype(np.int32)   # some outside the vocabulary
        h = np.where(r.random((N, L)) < 0.3, r.integers(-2, V, (N, L)), h).astype(np.int32)
        lens = r.integers(0, L + 1, N).astype(np.int32)
        lens[0] = L
        k.update(history=h, history_lens=lens, prompt_lens=(lens * r.random(N)).astype(np.int32),
                 repetition=(1 + 0.5 * r.random(N)).astype(np.float32), frequency=r.random(N).astype(np.float32),
                 presence=(r.random(N) - 0.3).astype(np.float32))
    if B:
        b = (3 * r.standard_normal((N, B))).astype(np.float32)
        b[r.random((N, B)) < 0.2] = -np.inf
        k.update(bias_ids=r.integers(-1, V + 1, (N, B)).astype(np.int32), bias=b)
    if mask:
        share = r.choice([0.0, 0.01, 0.5, 1.0], N, p=[0.1, 0.3, 0.3, 0.3])
        k["allowed"] = r.random((N, V)) < share[:, None]
    return k


def to_kw(torch, dev, k):
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
    names = {"repetition": "repetition_penalty", "frequency": "frequency_penalty", "presence": "presence_penalty"}
    kw = {names.get(n, n): up(a) for n, a in k.items() if n != "allowed"}
    if "allowed" in k:
        kw["mask"] = up(pack(k["allowed"]))
    return kw


def np64(a):
    return a.detach().double().cpu().numpy()


def near(got, want, tol, what):
    same = np.isneginf(want)
    np.testing.assert_array_equal(np.isneginf(got), same, err_msg=what)
    err = np.abs(np.where(same, 0, got) - np.where(same, 0, want))
    assert np.all(err <= tol + 2.0 ** -22 * np.where(same, 0, np.abs(want))), (what, np.nanmax(err))


def check(o, ref, K, scored, tol=4e-5):
    near(np64(o["lse"]), ref["lse"], tol, "lse")
    if scored:
        near(np64(o["logp"]), ref["logp"], tol, "logp")
    near(np64(o["entropy"]), ref["entropy"], tol * (1 + 2 * np.abs(ref["entropy"])), "entropy")
    if K:
        np.testing.assert_array_equal(o["top_ids"].cpu().numpy(), ref["top_ids"])
        near(np64(o["top_logp"]), ref["top_logp"], tol, "top_logp")


CASES = [  # N, H, V, K, L, B, mask, targets, T
    (1, 64, 1, 1, 3, 1, False, True, 1.0), (1, 8, 2, 2, 1, 0, True, False, 1.0),
    (1, 4096, 5003, 8, 57, 0, False, False, 1.0), (2, 72, 129, 32, 300, 7, True, True, 0.7),
    (5, 2048, 257, 1, 0, 5, False, True, 1.3), (16, 512, 16000, 5, 700, 0, True, False, 1.0),
    (17, 520, 1000, 20, 40, 40, False, True, 1.0), (33, 64, 31, 31, 9, 3, True, True, 1.0),
    (61, 136, 16007, 7, 2000, 16, True, False, 0.5), (64, 1024, 4096, 0, 33, 0, False, True, 1.0),
    (100, 264, 3001, 3, 0, 0, True, False, 2.0), (127, 128, 2000, 16, 513, 2, False, False, 1.0),
    (128, 128, 128, 32, 200, 9, True, True, 1.0), (128, 776, 70001, 8, 1000, 3, True, False, 1.0),
    (129, 64, 512, 9, 64, 0, True, True, 1.0), (257, 192, 1030, 4, 900, 11, True, False, 1.0),
    (300, 64, 512, 0, 0, 3, False, True, 0.9), (700, 520, 4099, 12, 100, 0, True, True, 1.0),
    (200, 8, 1, 1, 2, 2, True, True, 1.0), (200, 8, 300, 32, 310, 20, False, False, 1.0),
    (300, 1024, 9001, 6, 500, 4, True, True, 1.0), (131, 64, 40003, 8, 60, 0, False, False, 1.0),
    (150, 1024, 30000, 4, 900, 3, True, True, 1.0), (16500, 8, 300, 3, 20, 2, True, True, 1.0),
    (16500, 8, 40, 0, 9, 0, False, False, 1.0)]


@pytest.mark.parametrize("N,H,V,K,L,B,mask,scored,T", CASES)
def test_against_the_oracle(env, N, H, V, K, L, B, mask, scored, T):
    flce, torch, dev = env
    X, W = head(N, H, V, N + V)
    k = rules(N, V, L, B, mask, N)
    t = None
    if scored:
        t = np.random.default_rng(3).integers(0, V, N).astype(np.int32)
        t[np.random.default_rng(4).random(N) < 0.15] = -100
    f = lambda a: torch.from_numpy(a).to(torch.bfloat16).to(dev)  # noqa: E731
    o = flce.constrained_logprobs(f(X), f(W), None if t is None else torch.from_numpy(t).to(dev), temperature=T, top_k=K,
                                  **to_kw(torch, dev, k))
    assert flce.query_status(o["workspace"]) == flce.FLCE_OK
    assert (o["logp"] is None) == (t is None)
    check(o, constrained_oracle(rules_oracle(X @ W.T, **k), t, temperature=T, top_k=K), K, scored)


@pytest.mark.parametrize("N", [7, 200])
def test_without_rules_as_the_plain_operator(env, N):
    """No rule at all, and rules that change nothing, give what token_logprobs gives."""
    flce, torch, dev = env
    X, W = head(N, 128, 3000, 1)
    f = lambda a: torch.from_numpy(a).to(torch.bfloat16).to(dev)  # noqa: E731
    h, w, t = f(X), f(W), torch.arange(N, device=dev, dtype=torch.int32)
    a = flce.token_logprobs(h, w, t, top_k=9)
    b = flce.constrained_logprobs(h, w, t, top_k=9)
    for k in ("logp", "lse", "entropy", "top_ids", "top_logp"):
        assert torch.equal(a[k], b[k]), k
    ones = torch.ones(N, device=dev)
    c = flce.constrained_logprobs(h, w, t, top_k=9, history=torch.randint(0, 3000, (N, 50), device=dev, dtype=torch.int32),
                                  repetition_penalty=ones, frequency_penalty=0 * ones,
                                  mask=torch.full((N, 94), -1, dtype=torch.int32, device=dev))
    assert torch.equal(a["top_ids"], c["top_ids"])
    # 50 terms are added in another order: each sum is off by 3e-5 at most (above)
    torch.testing.assert_close(a["lse"], c["lse"], atol=8e-5, rtol=0)


@pytest.mark.parametrize("N", [9, 200])
def test_forbidden_places_may_hold_anything(env, N):
    """Weight rows of NaN and infinity behind the mask, rows of hidden states with NaN, rows that are left empty."""
    flce, torch, dev = env
    V = 2000
    X, W = head(N, 64, V, 2)
    k = rules(N, V, 300, 0, True, 2)
    k["allowed"][:] = np.random.default_rng(0).random((N, V)) < 0.5
    k["allowed"][:, [5, 700, 1999]] = False
    k["allowed"][4] = False
    ref = constrained_oracle(rules_oracle(X @ W.T, **k), np.full(N, 5, np.int32), top_k=5)
    f = lambda a: torch.from_numpy(a).to(torch.bfloat16).to(dev)  # noqa: E731
    h, w = f(X), f(W)
    w[5], w[700], w[1999] = float("nan"), float("inf"), -float("inf")
    h[2, 3] = float("nan")
    o = flce.constrained_logprobs(h, w, torch.full((N,), 5, dtype=torch.int32, device=dev), top_k=5,
                                  **to_kw(torch, dev, k))
    assert torch.isnan(o["lse"][2]) and torch.isnan(o["entropy"][2]) and torch.isnan(o["top_logp"][2]).all()
    assert (o["top_ids"][2] == -1).all()
    keep = [i for i in range(N) if i != 2]
    assert np.isneginf(np64(o["logp"])[keep]).all()
    got = {n: o[n][keep] for n in ("lse", "logp", "entropy", "top_ids", "top_logp")}
    check(got, {n: (v[keep] if isinstance(v, np.ndarray) else v) for n, v in ref.items()}, 5, True)
    assert got["lse"][keep.index(4)] == -float("inf")


@pytest.mark.parametrize("N", [6, 150])
def test_all_but_one_forbidden(env, N):
    flce, torch, dev = env
    V = 777
    X, W = head(N, 64, V, 3)
    allowed = np.zeros((N, V), bool)
    one = np.random.default_rng(0).integers(0, V, N)
    allowed[np.arange(N), one] = True
    f = lambda a: torch.from_numpy(a).to(torch.bfloat16).to(dev)  # noqa: E731
    o = flce.constrained_logprobs(f(X), f(W), torch.from_numpy(one.astype(np.int32)).to(dev), top_k=3,
                                  mask=torch.from_numpy(pack(allowed)).to(dev))
    assert o["top_ids"][:, 0].tolist() == one.tolist() and (o["top_ids"][:, 1:] == -1).all()
    assert not o["logp"].any()   # relative to the largest logit: 2^0 = 1, log2 1 = 0, exactly
    # The one term of the entropy is taken at the rounded product of the largest logit (|z| < 64 here) and log2(e): its
    # exponent is off by rho <= 2^-24 * 128, and what is left once rho is taken out again is rho (2^rho - 1), with an
    # approximate 2^x (2^-22): under 7.7e-6 * (7.7e-6 + 2.4e-7) < 1e-10.
    assert (o["entropy"].abs() <= 1e-10).all()
    assert not o["top_logp"][:, 0].any() and torch.isneginf(o["top_logp"][:, 1:]).all()


@pytest.mark.parametrize("N", [4, 140])
def test_strided_and_shared_rows(env, N):
    """Rows apart, one row for all, lengths past the arrays, and unaligned starts."""
    flce, torch, dev = env
    V, L = 1500, 61
    X, W = head(N, 64, V, 4)
    k = rules(N, V, L, 5, True, 4)
    f = lambda a: torch.from_numpy(a).to(torch.bfloat16).to(dev)  # noqa: E731
    h, w, kw = f(X), f(W), to_kw(torch, dev, k)
    want = flce.constrained_logprobs(h, w, top_k=4, **kw)

    def apart(a, fill):
        wide = torch.full((N, a.shape[1] + 7), fill, dtype=a.dtype, device=dev)
        wide[:, 3:3 + a.shape[1]] = a
        return wide[:, 3:3 + a.shape[1]]

    far = dict(kw, history=apart(kw["history"], 11), bias_ids=apart(kw["bias_ids"], 12), bias=apart(kw["bias"], 99.0),
               mask=apart(kw["mask"], 0))
    got = flce.constrained_logprobs(h, w, top_k=4, **far)
    for n in ("lse", "entropy", "top_ids", "top_logp"):
        assert torch.equal(got[n], want[n]), n
    long = dict(kw, history_lens=torch.where(kw["history_lens"] == L, 1 << 30, kw["history_lens"]))
    assert torch.equal(flce.constrained_logprobs(h, w, top_k=4, **long)["lse"], want["lse"])
    shared = flce.constrained_logprobs(h, w, top_k=4, history=kw["history"][1:2].expand(N, -1),
                                       history_lens=torch.arange(N, device=dev, dtype=torch.int32),
                                       repetition_penalty=kw["repetition_penalty"], mask=kw["mask"][:1].expand(N, -1))
    kk = dict(history=np.repeat(k["history"][1:2], N, 0), history_lens=np.arange(N), repetition=k["repetition"],
              allowed=np.repeat(k["allowed"][:1], N, 0))
    check(shared, constrained_oracle(rules_oracle(X @ W.T, **kk), top_k=4), 4, False)


@pytest.mark.parametrize("N", [3, 700])
def test_small_workspace_and_outputs_left_alone(env, N):
    flce, torch, dev = env
    V = 2000
    X, W = head(N, 128, V, 5)
    k = rules(N, V, 100, 4, True, 5)
    f = lambda a: torch.from_numpy(a).to(torch.bfloat16).to(dev)  # noqa: E731
    h, w, kw = f(X), f(W), to_kw(torch, dev, k)
    t = torch.arange(N, device=dev, dtype=torch.int32) % V
    t[1] = -100
    a = flce.constrained_logprobs(h, w, t, top_k=6, **kw)
    need = flce.library().flce_constrained_workspace_bytes(N, 128, V, 6, 100, 4)
    lo, hi = 0, need
    while hi - lo > 256:   # the smallest workspace that is accepted
        mid = (lo + hi) // 2
        try:
            flce.constrained_logprobs(h, w, t, top_k=6, workspace=flce.new_workspace(mid, dev), **kw)
            hi = mid
        except flce.FlceError as e:
            assert e.status == flce.FLCE_EWORKSPACE
            lo = mid
    assert N <= 128 or hi < need
    ws = torch.full((hi + 4096,), 171, dtype=torch.uint8, device=dev)
    big = torch.full((N + 8,), 7.0, device=dev)
    out = {"lse": big[:N]}
    b = flce.constrained_logprobs(h, w, t, top_k=6, workspace=ws[:hi], out=out, **kw)
    assert (big[N:] == 7).all() and (ws[hi:] == 171).all()
    for n in ("logp", "entropy", "lse", "top_ids", "top_logp"):
        assert torch.equal(a[n], b[n]), n
    bad = t.clone()
    bad[2] = V
    c = flce.constrained_logprobs(h, w, bad, top_k=6, workspace=ws[:hi], **kw)
    assert flce.query_status(ws[:hi]) == flce.FLCE_EBADTARGET
    assert torch.isnan(c["lse"][2]) and (c["top_ids"][2] == -1).all() and not c["lse"][1] and torch.equal(c["lse"][3:], a["lse"][3:])


@pytest.mark.parametrize("N", [2, 130])
def test_more_tokens_than_a_window(env, N):
    """Vocabularies whose bitmap does not fit in shared memory at once."""
    flce, torch, dev = env
    V = 786432 * 2 + 77
    X, W = head(N, 8, V, 6)
    r = np.random.default_rng(1)
    h = r.integers(0, V, (N, 900)).astype(np.int32)
    h[:, :6] = [0, 786431, 786432, 786433, V - 1, 1572864]
    bias_ids = np.tile(np.array([786432, V - 1, 5], np.int32), (N, 1))
    bias = np.tile(np.array([20.0, 21.0, 22.0], np.float32), (N, 1))
    k = dict(history=h, repetition=np.full(N, 1.5, np.float32), frequency=np.full(N, 0.5, np.float32), bias_ids=bias_ids,
             bias=bias)
    f = lambda a: torch.from_numpy(a).to(torch.bfloat16).to(dev)  # noqa: E731
    o = flce.constrained_logprobs(f(X), f(W), top_k=5, **to_kw(torch, dev, k))
    rows = [0, 1, N - 1]
    kk = {n: a[rows] for n, a in k.items()}
    ref = constrained_oracle(rules_oracle(X[rows] @ W.T, **kk), top_k=5)
    assert o["top_ids"][rows].cpu().tolist() == ref["top_ids"].tolist()
    # 12289 parts: (128 + 12289 / 32) 2^-24 of merges in sequence, and as many 2^-22 of their factors: 1.6e-4
    np.testing.assert_allclose(np64(o["lse"])[rows], ref["lse"], atol=2e-4)


@pytest.mark.parametrize("N", [5, 260])
def test_captured_and_on_another_stream(env, N):
    """A captured call replayed on new data, and calls on two streams at once."""
    flce, torch, dev = env
    V = 3000
    f = lambda a: torch.from_numpy(a).to(torch.bfloat16).to(dev)  # noqa: E731
    sets = []
    for seed in (1, 2):
        X, W = head(N, 64, V, seed)
        kw = to_kw(torch, dev, rules(N, V, 200, 3, True, seed))
        sets.append((f(X), f(W), kw, flce.constrained_logprobs(f(X), f(W), top_k=4, **kw)))
    h, w = sets[0][0].clone(), sets[0][1].clone()
    kw = {n: a.clone() for n, a in sets[0][2].items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        flce.constrained_logprobs(h, w, top_k=4, **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = flce.constrained_logprobs(h, w, top_k=4, **kw)
    for s in (1, 0):
        h.copy_(sets[s][0])
        w.copy_(sets[s][1])
        for n in kw:
            kw[n].copy_(sets[s][2][n])
        graph.replay()
        for n in ("lse", "entropy", "top_ids", "top_logp"):
            assert torch.equal(o[n], sets[s][3][n]), n
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [flce.constrained_logprobs(x, y, top_k=4, stream=st, **z) for st, (x, y, z, _) in zip(streams, sets)]
    torch.cuda.synchronize()
    for g, s in zip(got, sets):
        assert torch.equal(g["lse"], s[3]["lse"]) and torch.equal(g["top_ids"], s[3]["top_ids"])


@pytest.mark.parametrize("N", [8, 300])
def test_time_out_marks_every_row(env, N):
    flce, torch, dev = env
    X, W = head(N, 64, 900, 7)
    f = lambda a: torch.from_numpy(a).to(torch.bfloat16).to(dev)  # noqa: E731
    kw = to_kw(torch, dev, rules(N, 900, 30, 0, True, 7))
    good = flce.constrained_logprobs(f(X), f(W), top_k=3, **kw)
    flce.debug_arm_stall(20_000_000)
    o = flce.constrained_logprobs(f(X), f(W), top_k=3, **kw)
    assert flce.query_status(o["workspace"]) == flce.FLCE_ETIMEOUT
    assert torch.isnan(o["lse"]).all() and (o["top_ids"] == -1).all() and torch.isnan(o["top_logp"]).all()
    again = flce.constrained_logprobs(f(X), f(W), top_k=3, **kw)
    assert flce.query_status(again["workspace"]) == flce.FLCE_OK and torch.equal(again["lse"], good["lse"])


@pytest.mark.parametrize("N", [3, 130])
def test_rows_further_apart_than_32_bits(env, N):
    """Rows of the matrices whose offsets, in elements, pass 2^31."""
    flce, torch, dev = env
    V, L, B = 700, 40, 3
    X, W = head(N, 64, V, 8)
    k = rules(N, V, L, B, True, 8)
    f = lambda a: torch.from_numpy(a).to(torch.bfloat16).to(dev)  # noqa: E731
    kw = to_kw(torch, dev, k)
    want = flce.constrained_logprobs(f(X), f(W), top_k=4, **kw)
    stride = (1 << 31) // (N - 1) + 64
    ints = torch.empty((N - 1) * stride + 256, dtype=torch.int32, device=dev)
    assert (N - 1) * stride > 1 << 31

    def far(a, at):
        flat = ints if a.dtype == torch.int32 else ints.view(torch.float32)
        v = flat[at:].as_strided((N, a.shape[1]), (stride, 1), at)
        v.copy_(a)
        return v

    far_kw = dict(kw, history=far(kw["history"], 0), bias_ids=far(kw["bias_ids"], 50), bias=far(kw["bias"], 60),
                  mask=far(kw["mask"], 70))
    assert far_kw["history"].stride(0) == stride
    got = flce.constrained_logprobs(f(X), f(W), top_k=4, **far_kw)
    for n in ("lse", "entropy", "top_ids", "top_logp"):
        assert torch.equal(got[n], want[n]), n


@pytest.mark.parametrize("N", [2, 140])
def test_one_token_said_very_often(env, N):
    """Histories longer than a block holds, of few different tokens."""
    flce, torch, dev = env
    V, L = 900, 30011
    X, W = head(N, 64, V, 9)
    r = np.random.default_rng(9)
    h = np.where(r.random((N, L)) < 0.7, 17, r.integers(0, 30, (N, L))).astype(np.int32)
    k = dict(history=h, prompt_lens=np.full(N, 11, np.int32), frequency=np.full(N, 2.0 ** -12, np.float32),
             repetition=np.full(N, 1.25, np.float32))
    f = lambda a: torch.from_numpy(a).to(torch.bfloat16).to(dev)  # noqa: E731
    o = flce.constrained_logprobs(f(X), f(W), top_k=6, **to_kw(torch, dev, k))
    rows = [0, N - 1]
    ref = constrained_oracle(rules_oracle(X[rows] @ W.T, **{n: a[rows] for n, a in k.items()}), top_k=6)
    check({n: o[n][rows] for n in ("lse", "entropy", "top_ids", "top_logp")}, ref, 6, False)


@pytest.mark.parametrize("N", [3, 140])
@pytest.mark.parametrize("V,L", [(900, 1279), (900, 1280), (8192, 4096), (8193, 4097), (16000, 30000), (300000, 24001)])
def test_times_of_long_histories(env, N, V, L):
    """Around the length at which times are counted apart, and more different tokens than are counted so (8192)."""
    flce, torch, dev = env
    X, W = head(N, 64, V, 13)
    r = np.random.default_rng(13)
    h = r.integers(0, V, (N, L)).astype(np.int32)
    h[:, r.random(L) < 0.2] = V - 1
    k = dict(history=h, prompt_lens=r.integers(0, L + 1, N).astype(np.int32), frequency=np.full(N, 2.0 ** -10, np.float32),
             presence=np.full(N, 0.25, np.float32), repetition=np.full(N, 1.25, np.float32))
    f = lambda a: torch.from_numpy(a).to(torch.bfloat16).to(dev)  # noqa: E731
    o = flce.constrained_logprobs(f(X), f(W), top_k=6, **to_kw(torch, dev, k))
    rows = [0, 1, N - 1]
    ref = constrained_oracle(rules_oracle(X[rows] @ W.T, **{n: a[rows] for n, a in k.items()}), top_k=6)
    # 2344 parts at most: (128 + 2344 / 32) 2^-24 of merges in sequence, and as many 2^-22 of their factors: 6e-5
    check({n: o[n][rows] for n in ("lse", "entropy", "top_ids", "top_logp")}, ref, 6, False, 4e-5 if V < 70000 else 8e-5)


@pytest.mark.parametrize("N", [6, 150])
def test_repeated_calls_agree_bit_for_bit(env, N):
    flce, torch, dev = env
    X, W = head(N, 64, 2000, 10)
    kw = to_kw(torch, dev, rules(N, 2000, 3000, 40, True, 10))
    f = lambda a: torch.from_numpy(a).to(torch.bfloat16).to(dev)  # noqa: E731
    a = flce.constrained_logprobs(f(X), f(W), top_k=7, **kw)
    for _ in range(5):
        b = flce.constrained_logprobs(f(X), f(W), top_k=7, **kw)
        for n in ("lse", "entropy", "top_ids", "top_logp"):
            assert torch.equal(a[n], b[n]), n


def test_empty_histories_and_biases(env):
    flce, torch, dev = env
    for N in (4, 140):
        X, W = head(N, 64, 500, 11)
        f = lambda a: torch.from_numpy(a).to(torch.bfloat16).to(dev)  # noqa: E731
        h, w = f(X), f(W)
        ones = torch.ones(N, device=dev)
        want = flce.constrained_logprobs(h, w, top_k=3)
        got = flce.constrained_logprobs(h, w, top_k=3, history=torch.zeros((N, 0), dtype=torch.int32, device=dev),
                                        repetition_penalty=2 * ones, presence_penalty=ones,
                                        bias_ids=torch.zeros((N, 0), dtype=torch.int32, device=dev),
                                        bias=torch.zeros((N, 0), device=dev))
        none = flce.constrained_logprobs(h, w, top_k=3, history=torch.zeros((N, 9), dtype=torch.int32, device=dev),
                                         history_lens=torch.zeros(N, dtype=torch.int32, device=dev), presence_penalty=ones)
        for o in (got, none):
            for n in ("lse", "entropy", "top_ids", "top_logp"):
                assert torch.equal(o[n], want[n]), n
