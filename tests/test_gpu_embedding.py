"""The scaled embedding and its gradient against fp64, and a tied model that
runs embedding, LM-head log probabilities and both gradients.

Tolerances: the lookup rounds the fp32 product scale * w (2^-24 of it) and then
to the output type (finfo.eps / 2).  The gradient's sum of c rows is off by at
most c 2^-24 of the sum of magnitudes, the scaling and an accumulation by 2^-24
each, and the output type by finfo.eps / 2.
"""
import numpy as np
import pytest

from oracle.logprobs_fp64 import embedding_grad_oracle, embedding_oracle, logprobs_grad_oracle, logprobs_oracle
from tests.test_gpu_logprobs import env, np64, problem, to_gpu  # noqa: F401

pytestmark = pytest.mark.gpu

TYPES = ["bfloat16", "float16", "float32"]


def draw_ids(N, V, kind, seed=0):
    r = np.random.default_rng(seed)
    if kind == "zipf":
        p = np.arange(1, V + 1) ** -1.1
        return r.permutation(V)[r.choice(V, N, p=p / p.sum())].astype(np.int32)
    if kind == "one":
        return np.full(N, V - 1, np.int32)
    if kind == "sorted":
        return np.sort(r.integers(0, V, N)).astype(np.int32)
    return r.integers(0, V, N).astype(np.int32)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N,H,V,scale", [(1, 8, 1, 1.0), (3, 4096, 5, 64.0), (61, 520, 1000, 22.627417), (5000, 72, 333, -0.5)])
def test_lookup(env, dtype, N, H, V, scale):  # noqa: F811
    flce, torch, dev = env
    dt = getattr(torch, dtype)
    W = torch.randn(V, H, generator=torch.Generator().manual_seed(N)).to(dt)
    ids = draw_ids(N, V, "uniform")
    out = flce.embedding_fwd(W.to(dev), torch.from_numpy(ids).to(dev), scale)
    ref = embedding_oracle(W.double().numpy(), ids, np.float32(scale))
    tol = (torch.finfo(dt).eps / 2 + 2.0 ** -24) * np.abs(ref) + 2.0 ** -25 * (dtype == "float16")
    assert out.dtype == dt and np.all(np.abs(np64(out) - ref) <= tol)


def test_lookup_bad_ids_and_rows_behind(env):  # noqa: F811
    flce, torch, dev = env
    W = torch.randn(50, 64, device=dev).to(torch.bfloat16)
    ids = torch.tensor([3, -1, 50, 49, 2 ** 31 - 1], dtype=torch.int32, device=dev)
    buf = torch.full((7, 64), 5.0, device=dev, dtype=torch.bfloat16)
    flce.embedding_fwd(W, ids, 2.0, out=buf[:5])
    assert torch.isnan(buf[[1, 2, 4]]).all() and (buf[5:] == 5).all()
    assert torch.equal(buf[[0, 3]], 2 * W[[3, 49]])


CASES = [(1, 8, 1, "one"), (1, 64, 1000, "uniform"), (31, 264, 7, "uniform"), (32, 64, 40, "sorted"),
         (33, 72, 3, "zipf"), (4096, 136, 511, "uniform"), (4097, 64, 512, "zipf"), (10000, 520, 16000, "zipf"),
         (9000, 40, 513, "one"), (20001, 64, 262143, "uniform"), (5000, 8, 262144, "sorted"), (3000, 2048, 100, "zipf"),
         (70000, 16, 1200000, "zipf")]


@pytest.mark.parametrize("N,H,V,kind", CASES)
@pytest.mark.parametrize("dtype,grad", [("bfloat16", "float32"), ("float32", "float32"), ("float16", "float16"),
                                        ("bfloat16", "bfloat16")])
def test_gradient(env, N, H, V, kind, dtype, grad):  # noqa: F811
    flce, torch, dev = env
    dt, gt = getattr(torch, dtype), getattr(torch, grad)
    ids = draw_ids(N, V, kind, seed=N)
    d = torch.randn(N, H, generator=torch.Generator().manual_seed(V)).to(dt)
    pad = int(ids[N // 2]) if N > 40 else None
    scale = 0.37
    args = (d.to(dev), torch.from_numpy(ids).to(dev), V, scale, pad)
    o = flce.embedding_bwd(*args, grad_weight_dtype=gt)
    assert flce.query_status(o["workspace"]) == flce.FLCE_OK
    ref, mag = embedding_grad_oracle(d.double().numpy(), ids, V, np.float32(scale), pad)
    c = np.bincount(ids, minlength=V)[:, None]
    tol = (c + 2) * 2.0 ** -24 * mag + (torch.finfo(gt).eps / 2) * np.abs(ref) + 2.0 ** -25 * (grad == "float16")
    assert np.all(np.abs(np64(o["grad_weight"]) - ref) <= tol)
    again = flce.embedding_bwd(*args, grad_weight_dtype=gt)
    assert torch.equal(o["grad_weight"], again["grad_weight"])


@pytest.mark.parametrize("N,H,V,kind", [(16384, 16, 300, "zipf"), (16385, 16, 300, "zipf"), (131072, 8, 70000, "zipf"),
                                        (140001, 8, 5000, "zipf"), (300001, 8, 90, "uniform"), (300001, 8, 3, "one")])
def test_gradient_of_many_tokens(env, N, H, V, kind):  # noqa: F811
    """Every form of the sort, chunks of more than 64 tokens, and runs of thousands of chunks."""
    flce, torch, dev = env
    ids = draw_ids(N, V, kind, seed=N)
    d = torch.randn(N, H, generator=torch.Generator().manual_seed(V))
    o = flce.embedding_bwd(d.to(dev), torch.from_numpy(ids).to(dev), V, 1.5)
    assert flce.query_status(o["workspace"]) == flce.FLCE_OK
    ref, mag = np.zeros((V, H)), np.zeros((V, H))
    np.add.at(ref, ids, 1.5 * d.double().numpy())
    np.add.at(mag, ids, 1.5 * d.abs().double().numpy())
    c = np.bincount(ids, minlength=V)[:, None]
    assert np.all(np.abs(np64(o["grad_weight"]) - ref) <= (c + 2) * 2.0 ** -24 * mag)


@pytest.mark.parametrize("N,H,V,kind", [(1, 64, 9, "one"), (5000, 264, 700, "zipf"), (300, 64, 20000, "uniform")])
def test_accumulate(env, N, H, V, kind):  # noqa: F811
    flce, torch, dev = env
    ids = draw_ids(N, V, kind)
    d = torch.randn(N, H, device=dev).to(torch.bfloat16)
    base = torch.randn(V, H, device=dev)
    base[0] = float("nan")   # a row that is not touched is not read either
    if 0 in ids:
        ids[ids == 0] = V - 1
    g = base.clone()
    t = torch.from_numpy(ids).to(dev)
    flce.embedding_bwd(d, t, V, 2.0, accumulate=True, out={"grad_weight": g})
    ref, mag = embedding_grad_oracle(np64(d), ids, V, 2.0)
    c = np.bincount(ids, minlength=V)[:, None]
    b = np64(base)
    tol = (c + 2) * 2.0 ** -24 * mag + 2.0 ** -24 * (np.abs(b) + mag)
    assert np.all(np.abs(np64(g) - (b + ref))[1:] <= tol[1:])
    rest = torch.ones(V, dtype=torch.bool, device=dev)
    rest[t.long()] = False
    assert torch.equal(g[rest].nan_to_num(7), base[rest].nan_to_num(7))


def test_offsets_past_32_bits(env):  # noqa: F811
    """A table of 2.3e9 elements, its last rows looked up; a gradient of 9 GB, zero elsewhere."""
    flce, torch, dev = env
    V, H, N = 1_100_007, 2056, 300
    W = torch.zeros(V, H, dtype=torch.bfloat16, device=dev)
    W[V - 50:] = torch.randn(50, H, device=dev).to(torch.bfloat16)
    ids = V - 1 - (torch.arange(N, device=dev, dtype=torch.int32) * 7) % 50
    out = flce.embedding_fwd(W, ids, 2.0)
    assert torch.equal(out, 2 * W[ids.long()])
    g = flce.embedding_bwd(out, ids, V)["grad_weight"]
    ref, mag = embedding_grad_oracle(np64(out), (ids - (V - 50)).cpu().numpy(), 50)
    assert np.all(np.abs(np64(g[V - 50:]) - ref) <= 8 * 2.0 ** -24 * mag)
    assert not g[:V - 50].any()


def test_gradient_bad_ids(env):  # noqa: F811
    flce, torch, dev = env
    d = torch.randn(6, 64, device=dev)
    ids = torch.tensor([2, -1, 10, 2, 9, -2 ** 31], dtype=torch.int32, device=dev)
    o = flce.embedding_bwd(d, ids, 10)
    assert flce.query_status(o["workspace"]) == flce.FLCE_EBADTARGET
    want = torch.zeros(10, 64, device=dev)
    want[2], want[9] = d[0] + d[3], d[4]
    assert torch.equal(o["grad_weight"], want)
    none = flce.embedding_bwd(d, torch.full((6,), 4, dtype=torch.int32, device=dev), 10, padding_idx=4)
    assert flce.query_status(none["workspace"]) == flce.FLCE_OK and not none["grad_weight"].any()


def test_gradient_captured_and_on_two_streams(env):  # noqa: F811
    flce, torch, dev = env
    N, H, V = 6000, 128, 900
    ds = [torch.randn(N, H, device=dev).to(torch.bfloat16) for _ in range(2)]
    ids = [torch.from_numpy(draw_ids(N, V, "zipf", s)).to(dev) for s in range(2)]
    want = [flce.embedding_bwd(d, i, V)["grad_weight"] for d, i in zip(ds, ids)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = [flce.embedding_bwd(d, i, V, stream=s)["grad_weight"] for d, i, s in zip(ds, ids, streams)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    d, i = ds[0].clone(), ids[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = flce.embedding_bwd(d, i, V)["grad_weight"]
    for k in (1, 0):
        d.copy_(ds[k])
        i.copy_(ids[k])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[k])


def test_python_refusals_on_gpu(env):  # noqa: F811
    flce, torch, dev = env
    W, d = torch.zeros(10, 64, device=dev), torch.zeros(3, 64, device=dev)
    ids = torch.zeros(3, dtype=torch.int32, device=dev)
    bad = [lambda: flce.embedding_fwd(W.double(), ids), lambda: flce.embedding_fwd(W, ids.long()),
           lambda: flce.embedding_fwd(W[:, :60].contiguous(), ids), lambda: flce.embedding_fwd(W[:, :32], ids),
           lambda: flce.embedding_fwd(W.cpu(), ids), lambda: flce.embedding_fwd(W, ids.cpu()),
           lambda: flce.embedding_fwd(W, ids, out=torch.empty(3, 64, device=dev, dtype=torch.bfloat16)),
           lambda: flce.embedding_fwd(W, ids[:0]), lambda: flce.embedding_bwd(d, ids[:2], 10),
           lambda: flce.embedding_bwd(d, ids, 10, padding_idx=10), lambda: flce.embedding_bwd(d, ids, 10, accumulate=True),
           lambda: flce.embedding_bwd(d, ids, 0), lambda: flce.embedding(ids, W, padding_idx=-1),
           lambda: flce.embedding_bwd(d, ids, 10, workspace=flce.new_workspace(256, dev)),
           lambda: flce.embedding_bwd(d, ids, 10, grad_weight_dtype=torch.bfloat16, accumulate=True,
                                      out={"grad_weight": W.bfloat16()})]
    for f in bad:
        with pytest.raises((ValueError, TypeError, flce.FlceError)):
            f()


def test_captured_training_step(env):  # noqa: F811
    """Embedding, head and both gradients of a tied weight captured as one graph and replayed on new tokens."""
    flce, torch, dev = env
    N, H, V = 300, 64, 700
    _, W, t = problem(N, H, V, seed=3, ignored=0.1)
    w = torch.from_numpy(W).to(torch.bfloat16).to(dev)
    adv = torch.randn(N, device=dev)
    batches = [(torch.from_numpy(draw_ids(N, V, "zipf", s)).to(dev), torch.from_numpy(np.roll(t, s)).to(dev))
               for s in range(2)]

    def step(ids, targets):
        leaf = w.detach().requires_grad_(True)
        x = flce.embedding(ids, leaf, 8.0)
        logp, ent = flce.linear_logprobs(x, leaf, targets)
        loss = (logp * adv).sum() + 0.01 * ent.sum()
        return loss.detach(), torch.autograd.grad(loss, leaf)[0]

    want = [step(*b) for b in batches]
    ids, targets = (x.clone() for x in batches[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(ids, targets)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(ids, targets)
    for b, a in ((batches[1], want[1]), (batches[0], want[0])):
        ids.copy_(b[0])
        targets.copy_(b[1])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], a[0]) and torch.equal(out[1], a[1])


@pytest.mark.parametrize("leaf", ["hidden", "weight", "table"])
def test_capture_beside_a_living_graph(env, leaf):  # noqa: F811
    """A backward captured while an eager graph of the same leaf lives on the default stream is refused, before
    autograd orders that stream behind the capture; the forward alone, and the step once the graph is gone, are not."""
    flce, torch, dev = env
    N, H, V = 300, 64, 700
    X, W, t = problem(N, H, V, seed=5, ignored=0.1)
    x, w = (torch.from_numpy(a).to(torch.bfloat16).to(dev) for a in (X, W))
    t = torch.from_numpy(t).to(dev)
    ids = torch.from_numpy(draw_ids(N, V, "zipf", 2)).to(dev)
    up = torch.randn(N, H, device=dev, dtype=torch.bfloat16)
    u = {"hidden": x, "weight": w, "table": w}[leaf].clone().requires_grad_(True)

    def forward():
        if leaf == "table":
            return (flce.embedding(ids, u) * up).sum()
        return flce.linear_logprobs(*((u, w) if leaf == "hidden" else (x, u)), t)[0].sum()

    loss = forward()
    want = torch.autograd.grad(loss, u, retain_graph=True)[0]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        value = forward()
    graph.replay()
    assert torch.equal(value, loss)
    del value
    with pytest.raises(RuntimeError, match="alive"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            torch.autograd.grad(forward(), u)
    del loss
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = torch.autograd.grad(forward(), u)[0]
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_tied_model(env):  # noqa: F811
    """ids -> scaled embedding -> x + tanh(x) -> log probabilities against the same weight; both
    gradients through autograd, and through the calls that add into one fp32 grad_weight."""
    flce, torch, dev = env
    N, H, V, scale = 260, 64, 500, 8.0
    _, W, t = problem(N, H, V, seed=11, ignored=0.2)
    ids = draw_ids(N, V, "zipf", 3)
    g = np.random.default_rng(2).standard_normal(N).astype(np.float32)
    w = torch.from_numpy(W).to(torch.bfloat16).to(dev)
    ti, tt, tg = (torch.from_numpy(a).to(dev) for a in (ids, t, g))
    emb = flce.ScaledEmbedding(w.clone(), scale, padding_idx=int(ids[0]))
    head = flce.LinearLogProbs(emb.weight)
    x = emb(ti)
    h = x + torch.tanh(x)
    logp, ent = head(h, tt)
    (logp @ tg + 0.1 * ent.sum()).backward()

    u = torch.from_numpy(W).requires_grad_(True)
    look = u[torch.from_numpy(ids).long()]
    y = scale * torch.where(torch.from_numpy(ids)[:, None] == int(ids[0]), look.detach(), look)
    q = torch.log_softmax((y + torch.tanh(y)) @ u.T, 1)
    keep = torch.from_numpy(t != -100)
    at = torch.from_numpy(np.where(t < 0, 0, t)).long()[:, None]
    ((q.gather(1, at)[:, 0] * keep) @ torch.from_numpy(g).double()
     + 0.1 * (-(q.exp() * q).sum(1) * keep).sum()).backward()
    # h, dz, grad_hidden, its product with 1 + sech^2, and the two outputs are each rounded to bf16 (2^-8); a
    # rounded h moves the log probabilities themselves, whose gradient follows: a factor of four covers both
    ref = u.grad.numpy()
    assert np.linalg.norm(np64(emb.weight.grad) - ref) <= 4 * 2.0 ** -8 * np.linalg.norm(ref)

    # the same through the calls, into one fp32 gradient
    xe = flce.embedding_fwd(w, ti, scale)
    xr = xe.clone().requires_grad_(True)
    hh = xr + torch.tanh(xr)
    hc = hh.detach()
    o = flce.token_logprobs(hc, w, tt)
    d = flce.token_logprobs_bwd(hc, w, tt, o["lse"], o["entropy"], tg, torch.full((N,), 0.1, device=dev))
    hh.backward(d["grad_hidden"])
    one = d["grad_weight"].clone()
    flce.embedding_bwd(xr.grad, ti, V, scale, int(ids[0]), accumulate=True, out=d)
    ref2 = logprobs_grad_oracle(np64(hc), W, t, g, np.full(N, 0.1))
    assert np.linalg.norm(np64(one) - ref2["grad_weight"]) <= 2.0 ** -8 * np.linalg.norm(ref2["grad_weight"])
    e, mag = embedding_grad_oracle(np64(xr.grad), ids, V, scale, int(ids[0]))
    err = np.abs(np64(d["grad_weight"]) - (np64(one) + e))
    assert np.all(err <= (N + 3) * 2.0 ** -24 * (mag + np.abs(np64(one))))
    assert np.all(np.abs(np64(o["logp"]) - logprobs_oracle(np64(hc), W, t)["logp"]) <= 1e-4)


@pytest.mark.parametrize("N,H,V", [(1, 8, 1), (50, 64, 30), (3000, 520, 1000), (20000, 64, 5000)])
def test_nothing_is_read_behind_padding(env, N, H, V):  # noqa: F811
    """NaN in the gradients of padding tokens and a workspace full of NaN change no bit."""
    flce, torch, dev = env
    ids = torch.from_numpy(draw_ids(N, V, "uniform", 4)).to(dev)
    g = torch.randn(N, H, device=dev).to(torch.bfloat16)
    a = flce.embedding_bwd(g, ids, V, 2.0, 0)
    g[ids == 0] = float("nan")
    b = flce.embedding_bwd(g, ids, V, 2.0, 0, workspace=torch.full_like(a["workspace"], 255))
    assert torch.isfinite(a["grad_weight"]).all() and torch.equal(a["grad_weight"], b["grad_weight"])
    assert not a["grad_weight"][0].any()
