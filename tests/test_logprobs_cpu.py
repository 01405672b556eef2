"""Refusals and workspace sizes of the token log probabilities (no GPU)."""
import ctypes

import pytest

vp = ctypes.c_void_p
GOOD = vp(1 << 20)


@pytest.fixture(scope="module")
def flce():
    from linear_cross_entropy_ce_gb300 import flce
    try:
        flce.library()
    except RuntimeError:
        import __graft_entry__
        __graft_entry__.build()
    return flce


def fwd(lib, **kw):
    a = dict(h=GOOD, w=GOOD, t=GOOD, N=16, H=64, V=32, ii=-100, T=1.0, K=4, lp=GOOD, ent=GOOD, lse=GOOD, ids=GOOD,
             tl=GOOD, ws=GOOD, wsb=1 << 20)
    a.update(kw)
    return lib.flce_logprobs(*a.values(), None)


def bwd(lib, **kw):
    a = dict(h=GOOD, w=GOOD, t=GOOD, N=16, H=64, V=32, ii=-100, fl=0, T=1.0, lse=GOOD, ent=GOOD, gl=GOOD, ge=GOOD,
             gh=GOOD, gw=GOOD, ws=GOOD, wsb=1 << 20)
    a.update(kw)
    return lib.flce_logprobs_bwd(*a.values(), None)


NAN = float("nan")
INF = float("inf")


@pytest.mark.parametrize("kw,want", [
    (dict(h=None), 1), (dict(w=None), 1), (dict(t=None), 1), (dict(lp=None), 1), (dict(lse=None), 1),
    (dict(ws=None), 1), (dict(ids=None), 1), (dict(tl=None), 1), (dict(N=0), 1), (dict(V=0), 1), (dict(H=0), 1),
    (dict(T=0.0), 1), (dict(T=-1.0), 1), (dict(T=NAN), 1), (dict(T=INF), 1), (dict(T=1e-45), 1), (dict(K=-1), 1),
    (dict(K=33, V=32), 1), (dict(K=33, V=64), 2), (dict(H=60), 2), (dict(N=1 << 31), 2), (dict(V=1 << 31), 2),
    (dict(h=vp((1 << 20) + 8)), 2), (dict(w=vp((1 << 20) + 2)), 2), (dict(lp=vp((1 << 20) + 1)), 2),
    (dict(ent=vp((1 << 20) + 2)), 2), (dict(ids=vp((1 << 20) + 2)), 2)])
def test_forward_refusals(flce, kw, want):
    assert fwd(flce.library(), **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(h=None), 1), (dict(lse=None), 1), (dict(gl=None, ge=None), 1), (dict(ent=None), 1),
    (dict(gh=None, gw=None), 1), (dict(fl=1), 1), (dict(fl=4), 1), (dict(gw=None, fl=2), 1), (dict(T=0.0), 1),
    (dict(T=NAN), 1), (dict(N=0), 1), (dict(H=60), 2), (dict(gh=vp((1 << 20) + 8)), 2),
    (dict(gl=vp((1 << 20) + 2)), 2), (dict(ge=vp((1 << 20) + 2)), 2), (dict(lse=vp((1 << 20) + 2)), 2)])
def test_backward_refusals(flce, kw, want):
    assert bwd(flce.library(), **kw) == want


def test_workspace_sizes(flce):
    lib = flce.library()
    N, H, V = 16384, 4096, 128256
    assert 0 < lib.flce_logprobs_workspace_bytes(N, H, V, 0) <= 512 << 20
    assert 0 < lib.flce_logprobs_workspace_bytes(8 * N, H, V, 0) <= 0.05 * 8 * N * V * 2
    assert 0 < lib.flce_logprobs_workspace_bytes(64, H, V, 8) <= 256 << 20
    assert 0 < lib.flce_logprobs_workspace_bytes(N, H, V, 8) <= 2 << 30
    assert 0 < lib.flce_logprobs_bwd_workspace_bytes(N, H, V, 0) <= 2 << 30
    assert 0 < lib.flce_logprobs_bwd_workspace_bytes(16 * N, H, V, 0) <= 0.05 * 16 * N * V * 2
    assert lib.flce_logprobs_bwd_workspace_bytes(N, H, V, 2) > V * H * 4   # the accumulator of several chunks
    assert lib.flce_logprobs_bwd_workspace_bytes(4096, H, V, 2) < 2 << 30  # one chunk: none
    for bad in [(0, H, V, 0), (N, 63, V, 0), (N, H, V, 33), (N, H, 4, 5), (N, H, V, -1)]:
        assert lib.flce_logprobs_workspace_bytes(*bad) == 0
    assert lib.flce_logprobs_bwd_workspace_bytes(N, H, V, 1) == 0


def test_python_refusals(flce):
    torch = pytest.importorskip("torch")
    h, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(32, 64, dtype=torch.bfloat16)
    t = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        flce.token_logprobs(h, w, t)   # not CUDA tensors
    with pytest.raises(ValueError):
        flce.token_logprobs_bwd(h, w, t, torch.zeros(4), None, torch.zeros(4))


def test_capture_beside_a_living_graph(flce, monkeypatch):
    """The marks on a leaf's accumulator live as long as the graphs that use it, and only the default stream's refuse."""
    torch = pytest.importorskip("torch")
    now = {"stream": 0, "capturing": False}
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: now["stream"], raising=False)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: now["capturing"])

    class Double(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x):
            flce._mark_leaves(ctx, torch.device("cuda", 0))
            return 2 * x

        @staticmethod
        def backward(ctx, g):
            flce._check_capture(ctx)
            return 2 * g

    def step(stream, capturing):
        now.update(stream=stream, capturing=capturing)
        y = Double.apply(leaf)
        return y, lambda: torch.autograd.grad(y.sum(), leaf)[0]

    for eager_stream, refused in ((0, True), (7, False)):
        leaf = torch.ones(3, requires_grad=True)
        eager = step(eager_stream, False)
        eager[1]()
        captured = step(9, True)
        if refused:
            with pytest.raises(RuntimeError, match="alive"):
                captured[1]()
        else:
            assert captured[1]().tolist() == [2, 2, 2]
        del eager, captured
        assert step(9, True)[1]().tolist() == [2, 2, 2]
    assert Double.apply(2 * leaf).sum().item() == 12   # not a leaf: nothing to mark
