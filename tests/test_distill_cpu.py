"""Refusals and workspace sizes of the distillation loss (no GPU)."""
import ctypes

import pytest

vp = ctypes.c_void_p
GOOD = vp(1 << 20)
NAN, INF = float("nan"), float("inf")


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
    a = dict(h=GOOD, w=GOOD, ids=GOOD, tl=GOOD, N=16, H=64, V=32, K=4, T=1.0, tail=1, kl=GOOD, lse=GOOD, rest=GOOD,
             slp=GOOD, ws=GOOD, wsb=1 << 20)
    a.update(kw)
    return lib.flce_topk_distill(*a.values(), None)


def bwd(lib, **kw):
    a = dict(h=GOOD, w=GOOD, ids=GOOD, tl=GOOD, N=16, H=64, V=32, K=4, fl=0, T=1.0, tail=1, lse=GOOD, rest=GOOD, slp=GOOD,
             g=GOOD, gh=GOOD, gw=GOOD, ws=GOOD, wsb=1 << 20)
    a.update(kw)
    return lib.flce_topk_distill_bwd(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(h=None), 1), (dict(w=None), 1), (dict(ids=None), 1), (dict(tl=None), 1), (dict(kl=None), 1), (dict(lse=None), 1),
    (dict(rest=None), 1), (dict(slp=None), 1), (dict(ws=None), 1), (dict(N=0), 1), (dict(V=0), 1), (dict(H=0), 1),
    (dict(K=0), 1), (dict(K=257), 2), (dict(tail=2), 1), (dict(tail=-1), 1), (dict(T=0.0), 1), (dict(T=-1.0), 1),
    (dict(T=NAN), 1), (dict(T=INF), 1), (dict(T=1e-45), 1), (dict(H=60), 2), (dict(N=1 << 31), 2), (dict(V=1 << 31), 2),
    (dict(h=vp((1 << 20) + 8)), 2), (dict(w=vp((1 << 20) + 2)), 2), (dict(kl=vp((1 << 20) + 1)), 2),
    (dict(tl=vp((1 << 20) + 2)), 2), (dict(N=200, ws=vp((1 << 20) + 16)), 2)])
def test_forward_refusals(flce, kw, want):
    assert fwd(flce.library(), **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(h=None), 1), (dict(ids=None), 1), (dict(tl=None), 1), (dict(lse=None), 1), (dict(rest=None), 1),
    (dict(slp=None), 1), (dict(g=None), 1), (dict(gh=None, gw=None), 1), (dict(fl=1), 1), (dict(fl=4), 1),
    (dict(gw=None, fl=2), 1), (dict(T=0.0), 1), (dict(T=NAN), 1), (dict(N=0), 1), (dict(K=0), 1), (dict(K=300), 2),
    (dict(tail=7), 1), (dict(H=60), 2), (dict(gh=vp((1 << 20) + 8)), 2), (dict(g=vp((1 << 20) + 2)), 2),
    (dict(slp=vp((1 << 20) + 2)), 2), (dict(ws=vp((1 << 20) + 16)), 2), (dict(wsb=300), 3), (dict(wsb=0), 3)])
def test_backward_refusals(flce, kw, want):
    assert bwd(flce.library(), **kw) == want


def test_workspace_sizes(flce):
    lib = flce.library()
    N, H, V = 16384, 4096, 128256
    assert 0 < lib.flce_topk_distill_workspace_bytes(N, H, V, 32) <= 512 << 20
    assert 0 < lib.flce_topk_distill_workspace_bytes(8 * N, H, V, 64) <= 0.05 * 8 * N * V * 2
    assert 0 < lib.flce_topk_distill_workspace_bytes(64, H, V, 64) <= 2 << 20
    own = lib.flce_logprobs_bwd_workspace_bytes(N, H, V, 0)
    assert own < lib.flce_topk_distill_bwd_workspace_bytes(N, H, V, 32, 0) <= own + N * (12 + 64) + 2048
    for bad in [(0, H, V, 4), (N, 63, V, 4), (N, H, V, 0), (N, H, V, 257)]:
        assert lib.flce_topk_distill_workspace_bytes(*bad) == 0
        assert lib.flce_topk_distill_bwd_workspace_bytes(*bad, 0) == 0
    assert lib.flce_topk_distill_bwd_workspace_bytes(N, H, V, 4, 1) == 0


def test_python_refusals(flce):
    torch = pytest.importorskip("torch")
    h, w = torch.zeros((4, 64), dtype=torch.bfloat16), torch.zeros((40, 64), dtype=torch.bfloat16)
    ids, t = torch.zeros((4, 3), dtype=torch.int32), torch.zeros((4, 3))
    with pytest.raises(ValueError, match="CUDA"):
        flce.topk_distill(h, w, ids, t)
    with pytest.raises(ValueError, match="CUDA"):
        flce.topk_distill_bwd(h, w, ids, t, t[:, 0], t[:, 0], t, t[:, 0])
    check = lambda i, l, n=4: flce._check_teacher(i, l, n, ids.device)  # noqa: E731
    assert check(ids, t) == 3
    for args, err in [((ids.long(), t), TypeError), ((ids, t.double()), TypeError), ((ids, t[:, :2]), ValueError),
                      ((ids, t, 5), ValueError), ((ids[:, :0], t[:, :0]), ValueError), ((ids[0], t[0]), ValueError),
                      ((ids.expand(4, 3).t().contiguous().t(), t), ValueError),
                      ((torch.zeros((4, 257), dtype=torch.int32), torch.zeros((4, 257))), ValueError)]:
        with pytest.raises(err):
            check(*args)
