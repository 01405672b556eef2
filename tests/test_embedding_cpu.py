"""Refusals and workspace sizes of the scaled embedding and its gradient (no GPU)."""
import ctypes

import pytest

from tests.test_logprobs_cpu import flce  # noqa: F401 (fixture)

vp = ctypes.c_void_p
GOOD = vp(1 << 20)


def fwd(lib, **kw):
    a = dict(w=GOOD, ids=GOOD, N=16, H=64, V=32, dt=0, scale=2.0, out=GOOD)
    a.update(kw)
    return lib.flce_embedding(*a.values(), None)


def bwd(lib, **kw):
    a = dict(g=GOOD, ids=GOOD, N=16, H=64, V=32, dt=0, scale=2.0, pad=-1, fl=0, gw=GOOD, gdt=2, ws=GOOD, wsb=1 << 20)
    a.update(kw)
    return lib.flce_embedding_bwd(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(w=None), 1), (dict(ids=None), 1), (dict(out=None), 1), (dict(N=0), 1), (dict(V=0), 1), (dict(dt=3), 1),
    (dict(dt=-1), 1), (dict(H=60), 2), (dict(w=vp((1 << 20) + 8)), 2), (dict(out=vp((1 << 20) + 4)), 2),
    (dict(ids=vp((1 << 20) + 2)), 2), (dict(N=1 << 31), 2)])
def test_lookup_refusals(flce, kw, want):  # noqa: F811
    assert fwd(flce.library(), **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(g=None), 1), (dict(ids=None), 1), (dict(gw=None), 1), (dict(ws=None), 1), (dict(N=0), 1), (dict(H=0), 1),
    (dict(dt=3), 1), (dict(gdt=3), 1), (dict(fl=1), 1), (dict(fl=4, gdt=0), 1), (dict(pad=32), 1), (dict(H=12), 2),
    (dict(N=(1 << 30) + 1), 2), (dict(gw=vp((1 << 20) + 8)), 2), (dict(g=vp((1 << 20) + 8)), 2)])
def test_gradient_refusals(flce, kw, want):  # noqa: F811
    assert bwd(flce.library(), **kw) == want


def test_workspace_sizes(flce):  # noqa: F811
    f = flce.library().flce_embedding_bwd_workspace_bytes
    assert f(0, 64, 32) == 0 and f(16, 63, 32) == 0 and f(1 << 31, 64, 32) == 0
    assert 0 < f(1, 8, 1) < f(100000, 512, 16000) <= 8 * 512 * 100000


def test_python_refusals_of_leaves(flce):  # noqa: F811
    """A table that is not on a GPU is named as such, whether or not a gradient is wanted."""
    torch = pytest.importorskip("torch")
    ids = torch.zeros(4, dtype=torch.int32)
    for grad in (False, True):
        table = torch.zeros(32, 64, dtype=torch.bfloat16, requires_grad=grad)
        with pytest.raises(ValueError, match="CUDA"):
            flce.embedding(ids, table)
        with pytest.raises(ValueError, match="CUDA"):
            flce.ScaledEmbedding(table)(ids)
        with pytest.raises(ValueError, match="CUDA"):
            flce.linear_logprobs(table[:4], table, ids)
