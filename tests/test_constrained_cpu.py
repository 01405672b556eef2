"""Refusals and workspace sizes of the constrained log probabilities (no GPU)."""
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


def call(flce, rules=None, **kw):
    c = flce._Constraints()
    for k, v in dict(dict(history=1 << 20, history_len=9, history_stride=9), **(rules or {})).items():
        setattr(c, k, v)
    a = dict(h=GOOD, w=GOOD, t=GOOD, N=16, H=64, V=32, ii=-100, T=1.0, K=4, c=ctypes.byref(c), lp=GOOD, ent=GOOD,
             lse=GOOD, ids=GOOD, tl=GOOD, ws=GOOD, wsb=1 << 20)
    a.update(kw)
    return flce.library().flce_constrained_logprobs(*a.values(), None)


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("kw,want", [
    (dict(h=None), 1), (dict(w=None), 1), (dict(lp=None), 1), (dict(lse=None), 1), (dict(ws=None), 1), (dict(c=None), 1),
    (dict(ids=None), 1), (dict(tl=None), 1), (dict(N=0), 1), (dict(V=0), 1), (dict(H=0), 1), (dict(T=0.0), 1),
    (dict(T=-1.0), 1), (dict(T=NAN), 1), (dict(T=INF), 1), (dict(K=-1), 1), (dict(K=33, V=32), 1), (dict(K=33, V=64), 2),
    (dict(H=60), 2), (dict(N=1 << 31), 2), (dict(V=1 << 31), 2), (dict(h=vp((1 << 20) + 8)), 2),
    (dict(lse=vp((1 << 20) + 1)), 2), (dict(N=200, ws=vp((1 << 20) + 16)), 2)])
def test_refusals(flce, kw, want):
    assert call(flce, **kw) == want


@pytest.mark.parametrize("rules,want", [
    (dict(history=None), 1), (dict(history_len=-1), 1), (dict(history_stride=-1), 1), (dict(n_bias=-1), 1),
    (dict(n_bias=3), 1), (dict(n_bias=3, bias_ids=1 << 20), 1), (dict(mask_stride=-2), 1), (dict(bias_stride=-2), 1),
    (dict(bias_ids_stride=-2), 1), (dict(history_len=1 << 31), 2), (dict(history_len=(1 << 30) + 1), 2),
    (dict(n_bias=(1 << 20) + 1, bias_ids=1 << 20, bias=1 << 20), 2), (dict(history=(1 << 20) + 2), 2),
    (dict(mask=(1 << 20) + 1), 2), (dict(repetition_penalty=(1 << 20) + 2), 2), (dict(prompt_lens=(1 << 20) + 3), 2),
    (dict(bias=(1 << 20) + 3, bias_ids=1 << 20, n_bias=2), 2)])
def test_refused_rules(flce, rules, want):
    assert call(flce, rules) == want


def test_targets_may_be_absent(flce):
    # past every check of arguments: no device here
    assert call(flce, t=None, lp=None) == flce.FLCE_ECUDA


def test_workspace_sizes(flce):
    lib = flce.library()
    N, H, V = 2048, 4096, 128256
    plain = lib.flce_logprobs_workspace_bytes(64, H, V, 8)
    assert plain < lib.flce_constrained_workspace_bytes(64, H, V, 8, 1000, 0) <= plain + 64 * (8000 + 4 * 700) + 4096
    assert lib.flce_constrained_workspace_bytes(64, H, V, 8, 10 ** 6, 0) <= plain + 64 * (8 * V + 4 * 700) + 4096
    assert 0 < lib.flce_constrained_workspace_bytes(N, H, V, 0, 4000, 16) <= 512 << 20
    assert 0 < lib.flce_constrained_workspace_bytes(N, H, V, 8, 4000, 16) <= 2 << 30
    for bad in [(0, H, V, 0, 0, 0), (N, 63, V, 0, 0, 0), (N, H, V, 33, 0, 0), (N, H, 4, 5, 0, 0), (N, H, V, -1, 0, 0),
                (N, H, V, 0, -1, 0), (N, H, V, 0, 0, -1), (N, H, V, 0, 1 << 31, 0), (N, H, V, 0, (1 << 30) + 1, 0), (N, H, V, 0, 0, (1 << 20) + 1)]:
        assert lib.flce_constrained_workspace_bytes(*bad) == 0


def test_python_refusals(flce):
    torch = pytest.importorskip("torch")
    h, w = torch.zeros((4, 64), dtype=torch.bfloat16), torch.zeros((40, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        flce.constrained_logprobs(h, w)
    for t, err in [(torch.zeros((4, 3)), TypeError), (torch.zeros((3, 3), dtype=torch.int32), ValueError),
                   (torch.zeros(4, dtype=torch.int32), ValueError),
                   (torch.zeros((4, 6), dtype=torch.int32)[:, ::2], ValueError)]:
        with pytest.raises(err):
            flce._rows_of(t, "history", torch.int32, 4, torch.device("cpu"))
    rows = torch.zeros((1, 5), dtype=torch.int32).expand(4, -1)
    assert flce._rows_of(rows, "history", torch.int32, 4, rows.device) == 0
    assert flce._rows_of(torch.zeros((4, 9), dtype=torch.int32)[:, 2:7], "history", torch.int32, 4, rows.device) == 9
    with pytest.raises(ValueError):
        flce._row_values(torch.zeros(3), "repetition_penalty", torch.float32, 4, rows.device)
    assert flce._row_values(None, "repetition_penalty", torch.float32, 4, rows.device) is None
