"""The distillation's workspace holds what its kernels write, and no more (no GPU)."""
import pytest


@pytest.fixture(scope="module")
def flce():
    from linear_cross_entropy_ce_gb300 import flce
    try:
        flce.library()
    except RuntimeError:
        import __graft_entry__
        __graft_entry__.build()
    return flce


@pytest.mark.parametrize("N,H,V,K", [(300, 2048, 256007, 1), (300, 64, 512, 8), (1000, 512, 16000, 100)])
def test_one_chunk(flce, N, H, V, K):
    C, parts = (N + 127) // 128 * 128, (V + 127) // 128
    # a row: its hidden state, its target, two values and a table entry a part, its entries (id, mass, place), their
    # number, and the parts that hold any
    row = 2 * H + 4 + 8 * parts + 2 * (parts + 1) + 10 * K + 4 + 512 * min(K, parts)
    got = flce.library().flce_topk_distill_workspace_bytes(N, H, V, K)
    assert C * row < got <= C * row + 8 * N + 16 * 256
