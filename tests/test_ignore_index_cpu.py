"""An ignore index of more than 32 bits is refused by every call that takes one (no GPU: the library is stood in for)."""
import pytest

torch = pytest.importorskip("torch")

from linear_cross_entropy_ce_gb300 import flce  # noqa: E402

N, H, V = 4, 64, 32


class Reached(Exception):
    pass


class Library:
    """Sizes for every workspace; any other call is one too far."""

    def __getattr__(self, name):
        def call(*a):
            if name.endswith("_bytes"):
                return 1 << 20
            raise Reached(name)
        return call


@pytest.fixture
def calls(monkeypatch):
    class On:
        def __init__(self, device, stream):
            pass

        def __enter__(self):
            return 0

        def __exit__(self, *exc):
            pass

    monkeypatch.setattr(flce, "library", Library)
    monkeypatch.setattr(flce, "_check_inputs", lambda h, w, t: (N, H, V))
    monkeypatch.setattr(flce, "_on", On)
    monkeypatch.setattr(flce, "_stream", lambda s: 0)
    h, w = torch.zeros(N, H, dtype=torch.bfloat16), torch.zeros(V, H, dtype=torch.bfloat16)
    t, row = torch.zeros(N, dtype=torch.int32), torch.zeros(N)
    return {"token_logprobs": lambda i: flce.token_logprobs(h, w, t, i),
            "token_logprobs_bwd": lambda i: flce.token_logprobs_bwd(h, w, t, row, None, row, None, i),
            "linear_logprobs": lambda i: flce.linear_logprobs(h, w, t, i),
            "fwd_bwd": lambda i: flce.fwd_bwd(h, w, t, i), "loss": lambda i: flce.loss(h, w, t, i),
            "linear_cross_entropy": lambda i: flce.linear_cross_entropy(h, w, t, i),
            "vocab_shard_stats": lambda i: flce.vocab_shard_stats(h, w, t, 0, V, i),
            "vocab_shard_bwd": lambda i: flce.vocab_shard_bwd(h, w, t, row, 0, V, i),
            "vocab_finish": lambda i: flce.vocab_finish(row, row, row, t, i)}


NAMES = ["token_logprobs", "token_logprobs_bwd", "linear_logprobs", "fwd_bwd", "loss", "linear_cross_entropy",
         "vocab_shard_stats", "vocab_shard_bwd", "vocab_finish"]


@pytest.mark.parametrize("name", NAMES)
def test_more_than_32_bits(calls, name):
    for i in (2 ** 31, -2 ** 31 - 1, 2 ** 32, 2 ** 40 - 100):
        with pytest.raises(ValueError, match="32 bits"):
            calls[name](i)
    for i in (-100, 0, 2 ** 31 - 1, -2 ** 31):
        with pytest.raises(Reached):
            calls[name](i)
