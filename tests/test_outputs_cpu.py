"""The caller's output dict (no GPU): what a call does not produce is left in it."""
import pytest

torch = pytest.importorskip("torch")

from linear_cross_entropy_ce_gb300 import flce  # noqa: E402

CPU = torch.device("cpu")
ROW = ((4,), torch.float32)


def test_entries_not_asked_for_stay():
    mine = torch.zeros(4, 2, dtype=torch.int32)
    given = torch.zeros(4)
    out = {"logp": given, "top_ids": mine, "other": 3}
    o, made = flce._outputs(out, {"logp": ROW, "lse": ROW, "entropy": None, "top_ids": None}, CPU)
    assert o is out and o["top_ids"] is mine and o["other"] == 3
    assert made["top_ids"] is None and made["entropy"] is None and o["entropy"] is None
    assert made["logp"] is given and o["logp"] is given
    assert made["lse"] is o["lse"] and tuple(o["lse"].shape) == (4,)


def test_entries_of_none_are_made():
    o, made = flce._outputs({"lse": None}, {"lse": ROW}, CPU)
    assert o["lse"] is made["lse"] and made["lse"] is not None


def test_wrong_buffers_are_refused_before_any_is_made():
    out = {"lse": torch.zeros(5)}
    with pytest.raises(ValueError):
        flce._outputs(out, {"logp": ROW, "lse": ROW}, CPU)
    assert list(out) == ["lse"]
