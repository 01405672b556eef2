"""Workspaces that are 16- but not 32-byte aligned (no GPU: a call that took one would fault there).

The logits and their gradient are kept in the workspace by 32-byte stores, at
offsets that are multiples of 256, so those calls refuse such a workspace on
the host.  Calls that keep neither take it; without a GPU they get as far as
asking for the device."""
import ctypes

import pytest

from tests.test_embedding_cpu import bwd as embedding_bwd
from tests.test_logprobs_cpu import bwd, flce, fwd  # noqa: F401 (fixture)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses here are no device memory")

vp = ctypes.c_void_p
GOOD = vp(1 << 20)
SIZES = dict(N=200, H=64, V=32)
UNSUPPORTED = 2
BIG = 1 << 24


def loss_bwd(lib, ws):
    return lib.flce_fwd_bwd(GOOD, GOOD, GOOD, 16, 64, 32, -100, 0, GOOD, GOOD, None, GOOD, GOOD, ws, BIG, None)


def rmsnorm(lib, ws):
    return lib.flce_rmsnorm_fwd_bwd(GOOD, GOOD, 1e-6, GOOD, GOOD, 16, 64, 32, -100, 0, GOOD, GOOD, None, GOOD, GOOD, GOOD,
                                    ws, BIG, None)


def shard_bwd(lib, ws):
    return lib.flce_vocab_shard_bwd(GOOD, GOOD, GOOD, 16, 64, 32, 0, 64, -100, 0, GOOD, GOOD, GOOD, ws, BIG, None)


KEEP_LOGITS = {
    "logprobs with alternatives": lambda lib, ws: fwd(lib, ws=ws, wsb=BIG, **SIZES),
    "logprobs gradient": lambda lib, ws: bwd(lib, ws=ws, wsb=BIG, **SIZES),
    "logprobs gradient of few tokens": lambda lib, ws: bwd(lib, ws=ws, wsb=BIG, N=1),
    "loss and gradients": loss_bwd, "with the final norm": rmsnorm, "vocabulary shard": shard_bwd}

KEEP_NONE = {
    "logprobs": lambda lib, ws: fwd(lib, ws=ws, wsb=BIG, K=0, **SIZES),
    "logprobs of few tokens": lambda lib, ws: fwd(lib, ws=ws, wsb=BIG, N=128),
    "loss": lambda lib, ws: lib.flce_loss(GOOD, GOOD, GOOD, 16, 64, 32, -100, 0, GOOD, GOOD, None, ws, BIG, None),
    "embedding gradient": lambda lib, ws: embedding_bwd(lib, ws=ws, wsb=BIG)}


@pytest.mark.parametrize("call", sorted(KEEP_LOGITS))
@pytest.mark.parametrize("offset", [16, 48, 8, 4])
def test_refused_where_logits_are_kept(flce, call, offset):  # noqa: F811
    assert KEEP_LOGITS[call](flce.library(), vp((1 << 20) + offset)) == UNSUPPORTED


@pytest.mark.parametrize("call", sorted(KEEP_NONE))
def test_taken_elsewhere(flce, call):  # noqa: F811
    lib = flce.library()
    aligned = KEEP_NONE[call](lib, GOOD)   # the status without a device
    assert aligned != UNSUPPORTED and KEEP_NONE[call](lib, vp((1 << 20) + 16)) == aligned
    assert KEEP_NONE[call](lib, vp((1 << 20) + 8)) == UNSUPPORTED
