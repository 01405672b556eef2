"""Histories whose lists take longer to make than a pipeline may wait: the call is as good as any other.

The limit of the waits is lowered by the environment variable that a process reads once, so the calls are a child's."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

CHILD = """
import torch
from linear_cross_entropy_ce_gb300 import flce
dev = torch.device("cuda:0")
gen = torch.Generator(device=dev).manual_seed(0)
V, H, N, L = 600000, 64, 2, 1 << 23        # three windows of the streaming form's bitmap
w = (torch.randn((V, H), generator=gen, device=dev) / 8).to(torch.bfloat16)
h = torch.randn((N, H), generator=gen, device=dev).to(torch.bfloat16)
short = torch.randint(0, V, (N, 64), generator=gen, device=dev, dtype=torch.int32)
one = torch.full((N,), 1.5, device=dev)
want = flce.constrained_logprobs(h, w, history=short, repetition_penalty=one, top_k=4)
assert flce.query_status(want["workspace"]) == flce.FLCE_OK
for spread in (False, True):               # the same few tokens over and over, and padding between them
    long = torch.full((N, L), -1, dtype=torch.int32, device=dev) if spread else short.repeat(1, L // 64)
    long[:, :64] = short
    o = flce.constrained_logprobs(h, w, history=long, repetition_penalty=one, top_k=4)
    assert flce.query_status(o["workspace"]) == flce.FLCE_OK, "timed out"
    for k in ("lse", "entropy", "top_ids", "top_logp"):
        assert torch.equal(o[k], want[k]), k
print("right")
"""


def test_longer_than_a_wait():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    # 3 ms: the lists of 2^23 ids take longer, the weight of 77 MB streams in 20 us
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=root, capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, FLCE_WAIT_TIMEOUT_NS="3000000", PYTHONPATH=root))
    assert r.returncode == 0 and r.stdout.strip().endswith("right"), r.stdout + r.stderr
