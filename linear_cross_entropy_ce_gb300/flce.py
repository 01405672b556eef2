"""ctypes binding of libflce (argument marshalling only).

Every step of the fused linear cross-entropy runs in the CUDA kernels of
``libflce.so``; this module only checks tensor types, allocates outputs and
the workspace through PyTorch's caching allocator, and passes raw device
pointers and the current CUDA stream to the C ABI declared in
``include/flce.h``.  There is no fallback: if the library is missing or the
call fails, an exception is raised.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from typing import Optional

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_lib", "libflce.so")

FLCE_OK, FLCE_EINVAL, FLCE_EUNSUPPORTED, FLCE_EWORKSPACE, FLCE_EBADTARGET, FLCE_ETIMEOUT, FLCE_ECUDA = range(7)
STATUS_NAMES = {0: "FLCE_OK", 1: "FLCE_EINVAL", 2: "FLCE_EUNSUPPORTED", 3: "FLCE_EWORKSPACE",
                4: "FLCE_EBADTARGET", 5: "FLCE_ETIMEOUT", 6: "FLCE_ECUDA"}
REDUCE = {"mean": 0, "sum": 1}
FLCE_GW_BF16 = 0x2

_lib = None


class FlceError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        name = STATUS_NAMES.get(status, str(status))
        super().__init__(f"{what}: {name} ({_status_string(status)})" if what else name)


class PlanInfo(ctypes.Structure):
    _fields_ = [("chunk_rows", ctypes.c_int64), ("max_chunks", ctypes.c_int64),
                ("logits_row_stride", ctypes.c_int64), ("gemm_launches_per_chunk", ctypes.c_int32),
                ("dx_splits", ctypes.c_int32),
                ("vocab_tiles", ctypes.c_int32), ("workspace_bytes", ctypes.c_size_t)]


class _Constraints(ctypes.Structure):
    _fields_ = [("history", ctypes.c_void_p), ("history_len", ctypes.c_int64), ("history_stride", ctypes.c_int64),
                ("history_lens", ctypes.c_void_p), ("prompt_lens", ctypes.c_void_p),
                ("repetition_penalty", ctypes.c_void_p), ("frequency_penalty", ctypes.c_void_p),
                ("presence_penalty", ctypes.c_void_p), ("bias_ids", ctypes.c_void_p), ("bias", ctypes.c_void_p),
                ("n_bias", ctypes.c_int64), ("bias_ids_stride", ctypes.c_int64), ("bias_stride", ctypes.c_int64),
                ("mask", ctypes.c_void_p), ("mask_stride", ctypes.c_int64)]


def library() -> ctypes.CDLL:
    """Load libflce.so (built in-tree by ``linear_cross_entropy_ce_gb300.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError(f"{_LIB_PATH} is missing: build it with linear_cross_entropy_ce_gb300.build.build()")
    lib = ctypes.CDLL(_LIB_PATH)
    i64, u32, i32, sz, vp = ctypes.c_int64, ctypes.c_uint32, ctypes.c_int32, ctypes.c_size_t, ctypes.c_void_p
    lib.flce_workspace_bytes.argtypes = [i64, i64, i64, u32]
    lib.flce_workspace_bytes.restype = sz
    lib.flce_loss_workspace_bytes.argtypes = [i64, i64, i64, u32]
    lib.flce_loss_workspace_bytes.restype = sz
    lib.flce_workspace_bytes_for_chunk.argtypes = [i64, i64, i64, u32, i64]
    lib.flce_workspace_bytes_for_chunk.restype = sz
    lib.flce_plan.argtypes = [i64, i64, i64, u32, ctypes.c_int, sz, ctypes.POINTER(PlanInfo)]
    lib.flce_plan.restype = ctypes.c_int
    lib.flce_fwd_bwd.argtypes = [vp, vp, vp, i64, i64, i64, i32, u32, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.flce_fwd_bwd.restype = ctypes.c_int
    lib.flce_loss.argtypes = [vp, vp, vp, i64, i64, i64, i32, u32, vp, vp, vp, vp, sz, vp]
    lib.flce_loss.restype = ctypes.c_int
    lib.flce_query_status.argtypes = [vp, vp]
    lib.flce_query_status.restype = ctypes.c_int
    lib.flce_selftest_timeout.argtypes = [vp, ctypes.c_uint64, vp]
    lib.flce_selftest_timeout.restype = ctypes.c_int
    lib.flce_query_stall.argtypes = [vp, ctypes.POINTER(ctypes.c_int32), vp]
    lib.flce_query_stall.restype = ctypes.c_int
    lib.flce_debug_arm_stall.argtypes = [ctypes.c_uint64]
    lib.flce_debug_arm_stall.restype = ctypes.c_int
    lib.flce_debug_arm_stall_after.argtypes = [ctypes.c_uint64, i32]
    lib.flce_debug_arm_stall_after.restype = ctypes.c_int
    lib.flce_status_string.argtypes = [ctypes.c_int]
    lib.flce_status_string.restype = ctypes.c_char_p
    lib.flce_rmsnorm_workspace_bytes.argtypes = [i64, i64, i64, u32]
    lib.flce_rmsnorm_workspace_bytes.restype = sz
    lib.flce_rmsnorm_fwd_bwd.argtypes = [vp, vp, ctypes.c_float, vp, vp, i64, i64, i64, i32, u32, vp, vp, vp, vp, vp,
                                         vp, vp, sz, vp]
    lib.flce_rmsnorm_fwd_bwd.restype = ctypes.c_int
    lib.flce_vocab_shard_workspace_bytes.argtypes = [i64, i64, i64, u32]
    lib.flce_vocab_shard_workspace_bytes.restype = sz
    lib.flce_vocab_shard_stats.argtypes = [vp, vp, vp, i64, i64, i64, i64, i64, i32, vp, vp, vp, vp, vp, sz, vp]
    lib.flce_vocab_shard_stats.restype = ctypes.c_int
    lib.flce_vocab_rescale.argtypes = [vp, vp, vp, i64, vp]
    lib.flce_vocab_rescale.restype = ctypes.c_int
    lib.flce_vocab_finish.argtypes = [vp, vp, vp, vp, i64, i32, u32, vp, vp, vp, vp, vp]
    lib.flce_vocab_finish.restype = ctypes.c_int
    lib.flce_vocab_shard_bwd.argtypes = [vp, vp, vp, i64, i64, i64, i64, i64, i32, u32, vp, vp, vp, vp, sz, vp]
    lib.flce_vocab_shard_bwd.restype = ctypes.c_int
    f32 = ctypes.c_float
    lib.flce_logprobs_workspace_bytes.argtypes = [i64, i64, i64, i32]
    lib.flce_logprobs_workspace_bytes.restype = sz
    lib.flce_logprobs.argtypes = [vp, vp, vp, i64, i64, i64, i32, f32, i32, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.flce_logprobs.restype = ctypes.c_int
    lib.flce_logprobs_bwd_workspace_bytes.argtypes = [i64, i64, i64, u32]
    lib.flce_logprobs_bwd_workspace_bytes.restype = sz
    lib.flce_logprobs_bwd.argtypes = [vp, vp, vp, i64, i64, i64, i32, u32, f32, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.flce_logprobs_bwd.restype = ctypes.c_int
    lib.flce_constrained_workspace_bytes.argtypes = [i64, i64, i64, i32, i64, i64]
    lib.flce_constrained_workspace_bytes.restype = sz
    lib.flce_constrained_logprobs.argtypes = [vp, vp, vp, i64, i64, i64, i32, f32, i32, ctypes.POINTER(_Constraints),
                                              vp, vp, vp, vp, vp, vp, sz, vp]
    lib.flce_constrained_logprobs.restype = ctypes.c_int
    lib.flce_topk_distill_workspace_bytes.argtypes = [i64, i64, i64, i32]
    lib.flce_topk_distill_workspace_bytes.restype = sz
    lib.flce_topk_distill.argtypes = [vp, vp, vp, vp, i64, i64, i64, i32, f32, i32, vp, vp, vp, vp, vp, sz, vp]
    lib.flce_topk_distill.restype = ctypes.c_int
    lib.flce_topk_distill_bwd_workspace_bytes.argtypes = [i64, i64, i64, i32, u32]
    lib.flce_topk_distill_bwd_workspace_bytes.restype = sz
    lib.flce_topk_distill_bwd.argtypes = [vp, vp, vp, vp, i64, i64, i64, i32, u32, f32, i32, vp, vp, vp, vp, vp, vp, vp,
                                          sz, vp]
    lib.flce_topk_distill_bwd.restype = ctypes.c_int
    lib.flce_embedding.argtypes = [vp, vp, i64, i64, i64, i32, f32, vp, vp]
    lib.flce_embedding.restype = ctypes.c_int
    lib.flce_embedding_bwd_workspace_bytes.argtypes = [i64, i64, i64]
    lib.flce_embedding_bwd_workspace_bytes.restype = sz
    lib.flce_embedding_bwd.argtypes = [vp, vp, i64, i64, i64, i32, f32, i32, u32, vp, i32, vp, sz, vp]
    lib.flce_embedding_bwd.restype = ctypes.c_int
    lib.flce_scale_grads.argtypes = [vp, vp, i64, i64, i64, vp, vp]
    lib.flce_scale_grads.restype = ctypes.c_int
    lib.flce_profile_begin.argtypes = []
    lib.flce_profile_begin.restype = ctypes.c_int
    lib.flce_profile_end.argtypes = [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_int64),
                                     ctypes.POINTER(ctypes.c_int64)]
    lib.flce_profile_end.restype = ctypes.c_int
    lib.flce_version.argtypes = []
    lib.flce_version.restype = ctypes.c_char_p
    _lib = lib
    return lib


def _status_string(s: int) -> str:
    try:
        return library().flce_status_string(int(s)).decode()
    except Exception:  # pragma: no cover - library not loadable
        return "?"


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _check_inputs(hidden, weight, targets):
    if not (hidden.is_cuda and weight.is_cuda and targets.is_cuda):
        raise ValueError("hidden, weight and targets must be CUDA tensors")
    if hidden.dtype != torch.bfloat16 or weight.dtype != torch.bfloat16:
        raise TypeError("hidden and weight must be bfloat16")
    if targets.dtype != torch.int32:
        raise TypeError("targets must be int32")
    if hidden.dim() != 2 or weight.dim() != 2 or targets.dim() != 1:
        raise ValueError("expected hidden [N,H], weight [V,H], targets [N]")
    N, H = hidden.shape
    V, H2 = weight.shape
    if H2 != H or targets.shape[0] != N:
        raise ValueError("shape mismatch")
    for t in (hidden, weight, targets):
        if not t.is_contiguous():
            raise ValueError("inputs must be contiguous")
    return N, H, V


def _ignored(ignore_index) -> int:
    """The ignore index as the library takes it: what does not fit 32 bits would become some other token's id."""
    i = int(ignore_index)
    if not -2 ** 31 <= i < 2 ** 31:
        raise ValueError("ignore_index must fit in 32 bits, as the targets do")
    return i


def _flags(reduction: str, grad_weight_dtype=torch.float32) -> int:
    if grad_weight_dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("grad_weight_dtype must be torch.float32 or torch.bfloat16")
    return REDUCE[reduction] | (FLCE_GW_BF16 if grad_weight_dtype == torch.bfloat16 else 0)


def workspace_bytes(N: int, H: int, V: int, reduction: str = "mean", chunk_rows: Optional[int] = None,
                    forward_only: bool = False, grad_weight_dtype=torch.float32) -> int:
    """Workspace of the default plan (or of a given chunk size).  With a bf16
    grad_weight it includes the fp32 V x H accumulator of grad_weight."""
    lib = library()
    f = _flags(reduction, torch.float32 if forward_only else grad_weight_dtype)
    if forward_only:
        n = lib.flce_loss_workspace_bytes(N, H, V, f)
    elif chunk_rows is not None:
        n = lib.flce_workspace_bytes_for_chunk(N, H, V, f, chunk_rows)
    else:
        n = lib.flce_workspace_bytes(N, H, V, f)
    if n == 0:
        raise FlceError(FLCE_EINVAL, "workspace size")
    return int(n)


def plan(N: int, H: int, V: int, workspace_bytes: int, forward_only: bool = False,
         reduction: str = "mean", grad_weight_dtype=torch.float32) -> dict:
    info = PlanInfo()
    s = library().flce_plan(N, H, V, _flags(reduction, grad_weight_dtype), int(forward_only), workspace_bytes,
                            ctypes.byref(info))
    if s != FLCE_OK:
        raise FlceError(s, "flce_plan")
    return {k: getattr(info, k) for k, _ in PlanInfo._fields_}


def new_workspace(nbytes: int, device) -> torch.Tensor:
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def fwd_bwd(hidden: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor, ignore_index: int = -100,
            reduction: str = "mean", *, workspace: Optional[torch.Tensor] = None,
            chunk_rows: Optional[int] = None, row_loss: bool = False, out: Optional[dict] = None,
            stream=None, grad_weight_dtype=torch.float32) -> dict:
    """Loss, n_valid, grad_hidden (bf16 [N,H]) and grad_weight ([V,H], fp32 by
    default, or bf16 rounded once from the fp32 accumulation) in one call."""
    N, H, V = _check_inputs(hidden, weight, targets)
    dev = hidden.device
    flags = _flags(reduction, grad_weight_dtype)
    if workspace is None:
        workspace = new_workspace(workspace_bytes(N, H, V, reduction, chunk_rows,
                                                  grad_weight_dtype=grad_weight_dtype), dev)
    o = out if out is not None else {}
    if "loss" not in o:
        o["loss"] = torch.empty(1, dtype=torch.float32, device=dev)
        o["n_valid"] = torch.empty(1, dtype=torch.int32, device=dev)
        o["grad_hidden"] = torch.empty((N, H), dtype=torch.bfloat16, device=dev)
        o["grad_weight"] = torch.empty((V, H), dtype=grad_weight_dtype, device=dev)
        o["row_loss"] = torch.empty(N, dtype=torch.float32, device=dev) if row_loss else None
    if o["grad_weight"].dtype != grad_weight_dtype:
        raise TypeError("out['grad_weight'] does not have grad_weight_dtype")
    s = library().flce_fwd_bwd(_ptr(hidden), _ptr(weight), _ptr(targets), N, H, V, _ignored(ignore_index),
                               flags, _ptr(o["loss"]), _ptr(o["n_valid"]), _ptr(o.get("row_loss")),
                               _ptr(o["grad_hidden"]), _ptr(o["grad_weight"]), _ptr(workspace),
                               workspace.numel(), _stream(stream))
    if s != FLCE_OK:
        raise FlceError(s, "flce_fwd_bwd")
    o["workspace"] = workspace
    return o


def rmsnorm_fwd_bwd(hidden: torch.Tensor, gain: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor,
                    eps: float = 1e-6, ignore_index: int = -100, reduction: str = "mean", *,
                    workspace: Optional[torch.Tensor] = None, row_loss: bool = False, out: Optional[dict] = None,
                    stream=None, grad_weight_dtype=torch.float32) -> dict:
    """Final RMSNorm (x = h / rms(h) * gain) fused in front of the LM head loss.

    grad_hidden is the gradient with respect to the pre-norm hidden states;
    grad_gain (fp32 [H]) and grad_weight ([V,H], fp32 or bf16) as the parameters'."""
    N, H, V = _check_inputs(hidden, weight, targets)
    if gain.dtype != torch.bfloat16 or gain.shape != (H,) or not gain.is_cuda or not gain.is_contiguous():
        raise ValueError("gain must be a contiguous bf16 CUDA tensor of shape [H]")
    dev = hidden.device
    flags = _flags(reduction, grad_weight_dtype)
    if workspace is None:
        nb = library().flce_rmsnorm_workspace_bytes(N, H, V, flags)
        if nb == 0:
            raise FlceError(FLCE_EINVAL, "workspace size")
        workspace = new_workspace(nb, dev)
    o = out if out is not None else {}
    if "loss" not in o:
        o["loss"] = torch.empty(1, dtype=torch.float32, device=dev)
        o["n_valid"] = torch.empty(1, dtype=torch.int32, device=dev)
        o["grad_hidden"] = torch.empty((N, H), dtype=torch.bfloat16, device=dev)
        o["grad_gain"] = torch.empty(H, dtype=torch.float32, device=dev)
        o["grad_weight"] = torch.empty((V, H), dtype=grad_weight_dtype, device=dev)
        o["row_loss"] = torch.empty(N, dtype=torch.float32, device=dev) if row_loss else None
    if o["grad_weight"].dtype != grad_weight_dtype:
        raise TypeError("out['grad_weight'] does not have grad_weight_dtype")
    s = library().flce_rmsnorm_fwd_bwd(_ptr(hidden), _ptr(gain), float(eps), _ptr(weight), _ptr(targets), N, H, V,
                                       _ignored(ignore_index), flags, _ptr(o["loss"]), _ptr(o["n_valid"]),
                                       _ptr(o.get("row_loss")), _ptr(o["grad_hidden"]), _ptr(o["grad_gain"]),
                                       _ptr(o["grad_weight"]), _ptr(workspace), workspace.numel(), _stream(stream))
    if s != FLCE_OK:
        raise FlceError(s, "flce_rmsnorm_fwd_bwd")
    o["workspace"] = workspace
    return o


def loss(hidden: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor, ignore_index: int = -100,
         reduction: str = "mean", *, workspace: Optional[torch.Tensor] = None, row_loss: bool = False,
         out: Optional[dict] = None, stream=None) -> dict:
    """Forward only: loss, n_valid and optionally the per-token loss."""
    N, H, V = _check_inputs(hidden, weight, targets)
    dev = hidden.device
    if workspace is None:
        workspace = new_workspace(workspace_bytes(N, H, V, reduction, forward_only=True), dev)
    o = out if out is not None else {}
    if "loss" not in o:
        o["loss"] = torch.empty(1, dtype=torch.float32, device=dev)
        o["n_valid"] = torch.empty(1, dtype=torch.int32, device=dev)
        o["row_loss"] = torch.empty(N, dtype=torch.float32, device=dev) if row_loss else None
    s = library().flce_loss(_ptr(hidden), _ptr(weight), _ptr(targets), N, H, V, _ignored(ignore_index),
                            REDUCE[reduction], _ptr(o["loss"]), _ptr(o["n_valid"]), _ptr(o.get("row_loss")),
                            _ptr(workspace), workspace.numel(), _stream(stream))
    if s != FLCE_OK:
        raise FlceError(s, "flce_loss")
    o["workspace"] = workspace
    return o


# ---------------------------------------------------------------------------
# vocabulary-parallel LM head (see include/flce.h); the collectives between
# the calls are the caller's
# ---------------------------------------------------------------------------

def _ok(s, what):
    if s != FLCE_OK:
        raise FlceError(s, what)


def vocab_shard_stats(hidden, weight_shard, targets, v0: int, V_total: int, ignore_index: int = -100,
                      workspace=None, stream=None) -> dict:
    N, H = hidden.shape
    Vs = weight_shard.shape[0]
    dev = hidden.device
    if workspace is None:
        workspace = new_workspace(library().flce_vocab_shard_workspace_bytes(N, H, Vs, 0), dev)
    o = {k: torch.empty(N, dtype=torch.float32, device=dev) for k in ("row_max", "row_sumexp", "row_target_logit")}
    o["n_valid"] = torch.empty(1, dtype=torch.int32, device=dev)
    _ok(library().flce_vocab_shard_stats(_ptr(hidden), _ptr(weight_shard), _ptr(targets), N, H, Vs, v0, V_total,
                                         _ignored(ignore_index), _ptr(o["row_max"]), _ptr(o["row_sumexp"]),
                                         _ptr(o["row_target_logit"]), _ptr(o["n_valid"]), _ptr(workspace),
                                         workspace.numel(), _stream(stream)), "flce_vocab_shard_stats")
    o["workspace"] = workspace
    return o


def vocab_rescale(row_max_local, row_max_global, row_sumexp, stream=None) -> None:
    _ok(library().flce_vocab_rescale(_ptr(row_max_local), _ptr(row_max_global), _ptr(row_sumexp),
                                     row_sumexp.numel(), _stream(stream)), "flce_vocab_rescale")


def vocab_finish(row_max, row_sumexp, row_target_logit, targets, ignore_index: int = -100,
                 reduction: str = "mean", stream=None) -> dict:
    N = targets.shape[0]
    dev = targets.device
    o = {"lse": torch.empty(N, dtype=torch.float32, device=dev),
         "row_loss": torch.empty(N, dtype=torch.float32, device=dev),
         "loss": torch.empty(1, dtype=torch.float32, device=dev),
         "n_valid": torch.empty(1, dtype=torch.int32, device=dev)}
    _ok(library().flce_vocab_finish(_ptr(row_max), _ptr(row_sumexp), _ptr(row_target_logit), _ptr(targets), N,
                                    _ignored(ignore_index), REDUCE[reduction], _ptr(o["lse"]), _ptr(o["row_loss"]),
                                    _ptr(o["loss"]), _ptr(o["n_valid"]), _stream(stream)), "flce_vocab_finish")
    return o


def vocab_shard_bwd(hidden, weight_shard, targets, lse, v0: int, V_total: int, ignore_index: int = -100,
                    reduction: str = "mean", workspace=None, stream=None) -> dict:
    N, H = hidden.shape
    Vs = weight_shard.shape[0]
    dev = hidden.device
    if workspace is None:
        workspace = new_workspace(library().flce_vocab_shard_workspace_bytes(N, H, Vs, REDUCE[reduction]), dev)
    o = {"grad_hidden_partial": torch.empty((N, H), dtype=torch.float32, device=dev),
         "grad_weight": torch.empty((Vs, H), dtype=torch.float32, device=dev)}
    _ok(library().flce_vocab_shard_bwd(_ptr(hidden), _ptr(weight_shard), _ptr(targets), N, H, Vs, v0, V_total,
                                       _ignored(ignore_index), REDUCE[reduction], _ptr(lse),
                                       _ptr(o["grad_hidden_partial"]), _ptr(o["grad_weight"]), _ptr(workspace),
                                       workspace.numel(), _stream(stream)), "flce_vocab_shard_bwd")
    o["workspace"] = workspace
    return o


def scale_grads(grad_hidden: torch.Tensor, grad_weight: torch.Tensor, scale: torch.Tensor, stream=None) -> None:
    """grad_hidden and grad_weight *= scale (a one-element fp32 CUDA tensor), in place, on the device."""
    if scale.dtype != torch.float32 or scale.numel() != 1 or not scale.is_cuda:
        raise TypeError("scale must be a one-element float32 CUDA tensor")
    N, H = grad_hidden.shape
    V = grad_weight.shape[0]
    s = library().flce_scale_grads(_ptr(grad_hidden), _ptr(grad_weight), N, H, V, _ptr(scale.contiguous()),
                                   _stream(stream))
    if s != FLCE_OK:
        raise FlceError(s, "flce_scale_grads")


def _leaves(ctx):
    return [node for node, _ in ctx.next_functions if node is not None and type(node).__name__ == "AccumulateGrad"]


def _mark_leaves(ctx, device) -> None:
    """Notes on each leaf's accumulator the stream it was first used on.  The
    accumulator keeps that stream, and lives as long as any graph of the leaf.
    (What other libraries' operators made first has no note, or that of the first
    operator here: autograd does not tell an accumulator's stream.)"""
    for node in _leaves(ctx):
        if "flce_stream" not in node.metadata:
            node.metadata["flce_stream"] = torch._C._cuda_getCurrentRawStream(device.index)


def _check_capture(ctx) -> None:
    """Refuses a captured backward whose leaves belong to a living graph of the
    default stream: autograd would make that stream, which cannot be captured,
    wait for the capture, and the process would end."""
    if torch.cuda.is_current_stream_capturing():
        if any(node.metadata.get("flce_stream") == 0 for node in _leaves(ctx)):
            raise RuntimeError("backward captured while an eager graph of the same leaves, made on the default "
                               "stream, is alive: drop its loss and outputs first, or make it on another stream")


class _LinearCrossEntropyFn(torch.autograd.Function):
    """Forward computes the loss and both gradients in one library call; the
    backward only scales those gradients by the incoming gradient of the loss."""

    @staticmethod
    def forward(ctx, hidden, weight, targets, ignore_index, reduction):
        o = fwd_bwd(hidden.contiguous(), weight.contiguous(), targets.contiguous(), ignore_index, reduction)
        ctx.grads = (o["grad_hidden"], o["grad_weight"])
        ctx.n_valid = o["n_valid"]
        _mark_leaves(ctx, hidden.device)
        return o["loss"].reshape(())

    @staticmethod
    def backward(ctx, grad_loss):
        _check_capture(ctx)
        gh, gw = ctx.grads
        ctx.grads = None
        scale_grads(gh, gw, grad_loss.detach().reshape(1).to(torch.float32))
        # autograd casts grad_weight (fp32) to the weight's dtype if they differ
        return gh, gw, None, None, None


def linear_cross_entropy(hidden: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor,
                         ignore_index: int = -100, reduction: str = "mean") -> torch.Tensor:
    """Drop-in for ``F.cross_entropy(hidden @ weight.T, targets, ignore_index=...)``
    with autograd support; the N x V logits are never materialised."""
    return _LinearCrossEntropyFn.apply(hidden, weight, targets, ignore_index, reduction)


class LinearCrossEntropy(torch.nn.Module):
    """LM head + cross-entropy as one module: ``loss = module(hidden, targets)``."""

    def __init__(self, weight: torch.Tensor, ignore_index: int = -100, reduction: str = "mean"):
        super().__init__()
        self.weight = torch.nn.Parameter(weight)
        self.ignore_index = ignore_index
        self.reduction = reduction

    def forward(self, hidden: torch.Tensor, targets: torch.Tensor) -> torch.Tensor:
        return linear_cross_entropy(hidden, self.weight, targets, self.ignore_index, self.reduction)


# ---------------------------------------------------------------------------
# token log probabilities, with entropy and top alternatives
# ---------------------------------------------------------------------------

TOP_K_MAX = 32


def _addr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


class _on:
    """The device and stream of a call: outputs and workspaces allocated inside
    belong to that stream, so their memory is reused only behind its work.  The
    usual call (current device, current stream) switches nothing: entering
    torch's device and stream contexts costs 18 us, several times the launch of
    a small kernel."""

    __slots__ = ("device", "stream", "contexts")

    def __init__(self, device, stream):
        self.device, self.stream, self.contexts = device, stream, None

    def __enter__(self) -> int:
        if self.stream is None and self.device.index == torch.cuda.current_device():
            return torch._C._cuda_getCurrentRawStream(self.device.index)
        self.contexts = contextlib.ExitStack()
        self.contexts.enter_context(torch.cuda.device(self.device))
        stream = self.stream
        if stream is None:
            stream = torch.cuda.current_stream(self.device)
        elif not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream), device=self.device)
        self.contexts.enter_context(torch.cuda.stream(stream))
        return stream.cuda_stream

    def __exit__(self, *exc):
        if self.contexts is not None:
            self.contexts.__exit__(*exc)


def _check_buffer(t, name, shape, dtype, device):
    if not isinstance(t, torch.Tensor) or t.dtype != dtype:
        raise TypeError(f"{name} must be a {dtype} tensor")
    if tuple(t.shape) != tuple(shape) or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name} must be contiguous, of shape {tuple(shape)}, on {device}")


def _outputs(out, specs, device):
    """The caller's output dict (or a new one), checked and with what it lacks,
    and the tensors that the call writes.  A spec of None is not produced: what
    the dict holds there stays as it is."""
    o = out if out is not None else {}
    for name, spec in specs.items():
        if spec is not None and o.get(name) is not None:
            _check_buffer(o[name], name, spec[0], spec[1], device)
    made = {}
    for name, spec in specs.items():
        if spec is None:
            made[name] = None
            o.setdefault(name, None)
        else:
            if o.get(name) is None:
                o[name] = torch.empty(spec[0], dtype=spec[1], device=device)
            made[name] = o[name]
    return o, made


def _check_same_device(*tensors):
    dev = tensors[0].device
    for t in tensors[1:]:
        if t.device != dev:
            raise ValueError("all tensors must be on one device")
    return dev


def _check_workspace(workspace, device):
    if workspace.dtype != torch.uint8 or not workspace.is_contiguous() or workspace.device != device:
        raise ValueError(f"workspace must be a contiguous uint8 tensor on {device}")


def token_logprobs(hidden: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor, ignore_index: int = -100, *,
                   temperature: float = 1.0, top_k: int = 0, entropy: bool = True,
                   workspace: Optional[torch.Tensor] = None, out: Optional[dict] = None, stream=None) -> dict:
    """Log probabilities of the given tokens under ``softmax(hidden @ weight.T / temperature)``.

    Returns fp32 [N] ``logp``, ``lse`` and (unless ``entropy=False``) ``entropy``;
    with ``top_k`` > 0 also ``top_ids`` (int32 [N, top_k]) and ``top_logp`` (fp32),
    best first, equal logits by the lower id.  Rows whose target is
    ``ignore_index`` hold 0 (ids -1); rows whose target lies outside [0, V) hold
    NaN and set the status word.  ``out`` may hold outputs to write into; it is
    returned, and entries that are not asked for stay as they are."""
    N, H, V = _check_inputs(hidden, weight, targets)
    dev = _check_same_device(hidden, weight, targets)
    top_k = int(top_k)
    if not 0 <= top_k <= min(TOP_K_MAX, V):
        raise ValueError(f"top_k must lie in [0, {min(TOP_K_MAX, V)}]")
    with _on(dev, stream) as st:
        if workspace is None:
            nb = library().flce_logprobs_workspace_bytes(N, H, V, top_k)
            if nb == 0:
                raise FlceError(FLCE_EINVAL, "workspace size")
            workspace = new_workspace(nb, dev)
        else:
            _check_workspace(workspace, dev)
        if out is None:   # spelled out: a decode step is as short as its host work
            f32 = torch.float32
            o = {"logp": torch.empty(N, dtype=f32, device=dev), "lse": torch.empty(N, dtype=f32, device=dev),
                 "entropy": torch.empty(N, dtype=f32, device=dev) if entropy else None,
                 "top_ids": torch.empty((N, top_k), dtype=torch.int32, device=dev) if top_k else None,
                 "top_logp": torch.empty((N, top_k), dtype=f32, device=dev) if top_k else None}
            made = o
        else:
            row = ((N,), torch.float32)
            o, made = _outputs(out, {"logp": row, "lse": row, "entropy": row if entropy else None,
                                     "top_ids": ((N, top_k), torch.int32) if top_k else None,
                                     "top_logp": ((N, top_k), torch.float32) if top_k else None}, dev)
        _ok(library().flce_logprobs(_addr(hidden), _addr(weight), _addr(targets), N, H, V, _ignored(ignore_index),
                                    float(temperature), top_k, _addr(made["logp"]), _addr(made["entropy"]),
                                    _addr(made["lse"]), _addr(made["top_ids"]), _addr(made["top_logp"]),
                                    _addr(workspace), workspace.numel(), st), "flce_logprobs")
    o["workspace"] = workspace
    return o


def token_logprobs_bwd(hidden: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor, lse: torch.Tensor,
                       entropy: Optional[torch.Tensor], grad_logp: Optional[torch.Tensor],
                       grad_entropy: Optional[torch.Tensor] = None, ignore_index: int = -100, *,
                       temperature: float = 1.0, grad_weight_dtype=torch.float32, need_hidden: bool = True,
                       need_weight: bool = True, workspace: Optional[torch.Tensor] = None,
                       out: Optional[dict] = None, stream=None) -> dict:
    """Gradients of ``sum(grad_logp * logp + grad_entropy * entropy)``.

    ``lse`` and ``entropy`` are those of :func:`token_logprobs` on the same
    inputs (``entropy`` may be None without ``grad_entropy``).  Returns
    ``grad_hidden`` (bf16 [N, H]) and ``grad_weight`` ([V, H], fp32 or bf16), or
    only the one asked for: a frozen head or a frozen trunk saves its product."""
    N, H, V = _check_inputs(hidden, weight, targets)
    dev = _check_same_device(hidden, weight, targets)
    if not (need_hidden or need_weight):
        raise ValueError("need_hidden or need_weight must be set")
    if grad_logp is None and grad_entropy is None:
        raise ValueError("grad_logp or grad_entropy must be given")
    if grad_entropy is not None and entropy is None:
        raise ValueError("grad_entropy needs the entropy")
    for name, t in (("lse", lse), ("entropy", entropy), ("grad_logp", grad_logp), ("grad_entropy", grad_entropy)):
        if t is not None or name == "lse":
            _check_buffer(t, name, (N,), torch.float32, dev)
    flags = _flags("mean", grad_weight_dtype) if need_weight else 0
    with _on(dev, stream) as st:
        if workspace is None:
            nb = library().flce_logprobs_bwd_workspace_bytes(N, H, V, flags)
            if nb == 0:
                raise FlceError(FLCE_EINVAL, "workspace size")
            workspace = new_workspace(nb, dev)
        else:
            _check_workspace(workspace, dev)
        o, made = _outputs(out, {"grad_hidden": ((N, H), torch.bfloat16) if need_hidden else None,
                                 "grad_weight": ((V, H), grad_weight_dtype) if need_weight else None}, dev)
        _ok(library().flce_logprobs_bwd(_addr(hidden), _addr(weight), _addr(targets), N, H, V, _ignored(ignore_index), flags,
                                        float(temperature), _addr(lse), _addr(entropy), _addr(grad_logp),
                                        _addr(grad_entropy), _addr(made["grad_hidden"]),
                                        _addr(made["grad_weight"]), _addr(workspace), workspace.numel(), st), "flce_logprobs_bwd")
    o["workspace"] = workspace
    return o


class _LinearLogProbsFn(torch.autograd.Function):
    """The backward recomputes the logits chunk by chunk from the saved log-sum-exp."""

    @staticmethod
    def forward(ctx, hidden, weight, targets, ignore_index, temperature):
        hidden, weight, targets = hidden.contiguous(), weight.contiguous(), targets.contiguous()
        o = token_logprobs(hidden, weight, targets, ignore_index, temperature=temperature)
        ctx.save_for_backward(hidden, weight, targets, o["lse"], o["entropy"])
        ctx.args = (ignore_index, temperature)
        ctx.set_materialize_grads(False)
        _mark_leaves(ctx, hidden.device)
        return o["logp"], o["entropy"]

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_logp, grad_entropy):
        need_hidden, need_weight = ctx.needs_input_grad[:2]
        if not (need_hidden or need_weight) or (grad_logp is None and grad_entropy is None):
            return None, None, None, None, None
        _check_capture(ctx)
        hidden, weight, targets, lse, entropy = ctx.saved_tensors
        ignore_index, temperature = ctx.args
        gl = None if grad_logp is None else grad_logp.to(torch.float32).contiguous()
        ge = None if grad_entropy is None else grad_entropy.to(torch.float32).contiguous()
        o = token_logprobs_bwd(hidden, weight, targets, lse, entropy, gl, ge, ignore_index, temperature=temperature,
                               grad_weight_dtype=weight.dtype, need_hidden=need_hidden, need_weight=need_weight)
        return o["grad_hidden"], o["grad_weight"], None, None, None


def linear_logprobs(hidden: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor, ignore_index: int = -100,
                    temperature: float = 1.0):
    """``(logp, entropy)`` of the given tokens at the LM head, fp32 [N] each, with
    autograd support: the head of a policy-gradient or preference loss.  Forward
    and backward may be captured into one CUDA graph; an eager graph of the same
    leaves, made by this module on the default stream and still alive, is refused
    there.  (One made by other operators is not seen, and autograd ends the
    process: drop it before the capture.)"""
    return _LinearLogProbsFn.apply(hidden, weight, targets, ignore_index, temperature)


class LinearLogProbs(torch.nn.Module):
    """LM head as token log probabilities: ``logp, entropy = module(hidden, targets)``;
    the weight may be an embedding's (tied)."""

    def __init__(self, weight: torch.Tensor, ignore_index: int = -100, temperature: float = 1.0):
        super().__init__()
        self.weight = weight if isinstance(weight, torch.nn.Parameter) else torch.nn.Parameter(weight)
        self.ignore_index = ignore_index
        self.temperature = temperature

    def forward(self, hidden: torch.Tensor, targets: torch.Tensor):
        return linear_logprobs(hidden, self.weight, targets, self.ignore_index, self.temperature)


# ---------------------------------------------------------------------------
# the next token under constraints
# ---------------------------------------------------------------------------

def _check_head(hidden, weight):
    if not (hidden.is_cuda and weight.is_cuda):
        raise ValueError("hidden and weight must be CUDA tensors")
    if hidden.dtype != torch.bfloat16 or weight.dtype != torch.bfloat16:
        raise TypeError("hidden and weight must be bfloat16")
    if hidden.dim() != 2 or weight.dim() != 2 or weight.shape[1] != hidden.shape[1]:
        raise ValueError("expected hidden [N,H], weight [V,H]")
    if not (hidden.is_contiguous() and weight.is_contiguous()):
        raise ValueError("hidden and weight must be contiguous")
    return hidden.shape[0], hidden.shape[1], weight.shape[0], _check_same_device(hidden, weight)


def _rows_of(t, name, dtype, rows, device) -> int:
    """Row stride of a [rows, *] matrix whose rows are contiguous (0: one row for all, as expand gives)."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")
    if t.dim() != 2 or t.shape[0] != rows:
        raise ValueError(f"{name} must be a matrix of {rows} rows")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    return t.stride(0)


def _row_values(t, name, dtype, rows, device):
    """The address of a contiguous vector of one value per row, or of nothing."""
    if t is None:
        return None
    _check_buffer(t, name, (rows,), dtype, device)
    return t.data_ptr()


def constrained_logprobs(hidden: torch.Tensor, weight: torch.Tensor, targets: Optional[torch.Tensor] = None,
                         ignore_index: int = -100, *, history: Optional[torch.Tensor] = None,
                         history_lens: Optional[torch.Tensor] = None, prompt_lens: Optional[torch.Tensor] = None,
                         repetition_penalty: Optional[torch.Tensor] = None,
                         frequency_penalty: Optional[torch.Tensor] = None,
                         presence_penalty: Optional[torch.Tensor] = None, bias_ids: Optional[torch.Tensor] = None,
                         bias: Optional[torch.Tensor] = None, mask: Optional[torch.Tensor] = None,
                         temperature: float = 1.0, top_k: int = 0, entropy: bool = True,
                         workspace: Optional[torch.Tensor] = None, out: Optional[dict] = None, stream=None) -> dict:
    """:func:`token_logprobs` of logits that penalties, biases and a mask have changed, as a decode step samples them.

    For row n and token v, in this order: a token of the row's history has its
    logit divided by ``repetition_penalty[n]`` where it is positive, else
    multiplied; one that its output holds c > 0 times loses
    ``frequency_penalty[n] * c + presence_penalty[n]``; a token that
    ``bias_ids[n]`` names gets ``bias[n]`` added (of one named twice the last
    entry holds); a token whose bit in ``mask`` is not set is forbidden.

    ``history`` is int32 [N, L] (ids outside [0, V) are padding), of whose rows
    the first ``history_lens`` entries count, of these the first ``prompt_lens``
    as the prompt; ``bias_ids`` and ``bias`` are int32 and fp32 [N, B]; ``mask``
    is int32 [N, ceil(V / 32)], bit v % 32 of word v // 32; the penalties and
    lengths are [N].  The matrices' rows may be strided, or one row expanded.

    Returns what :func:`token_logprobs` does; without ``targets`` every row
    counts and ``logp`` is None.  A forbidden target has a log probability of
    -inf, forbidden tokens are no alternatives (ids -1), and a row with nothing
    left has ``lse`` -inf and entropy 0.  There is no gradient."""
    N, H, V, dev = _check_head(hidden, weight)
    if targets is not None:
        _check_buffer(targets, "targets", (N,), torch.int32, dev)
    top_k = int(top_k)
    if not 0 <= top_k <= min(TOP_K_MAX, V):
        raise ValueError(f"top_k must lie in [0, {min(TOP_K_MAX, V)}]")
    c = _Constraints()
    if history is not None:
        c.history_stride = _rows_of(history, "history", torch.int32, N, dev)
        c.history, c.history_len = history.data_ptr(), history.shape[1]
    elif history_lens is not None or prompt_lens is not None:
        raise ValueError("history_lens and prompt_lens need a history")
    c.history_lens = _row_values(history_lens, "history_lens", torch.int32, N, dev)
    c.prompt_lens = _row_values(prompt_lens, "prompt_lens", torch.int32, N, dev)
    for name, t in (("repetition_penalty", repetition_penalty), ("frequency_penalty", frequency_penalty),
                    ("presence_penalty", presence_penalty)):
        if t is not None:
            if history is None:
                raise ValueError(f"{name} needs a history")
            setattr(c, name, _row_values(t, name, torch.float32, N, dev))
    if (bias_ids is None) != (bias is None):
        raise ValueError("bias_ids and bias go together")
    if bias is not None:
        c.bias_ids_stride = _rows_of(bias_ids, "bias_ids", torch.int32, N, dev)
        c.bias_stride = _rows_of(bias, "bias", torch.float32, N, dev)
        if bias.shape != bias_ids.shape:
            raise ValueError("bias_ids and bias must have one shape")
        c.bias_ids, c.bias, c.n_bias = bias_ids.data_ptr(), bias.data_ptr(), bias.shape[1]
    if mask is not None:
        c.mask_stride = _rows_of(mask, "mask", torch.int32, N, dev)
        if mask.shape[1] < (V + 31) // 32:
            raise ValueError("mask must have a bit for every token")
        c.mask = mask.data_ptr()
    with _on(dev, stream) as st:
        if workspace is None:
            nb = library().flce_constrained_workspace_bytes(N, H, V, top_k, c.history_len, c.n_bias)
            if nb == 0:
                raise FlceError(FLCE_EINVAL, "workspace size")
            workspace = new_workspace(nb, dev)
        else:
            _check_workspace(workspace, dev)
        if out is None:   # spelled out: a decode step is as short as its host work
            f32 = torch.float32
            o = made = {"logp": torch.empty(N, dtype=f32, device=dev) if targets is not None else None,
                        "lse": torch.empty(N, dtype=f32, device=dev),
                        "entropy": torch.empty(N, dtype=f32, device=dev) if entropy else None,
                        "top_ids": torch.empty((N, top_k), dtype=torch.int32, device=dev) if top_k else None,
                        "top_logp": torch.empty((N, top_k), dtype=f32, device=dev) if top_k else None}
        else:
            row = ((N,), torch.float32)
            o, made = _outputs(out, {"logp": row if targets is not None else None, "lse": row,
                                     "entropy": row if entropy else None,
                                     "top_ids": ((N, top_k), torch.int32) if top_k else None,
                                     "top_logp": ((N, top_k), torch.float32) if top_k else None}, dev)
        _ok(library().flce_constrained_logprobs(_addr(hidden), _addr(weight), _addr(targets), N, H, V,
                                                _ignored(ignore_index), float(temperature), top_k, ctypes.byref(c),
                                                _addr(made["logp"]), _addr(made["entropy"]), _addr(made["lse"]),
                                                _addr(made["top_ids"]), _addr(made["top_logp"]), _addr(workspace),
                                                workspace.numel(), st), "flce_constrained_logprobs")
    o["workspace"] = workspace
    return o


# ---------------------------------------------------------------------------
# distillation from a teacher's top log probabilities
# ---------------------------------------------------------------------------

TEACHER_MAX = 256


def _check_teacher(teacher_ids, teacher_logp, N, device) -> int:
    if teacher_ids.dtype != torch.int32 or teacher_logp.dtype != torch.float32:
        raise TypeError("teacher_ids must be int32, teacher_logp float32")
    if teacher_ids.dim() != 2 or teacher_ids.shape[0] != N or teacher_logp.shape != teacher_ids.shape:
        raise ValueError("expected teacher_ids [N,K], teacher_logp [N,K]")
    if not (teacher_ids.is_contiguous() and teacher_logp.is_contiguous()):
        raise ValueError("teacher_ids and teacher_logp must be contiguous")
    if teacher_ids.device != device or teacher_logp.device != device:
        raise ValueError("all tensors must be on one device")
    K = teacher_ids.shape[1]
    if not 1 <= K <= TEACHER_MAX:
        raise ValueError(f"a row may have 1 to {TEACHER_MAX} teacher tokens")
    return K


def topk_distill(hidden: torch.Tensor, weight: torch.Tensor, teacher_ids: torch.Tensor, teacher_logp: torch.Tensor, *,
                 temperature: float = 1.0, tail: bool = True, workspace: Optional[torch.Tensor] = None,
                 out: Optional[dict] = None, stream=None) -> dict:
    """Kullback-Leibler divergence of ``softmax(hidden @ weight.T / temperature)`` from a teacher's list, per token.

    ``teacher_ids`` (int32 [N, K], K <= 256; negative: no entry) and
    ``teacher_logp`` (fp32 [N, K]) are a teacher's likeliest tokens and their log
    probabilities at the same temperature, as :func:`token_logprobs` gives them
    (``top_ids``, ``top_logp``).  With ``tail=True`` the mass that the list
    leaves is compared with the student's behind it; with ``tail=False`` the
    list is taken as the whole distribution (``softmax`` of ``teacher_logp``,
    which may then be logits).

    Returns fp32 ``kl`` [N] (not scaled by temperature squared), ``lse`` and
    ``rest_logp`` [N] (the log of the student's mass behind the list), and
    ``student_logp`` [N, K].  Rows without an entry hold 0; rows that name a
    token of V or more hold NaN and set the status word."""
    N, H, V, dev = _check_head(hidden, weight)
    K = _check_teacher(teacher_ids, teacher_logp, N, dev)
    with _on(dev, stream) as st:
        if workspace is None:
            nb = library().flce_topk_distill_workspace_bytes(N, H, V, K)
            if nb == 0:
                raise FlceError(FLCE_EINVAL, "workspace size")
            workspace = new_workspace(nb, dev)
        else:
            _check_workspace(workspace, dev)
        if out is None:   # spelled out: a small call is as short as its host work
            f32 = torch.float32
            o = made = {"kl": torch.empty(N, dtype=f32, device=dev), "lse": torch.empty(N, dtype=f32, device=dev),
                        "rest_logp": torch.empty(N, dtype=f32, device=dev),
                        "student_logp": torch.empty((N, K), dtype=f32, device=dev)}
        else:
            row = ((N,), torch.float32)
            o, made = _outputs(out, {"kl": row, "lse": row, "rest_logp": row, "student_logp": ((N, K), torch.float32)},
                               dev)
        _ok(library().flce_topk_distill(_addr(hidden), _addr(weight), _addr(teacher_ids), _addr(teacher_logp), N, H, V, K,
                                        float(temperature), int(bool(tail)), _addr(made["kl"]), _addr(made["lse"]),
                                        _addr(made["rest_logp"]), _addr(made["student_logp"]), _addr(workspace),
                                        workspace.numel(), st), "flce_topk_distill")
    o["workspace"] = workspace
    return o


def topk_distill_bwd(hidden: torch.Tensor, weight: torch.Tensor, teacher_ids: torch.Tensor, teacher_logp: torch.Tensor,
                     lse: torch.Tensor, rest_logp: torch.Tensor, student_logp: torch.Tensor, grad_kl: torch.Tensor, *,
                     temperature: float = 1.0, tail: bool = True, grad_weight_dtype=torch.float32,
                     need_hidden: bool = True, need_weight: bool = True, workspace: Optional[torch.Tensor] = None,
                     out: Optional[dict] = None, stream=None) -> dict:
    """Gradients of ``sum(grad_kl * kl)``; ``lse``, ``rest_logp`` and ``student_logp``
    are those of :func:`topk_distill` on the same inputs.  Returns
    ``grad_hidden`` (bf16 [N, H]) and ``grad_weight`` ([V, H], fp32 or bf16), or
    only the one asked for, as exact as an fp32 gradient of the logits gives them.
    The teacher gets no gradient."""
    N, H, V, dev = _check_head(hidden, weight)
    K = _check_teacher(teacher_ids, teacher_logp, N, dev)
    if not (need_hidden or need_weight):
        raise ValueError("need_hidden or need_weight must be set")
    for name, t, shape in (("lse", lse, (N,)), ("rest_logp", rest_logp, (N,)), ("student_logp", student_logp, (N, K)),
                           ("grad_kl", grad_kl, (N,))):
        _check_buffer(t, name, shape, torch.float32, dev)
    flags = _flags("mean", grad_weight_dtype) if need_weight else 0
    with _on(dev, stream) as st:
        if workspace is None:
            nb = library().flce_topk_distill_bwd_workspace_bytes(N, H, V, K, flags)
            if nb == 0:
                raise FlceError(FLCE_EINVAL, "workspace size")
            workspace = new_workspace(nb, dev)
        else:
            _check_workspace(workspace, dev)
        o, made = _outputs(out, {"grad_hidden": ((N, H), torch.bfloat16) if need_hidden else None,
                                 "grad_weight": ((V, H), grad_weight_dtype) if need_weight else None}, dev)
        _ok(library().flce_topk_distill_bwd(_addr(hidden), _addr(weight), _addr(teacher_ids), _addr(teacher_logp), N, H,
                                            V, K, flags, float(temperature), int(bool(tail)), _addr(lse),
                                            _addr(rest_logp), _addr(student_logp), _addr(grad_kl),
                                            _addr(made["grad_hidden"]), _addr(made["grad_weight"]), _addr(workspace),
                                            workspace.numel(), st), "flce_topk_distill_bwd")
    o["workspace"] = workspace
    return o


class _LinearTopKDistillFn(torch.autograd.Function):
    """The backward recomputes the logits chunk by chunk from the saved row values."""

    @staticmethod
    def forward(ctx, hidden, weight, teacher_ids, teacher_logp, temperature, tail):
        hidden, weight = hidden.contiguous(), weight.contiguous()
        teacher_ids, teacher_logp = teacher_ids.contiguous(), teacher_logp.contiguous()
        o = topk_distill(hidden, weight, teacher_ids, teacher_logp, temperature=temperature, tail=tail)
        ctx.save_for_backward(hidden, weight, teacher_ids, teacher_logp, o["lse"], o["rest_logp"], o["student_logp"])
        ctx.args = (temperature, tail)
        _mark_leaves(ctx, hidden.device)
        return o["kl"]

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_kl):
        need_hidden, need_weight = ctx.needs_input_grad[:2]
        if not (need_hidden or need_weight):
            return None, None, None, None, None, None
        _check_capture(ctx)
        temperature, tail = ctx.args
        o = topk_distill_bwd(*ctx.saved_tensors, grad_kl.to(torch.float32).contiguous(), temperature=temperature,
                             tail=tail, grad_weight_dtype=ctx.saved_tensors[1].dtype, need_hidden=need_hidden,
                             need_weight=need_weight)
        return o["grad_hidden"], o["grad_weight"], None, None, None, None


def linear_topk_distill(hidden: torch.Tensor, weight: torch.Tensor, teacher_ids: torch.Tensor,
                        teacher_logp: torch.Tensor, temperature: float = 1.0, tail: bool = True) -> torch.Tensor:
    """:func:`topk_distill`'s ``kl`` (fp32 [N]) with autograd support for hidden and
    weight; the teacher gets no gradient.  Captures as :func:`linear_logprobs`."""
    return _LinearTopKDistillFn.apply(hidden, weight, teacher_ids, teacher_logp, temperature, tail)


class LinearTopKDistill(torch.nn.Module):
    """LM head as a distillation loss: ``kl = module(hidden, teacher_ids, teacher_logp)``;
    the weight may be an embedding's (tied)."""

    def __init__(self, weight: torch.Tensor, temperature: float = 1.0, tail: bool = True):
        super().__init__()
        self.weight = weight if isinstance(weight, torch.nn.Parameter) else torch.nn.Parameter(weight)
        self.temperature = temperature
        self.tail = tail

    def forward(self, hidden: torch.Tensor, teacher_ids: torch.Tensor, teacher_logp: torch.Tensor) -> torch.Tensor:
        return linear_topk_distill(hidden, self.weight, teacher_ids, teacher_logp, self.temperature, self.tail)


# ---------------------------------------------------------------------------
# scaled embedding and its gradient
# ---------------------------------------------------------------------------

FLCE_ACCUMULATE = 0x4
EMBEDDING_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


def _check_rows(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in EMBEDDING_DTYPES:
        raise TypeError(f"{name} must be bfloat16, float16 or float32")
    if t.dim() != 2 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous matrix")
    return t.shape


def _check_ids(ids):
    if ids.dtype != torch.int32:
        raise TypeError("ids must be int32")
    if ids.dim() != 1 or not ids.is_contiguous():
        raise ValueError("ids must be a contiguous vector")
    return ids.shape[0]


def embedding_fwd(weight: torch.Tensor, ids: torch.Tensor, scale: float = 1.0, *, out: Optional[torch.Tensor] = None,
                  stream=None) -> torch.Tensor:
    """``scale * weight[ids]``, rounded once to the weight's dtype; rows of ids outside [0, V) are NaN."""
    V, H = _check_rows(weight, "weight")
    N = _check_ids(ids)
    dev = _check_same_device(weight, ids)
    if out is not None:
        _check_buffer(out, "out", (N, H), weight.dtype, dev)
    with _on(dev, stream) as st:
        if out is None:
            out = torch.empty((N, H), dtype=weight.dtype, device=dev)
        s = library().flce_embedding(weight.data_ptr(), ids.data_ptr(), N, H, V, EMBEDDING_DTYPES[weight.dtype],
                                     float(scale), out.data_ptr(), st)
    if s != FLCE_OK:
        raise FlceError(s, "flce_embedding")
    return out


def embedding_bwd(grad_out: torch.Tensor, ids: torch.Tensor, num_rows: int, scale: float = 1.0,
                  padding_idx: Optional[int] = None, *, grad_weight_dtype=torch.float32, accumulate: bool = False,
                  workspace: Optional[torch.Tensor] = None, out: Optional[dict] = None, stream=None) -> dict:
    """``grad_weight`` [num_rows, H] of :func:`embedding_fwd`, summed in fp32 in a fixed order.

    With ``accumulate=True`` the sums are added to ``out["grad_weight"]`` (fp32)
    in place, touching only the rows of ids that occur: the embedding's share of
    a tied weight's gradient on top of the head's."""
    N, H = _check_rows(grad_out, "grad_out")
    if _check_ids(ids) != N:
        raise ValueError("shape mismatch")
    dev = _check_same_device(grad_out, ids)
    V = int(num_rows)
    if grad_weight_dtype not in EMBEDDING_DTYPES:
        raise TypeError("grad_weight_dtype must be bfloat16, float16 or float32")
    if padding_idx is not None and not 0 <= padding_idx < V:
        raise ValueError("padding_idx must lie in [0, num_rows)")
    if accumulate and (out is None or out.get("grad_weight") is None):
        raise ValueError("accumulate needs out['grad_weight']")
    if accumulate and grad_weight_dtype != torch.float32:
        raise TypeError("accumulate needs a float32 grad_weight")
    with _on(dev, stream) as st:
        if workspace is None:
            nb = library().flce_embedding_bwd_workspace_bytes(N, H, V)
            if nb == 0:
                raise FlceError(FLCE_EINVAL, "workspace size")
            workspace = new_workspace(nb, dev)
        else:
            _check_workspace(workspace, dev)
        o, _ = _outputs(out, {"grad_weight": ((V, H), grad_weight_dtype)}, dev)
        _ok(library().flce_embedding_bwd(_addr(grad_out), _addr(ids), N, H, V, EMBEDDING_DTYPES[grad_out.dtype],
                                         float(scale), -1 if padding_idx is None else int(padding_idx),
                                         FLCE_ACCUMULATE if accumulate else 0, _addr(o["grad_weight"]),
                                         EMBEDDING_DTYPES[grad_weight_dtype], _addr(workspace), workspace.numel(), st),
            "flce_embedding_bwd")
    o["workspace"] = workspace
    return o


class _EmbeddingFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, weight, ids, scale, padding_idx):
        ids = ids.contiguous()
        ctx.save_for_backward(ids)
        ctx.args = (weight.shape[0], weight.dtype, scale, padding_idx)
        out = embedding_fwd(weight.contiguous(), ids, scale)
        _mark_leaves(ctx, weight.device)
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_out):
        if not ctx.needs_input_grad[0]:
            return None, None, None, None
        _check_capture(ctx)
        V, dtype, scale, padding_idx = ctx.args
        o = embedding_bwd(grad_out.contiguous(), ctx.saved_tensors[0], V, scale, padding_idx, grad_weight_dtype=dtype)
        return o["grad_weight"], None, None, None


def embedding(ids: torch.Tensor, weight: torch.Tensor, scale: float = 1.0,
              padding_idx: Optional[int] = None) -> torch.Tensor:
    """``scale * weight[ids]`` for int32 ids [N], with autograd support; tokens whose
    id is ``padding_idx`` are looked up but add nothing to the gradient."""
    if padding_idx is not None and not 0 <= padding_idx < weight.shape[0]:
        raise ValueError("padding_idx must lie in [0, V)")
    return _EmbeddingFn.apply(weight, ids, scale, padding_idx)


class ScaledEmbedding(torch.nn.Module):
    """Token embedding ``scale * weight[ids]``; the weight may be an LM head's (tied)."""

    def __init__(self, weight: torch.Tensor, scale: float = 1.0, padding_idx: Optional[int] = None):
        super().__init__()
        self.weight = weight if isinstance(weight, torch.nn.Parameter) else torch.nn.Parameter(weight)
        self.scale = scale
        self.padding_idx = padding_idx

    def forward(self, ids: torch.Tensor) -> torch.Tensor:
        return embedding(ids, self.weight, self.scale, self.padding_idx)


def query_status(workspace: torch.Tensor, stream=None) -> int:
    """Synchronise the stream and return the device status of the last call."""
    return int(library().flce_query_status(_ptr(workspace), _stream(stream)))


def selftest_timeout(workspace: torch.Tensor, timeout_ns: int, stream=None) -> int:
    return int(library().flce_selftest_timeout(_ptr(workspace), int(timeout_ns), _stream(stream)))


def query_stall(workspace: torch.Tensor, stream=None) -> dict:
    """Where the first pipeline wait of the last call ran out of time (site 0: none)."""
    info = (ctypes.c_int32 * 4)()
    s = library().flce_query_stall(_ptr(workspace), info, _stream(stream))
    if s != FLCE_OK:
        raise FlceError(s, "flce_query_stall")
    return {"site": info[0], "cta_rank": info[1], "block": info[2], "count": info[3]}


def debug_arm_stall(timeout_ns: int, after: int = 0) -> None:
    """Test hook: the next GEMM launch, or the one behind ``after`` others, withholds one pipeline signal (see flce.h)."""
    s = library().flce_debug_arm_stall_after(int(timeout_ns), int(after))
    if s != FLCE_OK:
        raise FlceError(s, "flce_debug_arm_stall")


def profile_begin() -> None:
    """Record CUDA events around every GEMM launch of the following calls."""
    library().flce_profile_begin()


def profile_end() -> dict:
    """Synchronise the recorded events; per GEMM mode summed ms and launch counts."""
    ms = (ctypes.c_double * 3)()
    n = (ctypes.c_int64 * 3)()
    total = ctypes.c_int64()
    s = library().flce_profile_end(ms, n, ctypes.byref(total))
    if s != FLCE_OK:
        raise FlceError(s, "flce_profile_end")
    names = ("logits", "backward", "logprobs")
    return {"gemm_ms": dict(zip(names, list(ms))), "gemm_launches": dict(zip(names, list(n))),
            "kernel_launches": int(total.value)}


def version() -> str:
    return library().flce_version().decode()
