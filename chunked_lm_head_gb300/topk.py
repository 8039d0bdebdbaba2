"""Distillation from a teacher's stored top logits, from PyTorch.

The teacher's head does not run: per token, the ids and logits of its best K
words were kept.  ``topk_distill_loss`` is differentiable in the student's
hidden states and head; ``topk_kd_forward``, ``topk_kd_backward`` and
``topk_kd_forward_backward`` are the calls below it.  Every arithmetic step runs
in libflce's CUDA kernels (include/flce.h states the formulas); this module
checks tensor properties, allocates outputs and passes pointers.
"""
from __future__ import annotations

import torch

from . import _lib
from .api import IGNORE_INDEX, _device_scalar, _first_order

_IDS = {torch.int32: _lib.DTYPES["i32"], torch.int64: _lib.DTYPES["i64"]}
_LOGITS = {torch.float32: _lib.DTYPES["f32"], torch.bfloat16: _lib.DTYPES["bf16"], torch.float16: _lib.DTYPES["f16"]}


_DW = {torch.float32: _lib.DTYPES["f32"], torch.bfloat16: _lib.DTYPES["bf16"]}


def _workspace(workspace, nbytes, stream, device):
    """(workspace, bytes): the caller's, or one from torch's allocator, which
    orders its reuse on the current stream; with a stream of the caller's the
    library allocates its own on that stream."""
    if workspace is None:
        if stream is not None:
            return None, 0
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
    elif not workspace.is_cuda:
        raise ValueError("workspace must be a CUDA tensor")
    return workspace, workspace.numel() * workspace.element_size()


def _check(h, W, ids, logits, lse_t, targets, weights, tail):
    """The teacher struct of a call, its tensors checked."""
    for x in (h, W):
        if not x.is_cuda or x.dtype != torch.bfloat16 or x.dim() != 2 or not x.is_contiguous():
            raise ValueError("h and W must be contiguous 2-D bfloat16 CUDA tensors")
    N = h.shape[0]
    if W.shape[1] != h.shape[1]:
        raise ValueError("expected h[N,H] and W[V,H]")
    if ids.dim() != 2 or ids.shape[0] != N or ids.shape != logits.shape or ids.shape[1] < 1:
        raise ValueError("expected ids[N,K] and logits[N,K] with K >= 1")
    if not (ids.is_cuda and logits.is_cuda) or ids.dtype not in _IDS or logits.dtype not in _LOGITS:
        raise ValueError("ids must be int32 or int64, logits float32, bfloat16 or float16, on CUDA")
    K = ids.shape[1]
    if K > 1 and (ids.stride(1) != 1 or logits.stride(1) != 1):
        raise ValueError("the rows of ids and logits must be contiguous")
    for x, dtype, name in ((lse_t, torch.float32, "lse_t"), (weights, torch.float32, "weights"),
                           (targets, torch.int64, "targets")):
        if x is not None and (not x.is_cuda or x.dtype != dtype or x.shape != (N,) or not x.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous {dtype} [N] CUDA tensor")
    if tail and lse_t is None:
        raise ValueError("tail needs lse_t, the teacher's log-sum-exp over the whole vocabulary")
    ld = [x.stride(0) if N > 1 else K for x in (ids, logits)]
    return _lib.TopLogits(ids.data_ptr(), logits.data_ptr(), _lib._ptr(lse_t), ld[0], ld[1], _IDS[ids.dtype],
                          _LOGITS[logits.dtype], K, 1 if tail else 0)


def _check_state(state, N, k):
    if state is None or state.numel() * state.element_size() != _lib.flce_topk_kd_state_bytes(N, k):
        raise ValueError("state must come from topk_kd_forward(for_backward=True) of the same N and k")
    if not state.is_cuda or not state.is_contiguous():
        raise ValueError("state must be a contiguous CUDA tensor")


def topk_kd_forward(h, W, ids, logits, lse_t=None, targets=None, weights=None, tail: bool = False,
                    chunk_rows: int = 256, ignore_index: int = IGNORE_INDEX, transform=None,
                    workspace: torch.Tensor | None = None, stream=None, skip_ignored: bool = False,
                    for_backward: bool = False):
    """dict(kl[N] f32, lse[N] f32, loss[], n_valid[] i64, state) on device.

    ids [N,K] (int32 or int64, a negative id is no entry), logits [N,K]: the
    teacher's logits after its own transform, or log-probs.  lse_t [N]: the
    teacher's log-sum-exp over the whole vocabulary (zeros for log-probs), or
    None: the list's mass is scaled to one.  tail: the mass outside the list is
    one more outcome.  skip_ignored: rows without loss are skipped, their lse
    NaN.  for_backward: state holds what topk_kd_backward reads (else None)."""
    t = _check(h, W, ids, logits, lse_t, targets, weights, tail)
    (N, H), V, dev = h.shape, W.shape[0], h.device
    kl = torch.empty(N, dtype=torch.float32, device=dev)
    lse = torch.empty(N, dtype=torch.float32, device=dev)
    loss = torch.empty((), dtype=torch.float32, device=dev)
    n_valid = torch.empty((), dtype=torch.int64, device=dev)
    state = None
    if for_backward:
        state = torch.empty(_lib.flce_topk_kd_state_bytes(N, t.k), dtype=torch.uint8, device=dev)
    ws, ws_bytes = _workspace(workspace, _lib.flce_topk_kd_workspace_bytes(N, H, V, t.k, chunk_rows), stream, dev)
    st = _lib.flce_topk_kd_forward(h, W, t, targets, weights, N, H, V, chunk_rows, ignore_index, transform,
                                   _lib.FORWARD_SKIP_IGNORED if skip_ignored else 0, kl, lse, loss, n_valid, state,
                                   ws, ws_bytes, stream)
    _lib.check("flce_topk_kd_forward", st)
    return {"kl": kl, "lse": lse, "loss": loss, "n_valid": n_valid, "state": state}


def topk_kd_backward(h, W, state, k: int, grad_scale: float, chunk_rows: int = 256, transform=None,
                     need_dH: bool = True, need_dW: bool = True, workspace: torch.Tensor | None = None, stream=None,
                     scale=None, count=None, dW_dtype=torch.float32):
    """(dH[N,H] bf16 or None, dW[V,H] of dW_dtype (float32 or bfloat16) or None)
    from the forward's state (same h, W, k and transform).  scale / count:
    device-side factors of grad_scale, as in backward()."""
    if dW_dtype not in _DW:
        raise ValueError("dW_dtype must be float32 or bfloat16")
    (N, H), V, dev = h.shape, W.shape[0], h.device
    if W.shape[1] != H or any(not x.is_cuda or x.dtype != torch.bfloat16 or not x.is_contiguous() for x in (h, W)):
        raise ValueError("h[N,H] and W[V,H] must be contiguous bfloat16 CUDA tensors")
    _check_state(state, N, k)
    dH = torch.empty_like(h) if need_dH else None
    dW = torch.empty((V, H), dtype=dW_dtype, device=dev) if need_dW else None
    scale = _device_scalar(scale, torch.float32, dev)
    count = _device_scalar(count, torch.int64, dev)
    ws, ws_bytes = _workspace(workspace, _lib.flce_topk_kd_backward_workspace_bytes(N, H, V, chunk_rows, _DW[dW_dtype]),
                              stream, dev)
    st = _lib.flce_topk_kd_backward(h, W, state, grad_scale, scale, count, dH, dW, _DW[dW_dtype], N, H, V, k,
                                    chunk_rows, transform, ws, ws_bytes, stream)
    _lib.check("flce_topk_kd_backward", st)
    return dH, dW


def topk_kd_forward_backward(h, W, ids, logits, lse_t=None, targets=None, weights=None, tail: bool = False,
                             chunk_rows: int = 4096, ignore_index: int = IGNORE_INDEX, grad_scale: float = 1.0,
                             need_dH: bool = True, need_dW: bool = True, workspace: torch.Tensor | None = None,
                             stream=None, transform=None, need_lse: bool = True, dW_dtype=torch.float32):
    """Loss and its gradients in one call without the logits recompute:
    dict(kl, lse, loss, n_valid, dH, dW), dW of dW_dtype (float32 or bfloat16).
    need_lse=False returns lse None and lets the call skip the rows without
    loss."""
    if dW_dtype not in _DW:
        raise ValueError("dW_dtype must be float32 or bfloat16")
    t = _check(h, W, ids, logits, lse_t, targets, weights, tail)
    (N, H), V, dev = h.shape, W.shape[0], h.device
    kl = torch.empty(N, dtype=torch.float32, device=dev)
    lse = torch.empty(N, dtype=torch.float32, device=dev) if need_lse else None
    loss = torch.empty((), dtype=torch.float32, device=dev)
    n_valid = torch.empty((), dtype=torch.int64, device=dev)
    dH = torch.empty_like(h) if need_dH else None
    dW = torch.empty((V, H), dtype=dW_dtype, device=dev) if need_dW else None
    ws, ws_bytes = _workspace(workspace, _lib.flce_topk_kd_forward_backward_workspace_bytes(N, H, V, t.k, chunk_rows,
                                                                                            _DW[dW_dtype]),
                              stream, dev)
    st = _lib.flce_topk_kd_forward_backward(h, W, t, targets, weights, N, H, V, chunk_rows, ignore_index, transform,
                                            grad_scale, kl, lse, loss, n_valid, dH, dW, _DW[dW_dtype], ws, ws_bytes,
                                            stream)
    _lib.check("flce_topk_kd_forward_backward", st)
    return {"kl": kl, "lse": lse, "loss": loss, "n_valid": n_valid, "dH": dH, "dW": dW}


class TopkDistill(torch.autograd.Function):
    """topk_distill_loss with the logits recomputed in the backward."""

    @staticmethod
    def forward(ctx, h, W, ids, logits, lse_t, targets, weights, tail, chunk_rows, ignore_index, transform):
        ctx.set_materialize_grads(False)  # no zeros for the outputs without a gradient
        out = topk_kd_forward(h, W, ids, logits, lse_t, targets, weights, tail, chunk_rows, ignore_index, transform,
                              skip_ignored=True, for_backward=True)
        ctx.save_for_backward(h, W, out["state"], out["n_valid"])
        ctx.k, ctx.chunk_rows, ctx.transform = ids.shape[1], chunk_rows, transform
        ctx.mark_non_differentiable(out["kl"], out["n_valid"])
        return out["loss"], out["kl"], out["n_valid"]

    @staticmethod
    def backward(ctx, grad_loss, grad_kl, grad_n):
        if grad_loss is None:
            return (None,) * 11
        h, W, state, n_valid = ctx.saved_tensors
        dH, dW = topk_kd_backward(h, W, state, ctx.k, 1.0, ctx.chunk_rows, ctx.transform, ctx.needs_input_grad[0],
                                  ctx.needs_input_grad[1], scale=grad_loss, count=n_valid, dW_dtype=W.dtype)
        return _first_order((dH, dW), (h, W, grad_loss)) + (None,) * 9


class TopkDistillOneCall(torch.autograd.Function):
    """topk_distill_loss with its gradients computed in the forward call; the
    backward only scales them by the incoming gradient of the loss."""

    @staticmethod
    def forward(ctx, h, W, ids, logits, lse_t, targets, weights, tail, chunk_rows, ignore_index, transform):
        ctx.set_materialize_grads(False)  # no zeros for the outputs without a gradient
        out = topk_kd_forward_backward(h, W, ids, logits, lse_t, targets, weights, tail, chunk_rows, ignore_index,
                                       1.0, ctx.needs_input_grad[0], ctx.needs_input_grad[1], transform=transform,
                                       need_lse=False, dW_dtype=W.dtype)
        ctx.grads = (out["dH"], out["dW"])
        ctx.save_for_backward(h, W)  # read under create_graph alone
        ctx.mark_non_differentiable(out["kl"], out["n_valid"])
        return out["loss"], out["kl"], out["n_valid"]

    @staticmethod
    def backward(ctx, grad_loss, grad_kl, grad_n):
        if grad_loss is None:
            return (None,) * 11
        if ctx.grads is None:
            raise RuntimeError("the one-call loss can be differentiated once: its gradients are scaled in place")
        dH, dW = ctx.grads
        ctx.grads = None
        if dH is not None or dW is not None:
            if grad_loss.dtype != torch.float32:
                grad_loss = grad_loss.float()
            _lib.check("flce_scale_grads_bf16", _lib.flce_scale_grads_bf16(
                dH, 0 if dH is None else dH.numel(), dW, 0 if dW is None else dW.numel(), grad_loss))
        if torch.is_grad_enabled():
            dH, dW = _first_order((dH, dW), (*ctx.saved_tensors, grad_loss))
        return (dH, dW) + (None,) * 9


def topk_distill_loss(h, W, ids, logits, lse_t=None, targets=None, weights=None, tail: bool = False,
                      chunk_rows: int = 256, ignore_index: int = IGNORE_INDEX, transform=None,
                      recompute: bool = True):
    """(loss, kl[N], n_valid): the (weighted) mean over the counted rows of
    KL(teacher || student) where the teacher is known by its top logits
    (topk_kd_forward's ids, logits, lse_t and tail).  h and W receive gradients.

    recompute=False computes the gradients in the forward call without the
    logits recompute (faster when chunk_rows >= 2,048; dH and dW are held from
    the forward to the backward).  The backward then multiplies them by the
    incoming gradient, a second rounding where that is no power of two, and a
    pass over them where it is not 1."""
    args = (h, W, ids, logits, lse_t, targets, weights, tail, chunk_rows, ignore_index, transform)
    if not torch.is_grad_enabled() or not (h.requires_grad or W.requires_grad):
        out = topk_kd_forward(*args, skip_ignored=True)
        return out["loss"], out["kl"], out["n_valid"]
    return TopkDistill.apply(*args) if recompute else TopkDistillOneCall.apply(*args)
