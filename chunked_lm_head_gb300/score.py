"""Scores of the LM head's distribution softmax(f(h W^T)), from PyTorch.

``selective_log_softmax_entropy`` gives the log-probability of each row's target
and the entropy, differentiable in both; ``top_logprobs`` the K likeliest words
of each row with their log-probabilities.  ``score_forward`` and
``score_backward`` are the calls below them.  Every arithmetic step runs in
libflce's CUDA kernels (include/flce.h states the formulas); this module checks
tensor properties, allocates outputs and passes pointers (the first two calls leave
the last two to csrc/torch_ops.cpp).
"""
from __future__ import annotations

import torch

from . import _lib
from .api import IGNORE_INDEX
from .topk import _DW, _workspace


def _elsewhere(x):
    """Whether x is on another CUDA device than the current one (whose streams and
    launches a call would take)."""
    return x.is_cuda and x.get_device() != torch._C._cuda_getDevice()


def _check(h, W, targets):
    for x in (h, W):
        if not x.is_cuda or x.dtype != torch.bfloat16 or x.dim() != 2 or not x.is_contiguous():
            raise ValueError("h and W must be contiguous 2-D bfloat16 CUDA tensors")
    if W.shape[1] != h.shape[1] or W.get_device() != h.get_device():
        raise ValueError("expected h[N,H] and W[V,H] on one device")
    if targets is not None and (targets.dtype != torch.int64 or targets.shape != (h.shape[0],) or
                                targets.get_device() != h.get_device() or not targets.is_contiguous()):
        raise ValueError("targets must be a contiguous int64 [N] tensor on h's device")


def _row_vector(x, h, name):
    if x is not None and (x.dtype != torch.float32 or x.shape != (h.shape[0],) or
                          x.get_device() != h.get_device() or not x.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous float32 [N] tensor on h's device")


def score_forward(h, W, targets=None, k: int = 0, ignore_index: int = IGNORE_INDEX, transform=None,
                  workspace: torch.Tensor | None = None, stream=None, keep_rows: int = 0):
    """dict(logp[N] or None, lse[N], entropy[N] f32, ids[N,k] i64 or None,
    logprobs[N,k] f32 or None, state) on device.

    logp: log-probability of each row's target (None without targets).  k > 0
    (at most 128 and V): the k words of largest logit in descending order, ties
    to the lowest index, and their log-probabilities; the order is that of the
    exact sums h W^T.  A row whose target is ignore_index is skipped: zeros, and
    ids of -1.  A row with a logit that is NaN or +infinity: NaN, ids of -1.
    transform: as in forward().

    keep_rows > 0 (with targets, k = 0): where N fits into as many rows, and it
    pays, state holds the logits in 16 bits (N V 2 bytes) for score_backward,
    which then needs no product again (else None)."""
    _check(h, W, targets)
    (N, H), V, dev = h.shape, W.shape[0], h.device
    if not 0 <= k <= V:
        raise ValueError("k must be between 0 and the vocabulary")
    if keep_rows and (k or targets is None):
        raise ValueError("keep_rows goes with targets and without words")
    if _elsewhere(h):
        with torch.cuda.device(h.device):
            return score_forward(h, W, targets, k, ignore_index, transform, workspace, stream, keep_rows)
    lse = torch.empty(N, dtype=torch.float32, device=dev)
    entropy = torch.empty_like(lse)
    logp = None if targets is None else torch.empty_like(lse)
    ids = torch.empty((N, k), dtype=torch.int64, device=dev) if k else None
    words = torch.empty((N, k), dtype=torch.float32, device=dev) if k else None
    nbytes = _lib.flce_score_state_bytes(N, H, V, keep_rows) if keep_rows else 0
    state = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
    ws, ws_bytes = _workspace(workspace, _lib.flce_score_workspace_bytes(N, H, V, k), stream, dev)
    _lib.check("flce_score", _lib.flce_score(h, W, targets, N, H, V, k, ignore_index, transform, logp, lse, entropy, ids,
                                             words, state, ws, ws_bytes, stream))
    return {"logp": logp, "lse": lse, "entropy": entropy, "ids": ids, "logprobs": words, "state": state}


def score_backward(h, W, targets, lse, entropy, grad_logp=None, grad_entropy=None, chunk_rows: int = 256,
                   ignore_index: int = IGNORE_INDEX, transform=None, need_dH: bool = True, need_dW: bool = True,
                   workspace: torch.Tensor | None = None, stream=None, dW_dtype=torch.float32, state=None):
    """(dH[N,H] bf16 or None, dW[V,H] of dW_dtype (float32 or bfloat16) or None)
    of sum_i grad_logp[i] logp[i] + grad_entropy[i] entropy[i] (either may be
    None: zero), from the forward's lse and entropy, and its state (of the same
    h, W, targets, ignore_index and transform) or the logits recomputed."""
    _check(h, W, targets)
    if targets is None:
        raise ValueError("targets are needed")
    if dW_dtype not in _DW:
        raise ValueError("dW_dtype must be float32 or bfloat16")
    for x, name in ((lse, "lse"), (entropy, "entropy"), (grad_logp, "grad_logp"), (grad_entropy, "grad_entropy")):
        _row_vector(x, h, name)
    (N, H), V, dev = h.shape, W.shape[0], h.device
    if state is not None and (state.device != dev or not state.is_contiguous() or not N or
                              state.numel() * state.element_size() != _lib.flce_score_state_bytes(N, H, V, N)):
        raise ValueError("state must come from score_forward of the same sizes")
    if state is not None:
        chunk_rows = max(chunk_rows, N)  # the kept rows are one block
    if _elsewhere(h):
        with torch.cuda.device(dev):
            return score_backward(h, W, targets, lse, entropy, grad_logp, grad_entropy, chunk_rows, ignore_index,
                                  transform, need_dH, need_dW, workspace, stream, dW_dtype, state)
    dH = torch.empty_like(h) if need_dH else None
    dW = torch.empty((V, H), dtype=dW_dtype, device=dev) if need_dW else None
    ws, ws_bytes = _workspace(workspace, _lib.flce_score_backward_workspace_bytes(N, H, V, chunk_rows, _DW[dW_dtype]),
                              stream, dev)
    _lib.check("flce_score_backward", _lib.flce_score_backward(
        h, W, targets, lse, entropy, grad_logp, grad_entropy, state, dH, dW, _DW[dW_dtype], N, H, V, chunk_rows,
        ignore_index, transform, ws, ws_bytes, stream))
    return dH, dW


def selective_log_softmax_entropy(h, W, targets, chunk_rows: int = 256, ignore_index: int = IGNORE_INDEX,
                                  transform=None, recompute: bool = False):
    """(logp[N], entropy[N]) fp32: log-probability of each row's target and entropy
    (natural units) of softmax(f(h W^T)), both differentiable in h and W; 0 on
    rows whose target is ignore_index.  For policy losses with an entropy term:
    both come out of one pass over the head, and both gradients of another.

    chunk_rows bounds the rows of dlogits that the backward holds.  A call of at
    most that many rows keeps its logits until then, 2 bytes each, and the
    backward saves their product; recompute=True keeps nothing.

    Captured into a CUDA graph, a call whose leaves an eager graph still holds is
    refused: PyTorch's backward could not be captured beside it."""
    if targets is None:
        raise ValueError("targets are needed")
    _check(h, W, targets)
    if _elsewhere(h):
        with torch.cuda.device(h.device):
            return selective_log_softmax_entropy(h, W, targets, chunk_rows, ignore_index, transform, recompute)
    try:
        return tuple((_lib._TORCH_OPS or _lib.torch_ops())[1](h, W, targets, chunk_rows, ignore_index,
                                                             _lib.transform_list(transform), recompute))
    except RuntimeError as e:
        raise _lib.torch_error(e) from None


def top_logprobs(h, W, k: int, targets=None, ignore_index: int = IGNORE_INDEX, transform=None,
                 workspace: torch.Tensor | None = None, stream=None):
    """score_forward with k words, dict(ids, logprobs, lse, entropy, logp): the
    alternatives of a sampled token, or the lists (ids, logprobs, and a log-sum-exp
    of 0) that topk_distill_loss takes of a teacher.  Not differentiable."""
    if k < 1:
        raise ValueError("k must be at least 1")
    if workspace is not None or stream is not None or _elsewhere(h):
        out = score_forward(h, W, targets, k, ignore_index, transform, workspace, stream)
        del out["state"]
        return out
    _check(h, W, targets)
    if k > W.shape[0]:
        raise ValueError("k must be between 0 and the vocabulary")
    try:
        out = (_lib._TORCH_OPS or _lib.torch_ops())[2](h, W, k, targets, ignore_index, _lib.transform_list(transform))
    except RuntimeError as e:
        raise _lib.torch_error(e) from None
    return {"ids": out[0], "logprobs": out[1], "lse": out[2], "entropy": out[3],
            "logp": None if targets is None else out[4]}
