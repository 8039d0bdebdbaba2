"""The layer norm in front of the LM head, from PyTorch: ``layer_norm`` normalises
x, or the residual stream with x added to it, and is differentiable.  Every
arithmetic step runs in libflce's CUDA kernels (include/flce.h states the
formulas); this module checks tensor properties, allocates outputs and passes
pointers (``layer_norm`` leaves the last two to csrc/torch_ops.cpp).
"""
from __future__ import annotations

import torch

from . import _lib
from .norm import _TYPES, _check
from .score import _elsewhere


def _check_all(x, weight, bias, residual):
    ld = _check(x, weight, residual)
    if bias is not None and (bias.dtype != weight.dtype or bias.shape != weight.shape or not bias.is_contiguous()):
        raise ValueError("bias must be contiguous, of weight's shape and type")
    dev = x.get_device()
    if weight.get_device() != dev or (bias is not None and bias.get_device() != dev) or (
            residual is not None and residual.get_device() != dev):
        raise ValueError("x, weight, bias and residual must be on one device")
    return ld


def layer_norm_forward(x, weight, bias=None, residual=None, eps: float = 1e-5, weight_offset: float = 0.0, stream=None,
                       need_stats: bool = True):
    """dict(y[N,H] bf16, residual[N,H] or None, mean[N], rstd[N] f32 or None) on
    device.  The stream s = round(x + residual) comes back as ``residual``, in the
    residual's type; y = (s - mean) rstd (weight + weight_offset) + bias."""
    ldx, ldr = _check_all(x, weight, bias, residual)
    if _elsewhere(x):
        with torch.cuda.device(x.device):
            return layer_norm_forward(x, weight, bias, residual, eps, weight_offset, stream, need_stats)
    N, H = x.shape
    y = torch.empty_like(x)  # contiguous, also for rows out of a wider buffer
    s = None if residual is None else torch.empty_like(residual)
    mean = rstd = None
    if need_stats:
        mean, rstd = torch.empty((2, N), dtype=torch.float32, device=x.device).unbind(0)
    _lib.check("flce_layer_norm", _lib.flce_layer_norm(
        x, ldx, residual, ldr, 0 if residual is None else _TYPES[residual.dtype], weight, bias, _TYPES[weight.dtype],
        weight_offset, eps, N, H, y, s, mean, rstd, stream))
    return {"y": y, "residual": s, "mean": mean, "rstd": rstd}


def layer_norm_backward(dy, s, weight, mean, rstd, ds=None, weight_offset: float = 0.0, need_dx: bool = True,
                        need_dr: bool = True, need_dweight: bool = True, need_dbias: bool = True,
                        workspace: torch.Tensor | None = None, stream=None):
    """(dx[N,H] bf16, dr[N,H] of s's type, dweight[H], dbias[H]) of layer_norm, each
    None where not needed.  s: the stream that was normed; ds: the gradient that
    reaches it past the norm, or None.  For a bf16 stream dx and dr are one
    tensor."""
    _, lds = _check_all(dy, weight, None, s)
    for x, name in ((mean, "mean"), (rstd, "rstd")):
        if x.dtype != torch.float32 or x.shape != (s.shape[0],) or not x.is_contiguous() or x.device != s.device:
            raise ValueError(f"{name} must be a contiguous float32 [N] CUDA tensor")
    if not dy.is_contiguous():
        raise ValueError("dy must be contiguous")
    if ds is not None and (ds.device != s.device or ds.dtype != s.dtype or ds.shape != s.shape or
                           not ds.is_contiguous()):
        raise ValueError("ds must be a contiguous CUDA tensor of s's shape and type")
    if workspace is not None and workspace.device != s.device:
        raise ValueError("workspace must be a CUDA tensor")
    if _elsewhere(s):
        with torch.cuda.device(s.device):
            return layer_norm_backward(dy, s, weight, mean, rstd, ds, weight_offset, need_dx, need_dr, need_dweight,
                                       need_dbias, workspace, stream)
    N, H = s.shape
    wide = s.dtype == torch.float32
    dx = torch.empty_like(dy) if need_dx or (need_dr and not wide) else None
    dr = torch.empty_like(s, memory_format=torch.contiguous_format) if need_dr and wide else None
    dw = torch.empty_like(weight) if need_dweight else None
    db = torch.empty_like(weight) if need_dbias else None
    ws_bytes = 0
    if need_dweight or need_dbias:
        if workspace is None and stream is None:  # torch's allocator keeps it for the next call
            workspace = torch.empty(_lib.flce_layer_norm_backward_workspace_bytes(N, H), dtype=torch.uint8,
                                    device=s.device)
        if workspace is not None:
            ws_bytes = workspace.numel() * workspace.element_size()
    elif dx is None and dr is None:
        return None, None, None, None
    _lib.check("flce_layer_norm_backward", _lib.flce_layer_norm_backward(
        dy, s, lds, _TYPES[s.dtype], ds, weight, _TYPES[weight.dtype], weight_offset, mean, rstd, N, H, dx, dr, dw, db,
        workspace, ws_bytes, stream))
    return dx if need_dx else None, (dr if wide else dx) if need_dr else None, dw, db


def layer_norm(x, weight, bias=None, residual=None, eps: float = 1e-5, weight_offset: float = 0.0):
    """y, or (y, stream) with a residual: the stream s = round(x + residual) in the
    residual's type, y = (s - mean(s)) (var(s) + eps)^(-1/2) (weight +
    weight_offset) + bias in bf16.  x [N,H] bf16; residual [N,H] bf16 or fp32;
    weight and bias [H] of one type, bf16 or fp32; differentiable in all four.

    Captured into a CUDA graph, a call whose leaves an eager graph still holds is
    refused: PyTorch's backward could not be captured beside it."""
    _check_all(x, weight, bias, residual)
    if _elsewhere(x):
        with torch.cuda.device(x.device):
            return layer_norm(x, weight, bias, residual, eps, weight_offset)
    try:
        out = (_lib._TORCH_OPS or _lib.torch_ops())[0](x, weight, bias, residual, eps, weight_offset)
    except RuntimeError as e:
        raise _lib.torch_error(e) from None
    return out[0] if residual is None else tuple(out)


class LayerNorm(torch.nn.Module):
    """Module form of layer_norm: forward(x, residual=None)."""

    def __init__(self, hidden_size: int, eps: float = 1e-5, bias: bool = True, weight_offset: float = 0.0,
                 dtype=torch.bfloat16, device=None):
        super().__init__()
        self.eps, self.weight_offset = eps, weight_offset
        self.weight = torch.nn.Parameter(torch.full((hidden_size,), 1.0 - weight_offset, dtype=dtype, device=device))
        self.bias = torch.nn.Parameter(torch.zeros(hidden_size, dtype=dtype, device=device)) if bias else None

    def forward(self, x, residual=None):
        return layer_norm(x, self.weight, self.bias, residual, self.eps, self.weight_offset)
