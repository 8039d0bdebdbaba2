"""The root-mean-square norm in front of the LM head, from PyTorch.

``rms_norm`` normalises x, or the residual stream with x added to it, and is
differentiable; ``rms_norm_e4m3`` gives the e4m3 operands of the e4m3 head
(``flce_forward_e4m3``) instead.  Every arithmetic step runs in libflce's CUDA
kernels (include/flce.h states the formulas); this module checks tensor
properties, allocates outputs and passes pointers.
"""
from __future__ import annotations

import torch

from . import _lib
from .api import _first_order

_TYPES = {torch.bfloat16: _lib.DTYPES["bf16"], torch.float32: _lib.DTYPES["f32"]}


def _rows(x, name):
    """Row stride of a 2-D tensor with contiguous rows."""
    if x.dim() != 2 or (x.shape[1] > 1 and x.stride(1) != 1):
        raise ValueError(f"{name} must be 2-D with contiguous rows")
    # a single row's stride is never stepped over (and may be anything)
    return x.stride(0) if x.shape[0] > 1 else x.shape[1]


def _check(x, weight, residual):
    if not (x.is_cuda and weight.is_cuda) or (residual is not None and not residual.is_cuda):
        raise ValueError("x, weight and residual must be CUDA tensors")
    if x.dtype != torch.bfloat16:
        raise ValueError("x must be bfloat16")
    if weight.dtype not in _TYPES or (residual is not None and residual.dtype not in _TYPES):
        raise ValueError("weight and residual must be bfloat16 or float32")
    ldx = _rows(x, "x")
    if weight.shape != (x.shape[1],) or not weight.is_contiguous():
        raise ValueError("expected x[N,H] and a contiguous weight[H]")
    ldr = 0
    if residual is not None:
        if residual.shape != x.shape:
            raise ValueError("residual must have x's shape")
        ldr = _rows(residual, "residual")
    return ldx, ldr


def _norm(x, weight, residual, eps, weight_offset, need_rstd, stream):
    """(y, stream or None, rstd or None)"""
    ldx, ldr = _check(x, weight, residual)
    N, H = x.shape
    y = torch.empty_like(x)  # contiguous, also for rows out of a wider buffer
    s = None if residual is None else torch.empty_like(residual)
    rstd = torch.empty(N, dtype=torch.float32, device=x.device) if need_rstd else None
    _lib.check("flce_rms_norm", _lib.flce_rms_norm(
        x, ldx, residual, ldr, 0 if residual is None else _TYPES[residual.dtype], weight, _TYPES[weight.dtype],
        weight_offset, eps, N, H, y, s, rstd, stream))
    return y, s, rstd


def rms_norm_forward(x, weight, residual=None, eps: float = 1e-6, weight_offset: float = 0.0, stream=None,
                     need_rstd: bool = True):
    """dict(y[N,H] bf16, residual[N,H] or None, rstd[N] f32) on device.

    The stream s = round(x + residual) comes back as ``residual``, in the
    residual's type; y = s rstd (weight + weight_offset)."""
    y, s, rstd = _norm(x, weight, residual, eps, weight_offset, need_rstd, stream)
    return {"y": y, "residual": s, "rstd": rstd}


def rms_norm_e4m3(x, weight, residual=None, eps: float = 1e-6, weight_offset: float = 0.0, stream=None,
                  need_rstd: bool = False):
    """dict(q[N,H] float8_e4m3fn, scale[N] f32, residual[N,H] or None, rstd[N] f32
    or None) on device: y of rms_norm quantised per row from its 32-bit value,
    with q * scale[:, None] = y up to e4m3's rounding.  The operand form of
    flce_forward_e4m3; not differentiable."""
    ldx, ldr = _check(x, weight, residual)
    N, H = x.shape
    q = torch.empty_like(x, dtype=torch.float8_e4m3fn)
    scale = torch.empty(N, dtype=torch.float32, device=x.device)
    s = None if residual is None else torch.empty_like(residual)
    rstd = torch.empty_like(scale) if need_rstd else None
    _lib.check("flce_rms_norm_e4m3", _lib.flce_rms_norm_e4m3(
        x, ldx, residual, ldr, 0 if residual is None else _TYPES[residual.dtype], weight, _TYPES[weight.dtype],
        weight_offset, eps, N, H, q, scale, s, rstd, stream))
    return {"q": q, "scale": scale, "residual": s, "rstd": rstd}


def _norm_grads(dy, s, lds, weight, rstd, ds, weight_offset, need_dx, need_dr, need_dweight, workspace, stream):
    """(dx, dr, dweight) of checked tensors."""
    N, H = s.shape
    wide = s.dtype == torch.float32
    dx = torch.empty_like(dy) if need_dx or (need_dr and not wide) else None
    dr = torch.empty_like(s, memory_format=torch.contiguous_format) if need_dr and wide else None
    dw = None
    if need_dweight:
        dw = torch.empty_like(weight)
        if workspace is None and stream is None:  # torch's allocator keeps it for the next call
            workspace = torch.empty(_lib.flce_rms_norm_backward_workspace_bytes(N, H), dtype=torch.uint8,
                                    device=s.device)
    elif dx is None and dr is None:
        return None, None, None
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _lib.check("flce_rms_norm_backward", _lib.flce_rms_norm_backward(
        dy, s, lds, _TYPES[s.dtype], ds, weight, _TYPES[weight.dtype], weight_offset, rstd, N, H, dx, dr, dw,
        workspace, ws_bytes, stream))
    return dx if need_dx else None, (dr if wide else dx) if need_dr else None, dw


def rms_norm_backward(dy, s, weight, rstd, ds=None, weight_offset: float = 0.0, need_dx: bool = True,
                      need_dr: bool = True, need_dweight: bool = True, workspace: torch.Tensor | None = None,
                      stream=None):
    """(dx[N,H] bf16, dr[N,H] of s's type, dweight[H]) of rms_norm, each None
    where not needed.  s: the stream that was normed; ds: the gradient that
    reaches it past the norm, or None.  For a bf16 stream dx and dr are one
    tensor."""
    _, lds = _check(dy, weight, s)
    if rstd.dtype != torch.float32 or rstd.shape != (s.shape[0],) or not rstd.is_contiguous() or not rstd.is_cuda:
        raise ValueError("rstd must be a contiguous float32 [N] CUDA tensor")
    if not dy.is_contiguous():
        raise ValueError("dy must be contiguous")
    if ds is not None and (not ds.is_cuda or ds.dtype != s.dtype or ds.shape != s.shape or not ds.is_contiguous()):
        raise ValueError("ds must be a contiguous CUDA tensor of s's shape and type")
    if workspace is not None and not workspace.is_cuda:
        raise ValueError("workspace must be a CUDA tensor")
    return _norm_grads(dy, s, lds, weight, rstd, ds, weight_offset, need_dx, need_dr, need_dweight, workspace, stream)


def _rows_of(g):
    """A gradient as the kernels read it: contiguous, from a 16-byte boundary on
    (a part of a flat buffer may start anywhere)."""
    g = g.contiguous()
    return g if g.data_ptr() % 16 == 0 else g.clone()


class RMSNormFunction(torch.autograd.Function):
    """rms_norm with its backward; the stream is returned beside y."""

    @staticmethod
    def forward(ctx, x, weight, residual, eps, weight_offset):
        ctx.set_materialize_grads(False)
        y, s, rstd = _norm(x, weight, residual, eps, weight_offset, True, None)
        ctx.save_for_backward(x if s is None else s, weight, rstd)
        ctx.weight_offset = weight_offset
        return y if s is None else (y, s)

    @staticmethod
    def backward(ctx, dy, ds=None):
        s, weight, rstd = ctx.saved_tensors
        need_x, need_w, need_r = ctx.needs_input_grad[:3]
        if dy is None:  # only the stream was used
            if ds is None:
                return None, None, None, None, None
            return ds.to(torch.bfloat16) if need_x else None, None, ds if need_r else None, None, None
        dx, dr, dw = _norm_grads(_rows_of(dy), s, s.stride(0) if s.shape[0] > 1 else s.shape[1], weight, rstd,
                                 None if ds is None else _rows_of(ds), ctx.weight_offset, need_x, need_r, need_w,
                                 None, None)
        dx, dw, dr = _first_order((dx, dw, dr), (s, weight, dy, ds))
        return dx, dw, dr, None, None


def rms_norm(x, weight, residual=None, eps: float = 1e-6, weight_offset: float = 0.0):
    """y, or (y, stream) with a residual: the stream s = round(x + residual) in
    the residual's type, y = s (mean(s^2) + eps)^(-1/2) (weight + weight_offset)
    in bf16.  x [N,H] bf16; residual [N,H] and weight [H] bf16 or fp32;
    differentiable in all three."""
    if torch.is_grad_enabled() and (x.requires_grad or weight.requires_grad or
                                    (residual is not None and residual.requires_grad)):
        return RMSNormFunction.apply(x, weight, residual, eps, weight_offset)
    y, s, _ = _norm(x, weight, residual, eps, weight_offset, False, None)
    return y if s is None else (y, s)


class RMSNorm(torch.nn.Module):
    """Module form of rms_norm: forward(x, residual=None)."""

    def __init__(self, hidden_size: int, eps: float = 1e-6, weight_offset: float = 0.0, dtype=torch.bfloat16,
                 device=None):
        super().__init__()
        self.eps, self.weight_offset = eps, weight_offset
        self.weight = torch.nn.Parameter(torch.full((hidden_size,), 1.0 - weight_offset, dtype=dtype, device=device))

    def forward(self, x, residual=None):
        return rms_norm(x, self.weight, residual, self.eps, self.weight_offset)
