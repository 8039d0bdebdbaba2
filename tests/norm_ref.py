"""The norm's definition in 64 bits, and the rounding bounds its tests use."""
import torch

EPS24 = 2.0 ** -24  # half a step of fp32, relative


def stream(x, residual):
    """s as it is stored: x, or x + residual rounded to the residual's type
    (the fp32 sum of two bf16 or fp32 values, then the type)."""
    return x if residual is None else (x.float() + residual.float()).to(residual.dtype)


def forward(s, weight, eps, offset):
    """(y, rstd) in 64 bits of the stream s."""
    sd = s.double()
    rstd = (sd.square().mean(1) + eps) ** -0.5
    return sd * rstd[:, None] * (weight.double() + offset), rstd


def backward(dy, ds, s, weight, eps, offset):
    """(d, dweight) in 64 bits: the stream's gradient and the weight's."""
    sd, dyd = s.double(), dy.double()
    rstd = ((sd.square().mean(1) + eps) ** -0.5)[:, None]
    g = dyd * (weight.double() + offset)
    d = rstd * g - sd * rstd ** 3 * (g * sd).mean(1, keepdim=True)
    if ds is not None:
        d = d + ds.double()
    return d, (dyd * sd * rstd).sum(0)


def half_step(t):
    """Half a rounding step relative to the value: bf16 2^-8, fp32 2^-24, e4m3 2^-4."""
    return torch.finfo(t).eps / 2
