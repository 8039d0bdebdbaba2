"""The layer norm's definition in 64 bits, and the rounding bounds its tests use."""
import torch

from norm_ref import EPS24, half_step, stream  # noqa: F401

# fp32 roundings along one value: two sums over the row (at most 32 terms in a
# thread, then at most 11 joins each), mean, variance, root and reciprocal, the
# products: under 2^7 half steps
FP32 = 2 ** 7 * EPS24


def stats(s, eps):
    sd = s.double()
    mean = sd.mean(1, keepdim=True)
    rstd = ((sd - mean).square().mean(1, keepdim=True) + eps) ** -0.5
    return sd, mean, rstd


def size(s, eps):
    """What a rounding of n = (s - mean) rstd is relative to: n itself, and the
    mean, whose sum's rounding is that of the row's magnitudes."""
    sd, mean, rstd = stats(s, eps)
    return ((sd - mean) * rstd).abs() + rstd * sd.abs().mean(1, keepdim=True) + rstd * EPS24 / FP32 * sd.abs()


def forward(s, weight, bias, eps, offset):
    """(y, mean, rstd) in 64 bits of the stream s."""
    sd, mean, rstd = stats(s, eps)
    y = (sd - mean) * rstd * (weight.double() + offset)
    return y if bias is None else y + bias.double(), mean[:, 0], rstd[:, 0]


def forward_bound(s, weight, bias, eps, offset):
    b = size(s, eps) * (weight.double() + offset).abs()
    return FP32 * (b if bias is None else b + bias.double().abs())


def backward(dy, ds, s, weight, eps, offset):
    """(d, dweight, dbias) in 64 bits: the stream's gradient and the parameters'."""
    sd, mean, rstd = stats(s, eps)
    n, dyd = (sd - mean) * rstd, dy.double()
    g = dyd * (weight.double() + offset)
    d = rstd * (g - g.mean(1, keepdim=True) - n * (g * n).mean(1, keepdim=True))
    if ds is not None:
        d = d + ds.double()
    return d, (dyd * n).sum(0), dyd.sum(0)


def backward_bounds(dy, ds, s, weight, eps, offset):
    """fp32 roundings of (d, dweight, dbias): of each term's magnitude."""
    _, _, rstd = stats(s, eps)
    n, dyd = size(s, eps), dy.double().abs()
    g = dyd * (weight.double() + offset).abs()
    b = rstd * (g + g.mean(1, keepdim=True) + n * (g * n).mean(1, keepdim=True))
    if ds is not None:
        b = b + ds.double().abs()
    return FP32 * b, 2 * FP32 * (dyd * n).sum(0), 2 * FP32 * dyd.sum(0)
