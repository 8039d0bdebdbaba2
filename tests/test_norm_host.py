"""The norm's argument checks: refused on the host, before any launch."""
import pytest
import torch

import chunked_lm_head_gb300 as flce
from chunked_lm_head_gb300 import _lib

P = 1 << 20  # a non-null, aligned value; never dereferenced on these paths
BF16, F32 = _lib.DTYPES["bf16"], _lib.DTYPES["f32"]
OK, INVALID, UNSUPPORTED = 0, 1, 3


def norm(x=P, ldx=64, r=None, ldr=0, rt=BF16, w=P, wt=BF16, off=0.0, eps=1e-6, N=4, H=64, y=P, s=None, rstd=None):
    return _lib.flce_rms_norm(x, ldx, r, ldr, rt, w, wt, off, eps, N, H, y, s, rstd, 0)


def norm8(x=P, ldx=64, r=None, ldr=0, rt=BF16, w=P, wt=BF16, off=0.0, eps=1e-6, N=4, H=64, q=P, sc=P, s=None):
    return _lib.flce_rms_norm_e4m3(x, ldx, r, ldr, rt, w, wt, off, eps, N, H, q, sc, s, None, 0)


def back(dy=P, s=P, lds=64, st=BF16, ds=None, w=P, wt=BF16, off=0.0, rstd=P, N=4, H=64, dx=P, dr=None, dw=P,
         ws=None, wb=0):
    return _lib.flce_rms_norm_backward(dy, s, lds, st, ds, w, wt, off, rstd, N, H, dx, dr, dw, ws, wb, 0)


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(y=None), INVALID), (dict(N=-1), INVALID),
    (dict(H=0), INVALID), (dict(ldx=56), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(off=float("inf")), INVALID), (dict(wt=2), INVALID), (dict(r=P, ldr=64, s=P, rt=4), INVALID),
    (dict(r=P, ldr=64), INVALID), (dict(s=P), INVALID), (dict(r=P, ldr=8, s=P), INVALID),
    (dict(N=1 << 31), INVALID),
    (dict(H=60), UNSUPPORTED), (dict(H=32776, ldx=32776), UNSUPPORTED), (dict(ldx=68), UNSUPPORTED),
    (dict(x=P + 2), UNSUPPORTED), (dict(w=P + 4), UNSUPPORTED), (dict(y=P + 8), UNSUPPORTED),
    (dict(r=P + 2, ldr=64, s=P), UNSUPPORTED), (dict(r=P, ldr=68, s=P), UNSUPPORTED),
    (dict(r=P, ldr=66, rt=F32, s=P), UNSUPPORTED), (dict(rstd=P + 2), UNSUPPORTED),
    (dict(N=0), OK), (dict(N=0, x=None, w=None, y=None), OK),
])
def test_norm_refusals(kw, want):
    assert norm(**kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), INVALID), (dict(sc=None), INVALID), (dict(H=72, ldx=72), UNSUPPORTED),
    (dict(q=P + 8), UNSUPPORTED), (dict(sc=P + 1), UNSUPPORTED), (dict(N=0), OK),
])
def test_norm_e4m3_refusals(kw, want):
    assert norm8(**kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(dy=None), INVALID), (dict(s=None), INVALID), (dict(w=None), INVALID), (dict(rstd=None), INVALID),
    (dict(dx=None, dw=None), INVALID), (dict(N=-1), INVALID), (dict(lds=8), INVALID), (dict(st=3), INVALID),
    (dict(wt=-1), INVALID), (dict(off=float("nan")), INVALID),
    (dict(H=68, lds=72), UNSUPPORTED), (dict(H=1 << 16, lds=1 << 16), UNSUPPORTED), (dict(lds=66), UNSUPPORTED),
    (dict(dy=P + 4), UNSUPPORTED), (dict(s=P + 8), UNSUPPORTED), (dict(dr=P + 4), UNSUPPORTED),
    (dict(dw=P + 2), UNSUPPORTED), (dict(ds=P + 2), UNSUPPORTED),
    (dict(ws=P, wb=16), INVALID), (dict(ws=P + 8, wb=1 << 30), INVALID),  # too small, misaligned
    (dict(N=0, dw=None), OK),
])
def test_norm_backward_refusals(kw, want):
    assert back(**kw) == want


def test_workspace_grows_with_the_row_slots_only():
    f = _lib.flce_rms_norm_backward_workspace_bytes
    assert f(-1, 64) == 0 and f(4, 0) == 0
    assert f(1, 4096) >= 4096 * 4
    assert f(1 << 20, 4096) == f(1 << 24, 4096) <= 64 << 20


def test_torch_checks_refuse_what_the_kernels_do_not_take():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.ones(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        flce.rms_norm(x, w)
    with pytest.raises(ValueError, match="CUDA"):
        flce.rms_norm_e4m3(x, w, x)
    m = flce.RMSNorm(64, weight_offset=1.0)
    assert m.weight.dtype == torch.bfloat16 and not bool(m.weight.detach().any())
