"""The layer norm's argument checks: refused on the host, before any launch."""
import pytest
import torch

import chunked_lm_head_gb300 as flce
from chunked_lm_head_gb300 import _lib

import layer_ref as R

P = 1 << 20  # a non-null, aligned value; never dereferenced on these paths
BF16, F32 = _lib.DTYPES["bf16"], _lib.DTYPES["f32"]
OK, INVALID, UNSUPPORTED = 0, 1, 3


def norm(x=P, ldx=64, r=None, ldr=0, rt=BF16, w=P, b=P, wt=BF16, off=0.0, eps=1e-6, N=4, H=64, y=P, s=None, mean=None,
         rstd=None):
    return _lib.flce_layer_norm(x, ldx, r, ldr, rt, w, b, wt, off, eps, N, H, y, s, mean, rstd, 0)


def back(dy=P, s=P, lds=64, st=BF16, ds=None, w=P, wt=BF16, off=0.0, mean=P, rstd=P, N=4, H=64, dx=P, dr=None, dw=P,
         db=P, ws=None, wb=0):
    return _lib.flce_layer_norm_backward(dy, s, lds, st, ds, w, wt, off, mean, rstd, N, H, dx, dr, dw, db, ws, wb, 0)


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(y=None), INVALID), (dict(N=-1), INVALID),
    (dict(H=0), INVALID), (dict(ldx=56), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(off=float("inf")), INVALID), (dict(wt=2), INVALID), (dict(r=P, ldr=64, s=P, rt=4), INVALID),
    (dict(r=P, ldr=64), INVALID), (dict(s=P), INVALID), (dict(r=P, ldr=8, s=P), INVALID), (dict(N=1 << 31), INVALID),
    (dict(N=(1 << 31) - 65536), INVALID),
    (dict(H=60), UNSUPPORTED), (dict(H=32776, ldx=32776), UNSUPPORTED), (dict(ldx=68), UNSUPPORTED),
    (dict(x=P + 2), UNSUPPORTED), (dict(w=P + 4), UNSUPPORTED), (dict(b=P + 8), UNSUPPORTED),
    (dict(y=P + 8), UNSUPPORTED), (dict(r=P + 2, ldr=64, s=P), UNSUPPORTED), (dict(r=P, ldr=68, s=P), UNSUPPORTED),
    (dict(r=P, ldr=66, rt=F32, s=P), UNSUPPORTED), (dict(rstd=P + 2), UNSUPPORTED), (dict(mean=P + 1), UNSUPPORTED),
    (dict(N=0), OK), (dict(N=0, x=None, w=None, y=None, b=None), OK),
])
def test_norm_refusals(kw, want):
    assert norm(**kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(dy=None), INVALID), (dict(s=None), INVALID), (dict(w=None), INVALID), (dict(rstd=None), INVALID),
    (dict(mean=None), INVALID), (dict(dx=None, dw=None, db=None), INVALID), (dict(N=-1), INVALID),
    (dict(lds=8), INVALID), (dict(st=3), INVALID), (dict(wt=-1), INVALID), (dict(off=float("nan")), INVALID),
    (dict(H=68, lds=72), UNSUPPORTED), (dict(H=1 << 16, lds=1 << 16), UNSUPPORTED), (dict(lds=66), UNSUPPORTED),
    (dict(dy=P + 4), UNSUPPORTED), (dict(s=P + 8), UNSUPPORTED), (dict(dr=P + 4), UNSUPPORTED),
    (dict(dw=P + 2), UNSUPPORTED), (dict(db=P + 4), UNSUPPORTED), (dict(ds=P + 2), UNSUPPORTED),
    (dict(mean=P + 2), UNSUPPORTED),
    (dict(ws=P, wb=16), INVALID), (dict(ws=P + 8, wb=1 << 30), INVALID),  # too small, misaligned
    (dict(N=0, dw=None, db=None), OK),
])
def test_norm_backward_refusals(kw, want):
    assert back(**kw) == want


def test_workspace_grows_with_the_row_slots_only():
    f = _lib.flce_layer_norm_backward_workspace_bytes
    assert f(-1, 64) == 0 and f(4, 0) == 0
    assert f(1, 4096) >= 2 * 4096 * 4
    assert f(1 << 20, 4096) == f(1 << 24, 4096) <= 64 << 20


def test_torch_checks_refuse_what_the_kernels_do_not_take():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.ones(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        flce.layer_norm(x, w)
    m = flce.LayerNorm(64, weight_offset=1.0)
    assert m.weight.dtype == torch.bfloat16 and not bool(m.weight.detach().any()) and not bool(m.bias.detach().any())


def test_reference_gradient_matches_differences():
    """The reference's gradients against central differences of its forward, in 64 bits."""
    g = torch.Generator().manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    s, w, b, dy, ds = rnd(4, 24) + 2, rnd(24), rnd(24), rnd(4, 24), rnd(4, 24)
    d, dw, db = R.backward(dy, ds, s, w, 1e-5, 1.0)
    e = 1e-6

    def loss(s, w, b):
        return (R.forward(s, w, b, 1e-5, 1.0)[0] * dy).sum() + (s * ds).sum()

    for _ in range(4):
        vs, vw, vb = rnd(4, 24), rnd(24), rnd(24)
        diff = (loss(s + e * vs, w + e * vw, b + e * vb) - loss(s - e * vs, w - e * vw, b - e * vb)) / (2 * e)
        assert torch.allclose((d * vs).sum() + (dw * vw).sum() + (db * vb).sum(), diff, rtol=1e-6, atol=1e-7)
