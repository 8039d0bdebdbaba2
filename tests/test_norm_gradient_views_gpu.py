"""Gradients that reach the norm as parts of flat buffers."""
import pytest
import torch

import chunked_lm_head_gb300 as flce

from test_norm_gpu import BF16, F32, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("residual", [None, BF16, F32], ids=["none", "bf16", "f32"])
def test_gradients_off_a_16_byte_boundary(residual):
    """What autograd hands back for a part of a flat buffer is contiguous, and
    starts anywhere."""
    N, H = 6, 72
    x, r, w, rnd = make(N, H, residual, BF16, 0.0)
    for v in (x, r, w):
        if v is not None:
            v.requires_grad_(True)
    ins = [v for v in (x, r, w) if v is not None]
    outs = flce.rms_norm(x, w, r)
    outs = [outs] if r is None else list(outs)
    pads = [torch.zeros(3, dtype=o.dtype, device="cuda", requires_grad=True) for o in outs]
    flat = [torch.cat([p, o.reshape(-1)]) for p, o in zip(pads, outs)]
    ups = [rnd(3 + N * H).to(o.dtype) for o in outs]
    got = torch.autograd.grad(flat, ins, ups)
    outs = flce.rms_norm(x, w, r)
    outs = [outs] if r is None else list(outs)
    want = torch.autograd.grad(outs, ins, [u[3:].reshape(N, H).clone() for u in ups])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
