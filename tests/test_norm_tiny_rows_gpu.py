"""The e4m3 norm's rows of tiny values, whose factor 448 / max|s gain| is past
fp32 although y / scale is not."""
import pytest
import torch

import chunked_lm_head_gb300 as flce

import norm_ref as R
from test_norm_gpu import BF16, E4M3, F32, FP32, assert_within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("residual", [None, BF16, F32], ids=["none", "bf16", "f32"])
@pytest.mark.parametrize("H", [64, 512, 2560, 4096, 8192, 16400])
def test_e4m3_rows_of_tiny_values(H, residual):
    """Rows whose largest value is down to 2^-126, bf16's smallest normal one."""
    N = 6
    g = torch.Generator(device="cuda").manual_seed(71 + H)
    x = torch.randn(N, H, generator=g, device="cuda").clamp(-2, 2)
    x[:, 0] = 2.0
    x[:, 3] = 0.0
    x = (x * 2.0 ** torch.tensor([-127.0, -124.0, -120.0, -118.0, -100.0, 0.0], device="cuda")[:, None]).bfloat16()
    r = None if residual is None else torch.zeros(N, H, dtype=residual, device="cuda")
    w = torch.ones(H, dtype=BF16, device="cuda")
    out = flce.rms_norm_e4m3(x, w, r)
    y, _ = R.forward(x, w, 1e-6, 0.0)
    scale = y.abs().amax(1) / 448
    # scale: roundings as for any row, and half of fp32's smallest step
    assert_within(out["scale"], scale, scale * FP32 + 2.0 ** -150, "scale")
    sc = out["scale"].double()[:, None]
    got = out["q"].float().double()
    assert_within(got, y / sc, torch.maximum((y / sc).abs() * R.half_step(E4M3), torch.full_like(sc, 2.0 ** -10))
                  + (y / sc).abs() * FP32, "q")
    assert not out["q"].float()[:, 3].any()


def test_e4m3_row_below_the_smallest_scale():
    """A scale that rounds to zero counts as that of a row of zeros."""
    x = torch.full((2, 512), 2.0 ** -133, device="cuda").bfloat16()
    w = torch.full((512,), 2.0 ** -12, device="cuda")
    for r in (None, torch.zeros(2, 512, device="cuda")):
        out = flce.rms_norm_e4m3(x, w, r, eps=1.0)
        assert bool((out["scale"] == 1).all()) and not out["q"].float().any()
