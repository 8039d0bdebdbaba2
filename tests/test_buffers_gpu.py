"""The public calls refuse a state or a workspace of the host."""
import pytest
import torch

import chunked_lm_head_gb300 as flce

from test_topk_gpu import make

pytestmark = pytest.mark.gpu


def test_host_buffers_are_refused():
    c = make(8, 64, 300, 4, seed=91)
    args = (c["h"], c["W"], c["ids"], c["logits"])
    out = flce.topk_kd_forward(*args, for_backward=True)
    host = torch.zeros(1 << 24, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        flce.topk_kd_backward(c["h"], c["W"], out["state"].cpu(), 4, 1.0)
    for call in (lambda: flce.topk_kd_forward(*args, workspace=host),
                 lambda: flce.topk_kd_forward_backward(*args, workspace=host),
                 lambda: flce.topk_kd_backward(c["h"], c["W"], out["state"], 4, 1.0, workspace=host)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    x, w = c["h"], torch.ones(64, device="cuda")
    n = flce.rms_norm_forward(x, w)
    with pytest.raises(ValueError, match="CUDA"):
        flce.rms_norm_backward(torch.ones_like(x), x, w, n["rstd"], workspace=host)
