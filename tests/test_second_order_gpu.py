"""The norm's and the distillation's gradients are kernels without a graph: a
second derivative through them is refused, not taken for zero."""
import pytest
import torch

import chunked_lm_head_gb300 as flce

from test_topk_gpu import make

pytestmark = pytest.mark.gpu


def refused(first, x):
    """d/dx of (|first|^2 + a term whose graph is alive)."""
    with pytest.raises(RuntimeError, match="once_differentiable"):
        torch.autograd.grad(first.float().square().sum() + x.float().square().sum(), x)


def test_norm():
    x = torch.randn(8, 64, device="cuda").bfloat16().requires_grad_(True)
    r = torch.randn(8, 64, device="cuda").requires_grad_(True)
    w = torch.ones(64, device="cuda", requires_grad=True)
    g, = torch.autograd.grad(flce.rms_norm(x, w).float().square().sum(), x, create_graph=True)
    refused(g, x)
    y, s = flce.rms_norm(x, w, r)
    g, = torch.autograd.grad(y.float().square().sum() + s.square().sum(), r, create_graph=True)
    refused(g, r)


@pytest.mark.parametrize("recompute", [True, False])
def test_distillation(recompute):
    c = make(40, 64, 500, 6, seed=81)
    h = c["h"].requires_grad_(True)
    loss, _, _ = flce.topk_distill_loss(h, c["W"], c["ids"], c["logits"], recompute=recompute)
    g, = torch.autograd.grad(loss, h, create_graph=True)
    refused(g, h)
    # a first derivative is as before
    loss, _, _ = flce.topk_distill_loss(h, c["W"], c["ids"], c["logits"], recompute=recompute)
    assert torch.equal(torch.autograd.grad(loss, h)[0], g)
