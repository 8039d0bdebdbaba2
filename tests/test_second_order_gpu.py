"""The norm's and the distillation's gradients are kernels without a graph: a
second derivative through them is refused, not taken for zero."""
import pytest
import torch

import chunked_lm_head_gb300 as flce

from test_topk_gpu import make

pytestmark = pytest.mark.gpu


def refused(first, *xs):
    """d/dx of |first|^2 + a term whose graph is alive."""
    for x in xs:
        with pytest.raises(RuntimeError, match="second derivative"):
            torch.autograd.grad(first.float().square().sum() + x.float().square().sum(), x, retain_graph=True)


def test_norm():
    x = torch.randn(8, 64, device="cuda").bfloat16().requires_grad_(True)
    r = torch.randn(8, 64, device="cuda").requires_grad_(True)
    w = torch.ones(64, device="cuda", requires_grad=True)
    g, = torch.autograd.grad(flce.rms_norm(x, w).float().square().sum(), x, create_graph=True)
    refused(g, x, w)
    g, = torch.autograd.grad(flce.rms_norm(x, w), x, torch.ones_like(x), create_graph=True)  # an upstream constant
    refused(g, x, w)
    y, s = flce.rms_norm(x, w, r)
    gr, gw = torch.autograd.grad(y.float().square().sum() + s.square().sum(), (r, w), create_graph=True)
    refused(gr, x, r, w)
    refused(gw, x, r, w)


@pytest.mark.parametrize("recompute", [True, False])
def test_distillation(recompute):
    c = make(40, 64, 500, 6, seed=81)
    h, W = c["h"].requires_grad_(True), c["W"].requires_grad_(True)
    first = []
    for create in (True, False):
        loss, _, _ = flce.topk_distill_loss(h, W, c["ids"], c["logits"], recompute=recompute)
        first.append(torch.autograd.grad(loss, (h, W), create_graph=create))
    refused(first[0][0], h, W)
    refused(first[0][1], h, W)
    assert all(torch.equal(a, b) for a, b in zip(*first))  # a first derivative is as before


def test_the_stream_s_gradient_alone_keeps_its_graph():
    """No kernel ran: the stream's gradient passes through."""
    x = torch.randn(8, 64, device="cuda").bfloat16().requires_grad_(True)
    r = torch.randn(8, 64, device="cuda").requires_grad_(True)
    _, s = flce.rms_norm(x, torch.ones(64, device="cuda"), r)
    g, = torch.autograd.grad(s.square().sum(), r, create_graph=True)
    gg, = torch.autograd.grad(g.sum(), r)
    assert torch.equal(gg, torch.full_like(r, 2.0))
