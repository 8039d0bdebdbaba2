"""Distillation from top logits: lists whose entries have no mass, or no number
for it."""
import math

import pytest
import torch

import chunked_lm_head_gb300 as flce

from test_topk_gpu import make

pytestmark = pytest.mark.gpu


def grads(c):
    """(dH, dW) of the recomputing backward and of the one-call step."""
    K = c["ids"].shape[1]
    out = flce.topk_kd_forward(c["h"], c["W"], c["ids"], c["logits"], c["lse_t"], for_backward=True)
    two = flce.topk_kd_backward(c["h"], c["W"], out["state"], K, 1.0, count=out["n_valid"])
    one = flce.topk_kd_forward_backward(c["h"], c["W"], c["ids"], c["logits"], c["lse_t"])
    assert torch.equal(torch.isnan(out["kl"]), torch.isnan(one["kl"])) and out["n_valid"] == one["n_valid"]
    return out, (two, (one["dH"], one["dW"]))


def test_a_list_without_mass_beside_an_id_outside_the_vocabulary():
    """The id makes kl NaN; what is left of the list holds nothing, so the row
    takes no part in the gradients."""
    c = make(20, 64, 500, 6, seed=33)
    c["logits"][3] = -math.inf
    c["ids"][3, 2] = 500
    out, both = grads(c)
    assert torch.isnan(out["kl"][3]) and int(torch.isnan(out["kl"]).sum()) == 1
    for dH, dW in both:
        assert not dH[3].any() and torch.isfinite(dH.float()).all() and torch.isfinite(dW).all()


@pytest.mark.parametrize("whole", [False, True])
def test_a_teacher_logit_that_is_not_a_number(whole):
    c = make(20, 64, 500, 6, seed=34, whole=whole)
    c["logits"][4, 1] = float("nan")
    c["logits"][9] = float("nan")
    out, both = grads(c)
    assert torch.isnan(out["kl"][[4, 9]]).all() and int(torch.isnan(out["kl"]).sum()) == 2
    assert int(out["n_valid"]) == 20 and torch.isnan(out["loss"])
