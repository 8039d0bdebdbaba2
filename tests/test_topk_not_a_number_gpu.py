"""Distillation from top logits: logits that are not numbers reach the outputs
of their rows, whatever kernel reads the head and wherever the word lies, and
lists whose entries have no mass, or no number, for it."""
import math

import pytest
import torch

import chunked_lm_head_gb300 as flce
from chunked_lm_head_gb300 import _lib

from test_topk_gpu import make

pytestmark = pytest.mark.gpu

LISTED = [4000, 4001, 4002, 4003]
WORDS = {"first": [0], "later": [3111], "last": [5002], "a chunk": list(range(2048, 2080)),
         "the first chunk": list(range(32)), "all but the list": [v for v in range(5003) if v not in LISTED]}


@pytest.mark.parametrize("tf", [None, {"softcap": 5.0}], ids=["linear", "softcap"])
@pytest.mark.parametrize("where", list(WORDS))
@pytest.mark.parametrize("N", [1, 4, 5, 200])
def test_a_word_that_is_not_a_number(N, where, tf):
    """N <= 4: the matrix-vector forward; beyond, tiles.  One call: tiles that
    keep their exponentials."""
    c = make(N, 64, 5003, 4, seed=31, whole=True)
    c["ids"][:] = torch.tensor(LISTED, device="cuda")
    c["W"][WORDS[where]] = float("nan")
    for tail in (False, True):
        args = (c["h"], c["W"], c["ids"], c["logits"], c["lse_t"], None, None, tail)
        out = flce.topk_kd_forward(*args, transform=tf)
        assert torch.isnan(out["lse"]).all() and torch.isnan(out["kl"]).all() and torch.isnan(out["loss"])
        one = flce.topk_kd_forward_backward(*args, transform=tf)
        assert torch.isnan(one["lse"]).all() and torch.isnan(one["kl"]).all() and torch.isnan(one["loss"])
    assert _lib.flce_device_status() == 0


@pytest.mark.parametrize("N", [4, 5, 200])
def test_a_token_that_is_not_a_number(N):
    c = make(N, 64, 5003, 4, seed=32, whole=True)
    want = flce.topk_kd_forward(c["h"], c["W"], c["ids"], c["logits"], c["lse_t"])
    c["h"][2, 5] = float("nan")
    for call in (flce.topk_kd_forward, flce.topk_kd_forward_backward):
        out = call(c["h"], c["W"], c["ids"], c["logits"], c["lse_t"])
        assert torch.isnan(out["lse"][2]) and torch.isnan(out["kl"][2]) and torch.isnan(out["loss"])
        rest = torch.arange(N, device="cuda") != 2
        assert torch.isfinite(out["lse"][rest]).all()
        if call is flce.topk_kd_forward:
            assert torch.equal(out["kl"][rest], want["kl"][rest])


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
