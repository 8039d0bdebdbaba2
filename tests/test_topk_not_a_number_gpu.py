"""Distillation from top logits: logits that are not numbers reach the outputs
of their rows, whatever kernel reads the head and wherever the word lies."""
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
