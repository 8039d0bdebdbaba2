"""The norm, the distillation from stored top logits and the e4m3 head run
together (examples/distill_from_top_logits.py)."""
import os
import sys

import pytest
import torch

from gpu_util import LOGP_ATOL, LOGP_RTOL

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,hidden,vocab", [(300, 256, 3000), (37, 1040, 1001)])
def test_example_trains_and_scores(tokens, hidden, vocab):
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import distill_from_top_logits as ex
    r = ex.main(tokens, hidden, vocab, k=16, steps=6)
    losses = r["losses"].tolist()
    assert all(b < a for a, b in zip(losses, losses[1:])), losses  # plain gradient descent, small steps
    # the e4m3 head's log-probs against 64 bits on the operands it was given
    h = r["normed"]["q"].double() * r["normed"]["scale"].double()[:, None]
    W = r["W8"].view(torch.float8_e4m3fn).double() * r["W_scale"].double()[:, None]
    keep = r["targets"] >= 0
    want = (h @ W.t()).log_softmax(1).gather(1, r["targets"].clamp(min=0)[:, None])[:, 0]
    err = (r["logp"].double() - want).abs()[keep]
    assert bool((err <= LOGP_ATOL + LOGP_RTOL * want[keep].abs()).all())
    assert not r["logp"][~keep].any()
