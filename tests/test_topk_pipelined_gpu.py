"""The recomputing backward of the distillation from top logits over several
vocabulary slabs: the pipelined row blocks that the default chunk takes at
large sizes, on SM pairs and on single CTAs, against the definition in 64
bits."""
import pytest
import torch

import chunked_lm_head_gb300 as flce
from chunked_lm_head_gb300 import _lib

import topk_ref as R
from test_topk_gpu import make, run_all

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cta_group", [2, 1])
@pytest.mark.parametrize("tail,tf", [(False, None), (True, None), (True, {"softcap": 5.0, "temperature": 0.8})],
                         ids=["given", "tail", "tail-softcap"])
@pytest.mark.parametrize("N,H,V,K,masks", [(700, 128, 3000, 30, True), (513, 264, 4099, 64, False),
                                           (1100, 64, 5003, 200, True)])
def test_pipelined_row_blocks(N, H, V, K, masks, tail, tf, cta_group):
    c = make(N, H, V, K, seed=51, mask=masks, pad=masks, weights=masks, whole=True)
    with _lib.options(bwd_rows=256, cta_group=cta_group):
        plan = _lib.flce_backward_plan(N, H, V, 128)
        assert plan["dlogits_buffers"] == 2 and plan["vocab_slabs"] > 1 and plan["row_blocks"] > 1, plan
        run_all(c, tail=tail, tf=tf, chunk=128, one_call_chunk=128)


def test_pipelined_row_blocks_on_few_workers():
    """Units drawn by 3 SM pairs: every wait is met whatever is resident."""
    c = make(700, 128, 3000, 30, seed=52, mask=True, pad=True, whole=True)
    with _lib.options(bwd_rows=256, grid_workers=3):
        assert _lib.flce_backward_plan(700, 128, 3000, 128)["dlogits_buffers"] == 2
        run_all(c, tail=True, chunk=128)


def test_recompute_past_32_bit_offsets():
    """N V past 2^31 through the recomputing backward: dH of the last rows, dW
    of the last words, against the definition."""
    N, H, V, K = 16500, 64, 131072, 4
    g = torch.Generator(device="cuda").manual_seed(53)
    h = torch.randn(N, H, generator=g, device="cuda").bfloat16()
    W = (0.1 * torch.randn(V, H, generator=g, device="cuda")).bfloat16()
    ids = torch.randint(0, V, (N, K), generator=g, device="cuda")
    ids[::3, 0] = V - 1 - torch.arange(len(range(0, N, 3)), device="cuda") % 500  # the last words are listed too
    logits = torch.randn(N, K, generator=g, device="cuda")
    out = flce.topk_kd_forward(h, W, ids, logits, for_backward=True)
    dH, dW = flce.topk_kd_backward(h, W, out["state"], K, 1.0, 256, count=out["n_valid"])
    assert _lib.flce_device_status() == 0
    s = slice(N - 40, N)
    ref = R.reference(h[s], W, ids[s], logits[s])
    R.check({"kl": out["kl"][s], "dH": (dH[s].double() * (N / 40)).bfloat16()}, ref, roundings=2)
    # the last 500 words' dW over all rows, from D in 64 bits
    last = 500
    want = torch.zeros(last, H, dtype=torch.float64, device="cuda")
    for a in range(0, N, 500):
        z = h[a:a + 500].double() @ W.double().t()
        q, _, _ = R.teacher(ids[a:a + 500], logits[a:a + 500], None, V)
        D = (z[:, V - last:] - z.logsumexp(1, keepdim=True)).exp() * q.sum(1, keepdim=True) - q[:, V - last:]
        want += (D / N).t() @ h[a:a + 500].double()
    # one bf16 rounding of D (2^-8 of each term at most, pointing both ways)
    assert float((dW[V - last:].double() - want).norm()) <= 2.0 ** -8 * float(want.norm())
