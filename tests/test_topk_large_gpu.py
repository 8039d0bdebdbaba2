"""The one-call step of the distillation from top logits past 32-bit offsets
into its exponentials, and over more rows than one CTA lists."""
import pytest
import torch

import chunked_lm_head_gb300 as flce
from chunked_lm_head_gb300 import _lib

import topk_ref as R
from test_topk_gpu import make, run_all

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_one_row_block_past_32_bit_offsets(dtype):
    """17,000 x 131,072 exponentials in one block: kl and dH of the last rows,
    dW of the last words."""
    N, H, V, K, last = 17000, 64, 131072, 4, 500
    g = torch.Generator(device="cuda").manual_seed(101)
    h = torch.randn(N, H, generator=g, device="cuda").bfloat16()
    W = (0.1 * torch.randn(V, H, generator=g, device="cuda")).bfloat16()
    ids = torch.randint(0, V, (N, K), generator=g, device="cuda")
    ids[::3, 0] = V - 1 - torch.arange(len(range(0, N, 3)), device="cuda") % last
    logits = torch.randn(N, K, generator=g, device="cuda")
    one = flce.topk_kd_forward_backward(h, W, ids, logits, chunk_rows=N, dW_dtype=dtype)
    assert _lib.flce_device_status() == 0
    s = slice(N - 40, N)
    ref = R.reference(h[s], W, ids[s], logits[s])
    R.check({"kl": one["kl"][s], "lse": one["lse"][s], "dH": (one["dH"][s].double() * (N / 40)).bfloat16()}, ref,
            roundings=2)
    want = torch.zeros(last, H, dtype=torch.float64, device="cuda")
    for a in range(0, N, 500):
        z = h[a:a + 500].double() @ W.double().t()
        q, _, _ = R.teacher(ids[a:a + 500], logits[a:a + 500], None, V)
        D = (z[:, V - last:] - z.logsumexp(1, keepdim=True)).exp() * q.sum(1, keepdim=True) - q[:, V - last:]
        want += (D / N).t() @ h[a:a + 500].double()
    # one bf16 rounding of D and one of dW (2^-8 of each at most)
    assert float((one["dW"][V - last:].double() - want).norm()) <= 2 * 2.0 ** -8 * float(want.norm())


@pytest.mark.parametrize("options", [{}, {"compact": 0}, {"cta_group": 1}],
                         ids=lambda o: "-".join(f"{k}{v}" for k, v in o.items()) or "default")
def test_more_rows_than_one_cta_lists(options):
    c = make(33001, 64, 520, 6, seed=102, mask=True, pad=True, weights=True, whole=True)
    with _lib.options(**options):
        run_all(c, tail=True, one_call_chunk=4096)
