"""How often the distillation from top logits rounds, and that no rounding is
common to many of its sums."""
import pytest
import torch

import chunked_lm_head_gb300 as flce
from chunked_lm_head_gb300 import _lib

import topk_ref as R
from test_topk_gpu import make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("N", [200, 300, 900])
def test_one_rounding_of_the_dlogits(N, tail):
    """One counted row: every word's dW is a single product, so the bound on it
    is one rounding's.  The one-call step rounds its exponentials to fp16 (half
    a step 2^-11, an eighth of bf16's 2^-8) and D to bf16 once; the recomputing
    backward D alone.  (A quarter of bf16's half step covers the eighth and the
    fp32 steps between.)"""
    c = make(N, 64, 3001, 16, seed=61, whole=True)
    c["targets"] = torch.full((N,), -100, device="cuda")
    c["targets"][137] = 0
    ref = R.reference(**c, tail=tail)
    args = (c["h"], c["W"], c["ids"], c["logits"], c["lse_t"], c["targets"], None, tail)
    one = flce.topk_kd_forward_backward(*args)
    R.check(one, ref, roundings=1.25, what="one call")
    half = flce.topk_kd_forward_backward(*args, dW_dtype=torch.bfloat16)
    R.check(half, ref, roundings=1.25, what="one call, bf16 dW")
    out = flce.topk_kd_forward(*args, for_backward=True)
    dH, dW = flce.topk_kd_backward(c["h"], c["W"], out["state"], 16, 1.0, count=out["n_valid"])
    R.check(dict(dH=dH, dW=dW), ref, roundings=1.0, what="recompute")
    assert _lib.flce_device_status() == 0


def test_no_rounding_of_the_common_scale():
    """1 / n is a factor of every gradient.  With the n (of 129 to 400) at which
    bf16 rounds it worst, gradients scaled by the rounded factor would all be
    off by that much; a quarter of it is allowed."""
    inv = [(abs(float(torch.tensor(1.0 / n).bfloat16()) * n - 1), n) for n in range(129, 401)]
    off, n = max(inv)
    assert off > 2.0 ** -9
    c = make(n, 64, 2000, 16, seed=62, whole=True)
    ref = R.reference(**c, tail=True)
    for dtype in (torch.float32, torch.bfloat16):
        got = flce.topk_kd_forward_backward(c["h"], c["W"], c["ids"], c["logits"], c["lse_t"], tail=True,
                                            dW_dtype=dtype)
        for k in ("dH", "dW"):
            along = float((got[k].double() * ref[k]).sum() / ref[k].square().sum()) - 1
            assert abs(along) <= off / 4, (k, dtype, along, off)


def one_way(N, H, V, seed):
    """h and W whose logits lie near 30, their partial sums all growing."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    h = (1 + 0.25 * torch.randn(N, H, generator=g, device="cuda")).bfloat16()
    W = (30 / H + 0.5 / H ** 0.5 * torch.randn(V, H, generator=g, device="cuda")).bfloat16()
    ids = torch.randint(0, V, (N, 4), generator=g, device="cuda")
    return h, W, ids, torch.randn(N, 4, generator=g, device="cuda")


def cut(H, size):
    """What the tensor cores' sums of H products lack of a logit of this size:
    0.26 x 2^-24 of it at every step of 16."""
    return 0.26 * (H / 16) * 2.0 ** -24 * size


@pytest.mark.parametrize("H", [4096, 8192])
def test_the_forward_puts_back_what_the_tensor_cores_cut(H):
    """Its log-sum-exp is less than half as far off, on average, as the
    cross-entropy's of the same logits, which has no correction (a missing
    one would be as far off, one of the wrong sign twice as far)."""
    h, W, ids, logits = one_way(256, H, 1500, 63)
    want = (h.double() @ W.double().t()).logsumexp(1)
    plain = flce.forward(h, W, torch.zeros(256, dtype=torch.int64, device="cuda"))["lse"]
    off = abs(float((plain.double() - want).mean()))
    for call in (flce.topk_kd_forward, flce.topk_kd_forward_backward):
        got = call(h, W, ids, logits)["lse"]
        assert abs(float((got.double() - want).mean())) <= off / 2, (call.__name__, off)


@pytest.mark.parametrize("N", [4, 64])
def test_the_recomputed_logits_are_those_of_the_forward(N):
    """A logit that the backward recomputes short, against a log-sum-exp that is
    not, makes every unlisted word's gradient short by that much: half of what
    the cut alone would do is allowed."""
    H, V = 8192, 1500
    h, W, ids, logits = one_way(N, H, V, 64)
    ref = R.reference(h, W, ids, logits)
    out = flce.topk_kd_forward(h, W, ids, logits, for_backward=True)
    _, dW = flce.topk_kd_backward(h, W, out["state"], 4, 1.0, count=out["n_valid"])
    one = flce.topk_kd_forward_backward(h, W, ids, logits)
    unlisted = torch.ones(V, dtype=torch.bool, device="cuda")
    unlisted[ids.flatten()] = False
    want = ref["dW"][unlisted]
    for name, got in (("recompute", dW), ("one call", one["dW"])):
        along = float((got[unlisted].double() * want).sum() / want.square().sum()) - 1
        assert abs(along) <= cut(H, 30) / 2, (name, along, cut(H, 30))
