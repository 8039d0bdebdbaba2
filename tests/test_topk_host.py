"""The distillation from top logits: refusals on the host, before any launch,
and its sizes."""
import ctypes

import pytest
import torch

import chunked_lm_head_gb300 as flce
from chunked_lm_head_gb300 import _lib

import topk_ref as R

P = 1 << 20  # a non-null, aligned value; never dereferenced on these paths
D = _lib.DTYPES
OK, INVALID, UNSUPPORTED = 0, 1, 3


def teacher(ids=P, logits=P, lse=None, ld_ids=8, ld_logits=8, it=D["i64"], lt=D["f32"], k=8, tail=0):
    return _lib.TopLogits(ids, logits, lse, ld_ids, ld_logits, it, lt, k, tail)


def fwd(t, h=P, W=P, targets=None, weights=None, N=4, H=64, V=100, tf=None, flags=0, kl=P, lse=None, loss=None,
        nv=None, state=None, ws=None, wb=0):
    return _lib.flce_topk_kd_forward(h, W, t, targets, weights, N, H, V, 256, -100, tf, flags, kl, lse, loss, nv,
                                     state, ws, wb, 0)


def fb(t, h=P, W=P, N=4, H=64, V=100, tf=None, g=1.0, dH=P, dW=P, dt=D["f32"], loss=None, ws=None, wb=0):
    return _lib.flce_topk_kd_forward_backward(h, W, t, None, None, N, H, V, 256, -100, tf, g, None, None, loss, None,
                                              dH, dW, dt, ws, wb, 0)


def bwd(state=P, h=P, W=P, N=4, H=64, V=100, k=8, tf=None, dH=P, dW=P, dt=D["f32"], ws=None, wb=0):
    return _lib.flce_topk_kd_backward(h, W, state, 1.0, None, None, dH, dW, dt, N, H, V, k, 256, tf, ws, wb, 0)


BAD_TEACHERS = [
    (dict(k=0), INVALID), (dict(k=-3), INVALID), (dict(ids=None), INVALID), (dict(logits=None), INVALID),
    (dict(ld_ids=7), INVALID), (dict(ld_logits=4), INVALID), (dict(it=D["f32"]), INVALID),
    (dict(lt=D["i32"]), INVALID), (dict(tail=1), INVALID), (dict(tail=2, lse=P), INVALID),
    (dict(k=1025, ld_ids=1025, ld_logits=1025), UNSUPPORTED), (dict(ids=P + 4), UNSUPPORTED),
    (dict(logits=P + 2), UNSUPPORTED), (dict(lse=P + 2), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,want", BAD_TEACHERS)
def test_bad_teachers_are_refused(kw, want):
    assert fwd(teacher(**kw)) == want
    assert fb(teacher(**kw)) == want


@pytest.mark.parametrize("kw,want", [
    (dict(kl=None), INVALID), (dict(h=None), INVALID), (dict(W=None), INVALID), (dict(N=-1), INVALID),
    (dict(H=0), INVALID), (dict(V=0), INVALID), (dict(flags=2), INVALID), (dict(tf={"temperature": 0.0}), INVALID),
    (dict(ws=P, wb=64), INVALID), (dict(H=68), UNSUPPORTED), (dict(h=P + 2), UNSUPPORTED),
    (dict(targets=P + 4), UNSUPPORTED), (dict(weights=P + 1), UNSUPPORTED), (dict(kl=P + 2), UNSUPPORTED),
    (dict(state=P + 16), UNSUPPORTED),
])
def test_forward_refusals(kw, want):
    assert fwd(teacher(), **kw) == want
    assert fwd(None) == INVALID


@pytest.mark.parametrize("kw,want", [
    (dict(dH=None, dW=None), INVALID), (dict(h=None), INVALID), (dict(g=float("inf")), INVALID),
    (dict(tf={"softcap": -1.0}), INVALID), (dict(ws=P, wb=64), INVALID), (dict(H=60), UNSUPPORTED),
    (dict(dt=D["f16"]), INVALID),
    (dict(dW=P + 4), UNSUPPORTED), (dict(loss=P + 2), UNSUPPORTED),
])
def test_one_call_refusals(kw, want):
    assert fb(teacher(), **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(state=None), INVALID), (dict(k=0), INVALID), (dict(dH=None, dW=None), INVALID), (dict(h=None), INVALID),
    (dict(tf={"temperature": -1.0}), INVALID), (dict(ws=P, wb=64), INVALID), (dict(k=1025), UNSUPPORTED),
    (dict(dt=D["i64"]), INVALID), (dict(dW=P + 8), UNSUPPORTED),
    (dict(state=P + 8), UNSUPPORTED), (dict(H=12), UNSUPPORTED),
])
def test_backward_refusals(kw, want):
    assert bwd(**kw) == want


def test_sizes():
    assert ctypes.sizeof(_lib.TopLogits) == 56
    s, w = _lib.flce_topk_kd_state_bytes, _lib.flce_topk_kd_workspace_bytes
    assert s(-1, 4) == 0 and s(4, 0) == 0 and s(4, 1025) == 0 and w(4, 64, 100, 0, 256) == 0
    assert s(4096, 64) >= 4096 * (64 * 8 + 16) and s(4096, 64) <= 4096 * (64 * 8 + 16) + 2048
    # beside the cross-entropy's workspace: 12 bytes per entry and a few per row
    extra = w(4096, 512, 20000, 64, 256) - _lib.flce_workspace_bytes(4096, 512, 20000, 256)
    assert extra <= 4096 * (64 * 12 + 64) + (1 << 16)
    # a bf16 dW takes fp32 scratch only where several row blocks are summed
    f = _lib.flce_topk_kd_forward_backward_workspace_bytes
    assert f(4096, 512, 20000, 64, 4096, D["bf16"]) == f(4096, 512, 20000, 64, 4096, D["f32"])
    assert f(4096, 512, 20000, 64, 2048, D["bf16"]) == f(4096, 512, 20000, 64, 2048, D["f32"]) + 20000 * 512 * 4


def test_torch_checks():
    h, W = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(100, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        flce.topk_distill_loss(h, W, torch.zeros(4, 3, dtype=torch.int64), torch.zeros(4, 3))


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("tf", [None, {"softcap": 4.0, "temperature": 0.7, "scale_multiply": 1.5}])
def test_reference_gradient_matches_differences(tail, tf):
    """The reference's D against central differences of its kl, in 64 bits."""
    g = torch.Generator().manual_seed(3)
    N, V, K = 5, 23, 6
    z = torch.randn(N, V, generator=g, dtype=torch.float64) * 2
    t = torch.randn(N, V, generator=g, dtype=torch.float64) * 2
    logits, ids = t.topk(K, dim=1)
    ids[1, 3:] = -1
    ids[2, 1] = ids[2, 0]  # listed twice
    q, listed, counted = R.teacher(ids, logits, t.logsumexp(1) if tail else None, V)
    assert counted.all()
    _, _, D, _ = R.loss_terms(z, q, listed, tail, tf)
    e = 1e-6
    for _ in range(6):
        d = torch.randn(N, V, generator=g, dtype=torch.float64)
        up, dn = (R.loss_terms(z + s * e * d, q, listed, tail, tf)[0] for s in (1, -1))
        diff = (up - dn) / (2 * e)
        assert torch.allclose((D * d).sum(1), diff, rtol=1e-6, atol=1e-8)
