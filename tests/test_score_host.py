"""The scores: refusals on the host, before any launch, and their sizes."""
import pytest
import torch

import chunked_lm_head_gb300 as flce
from chunked_lm_head_gb300 import _lib

import score_ref as R

P = 1 << 20  # a non-null, aligned value; never dereferenced on these paths
D = _lib.DTYPES
OK, INVALID, UNSUPPORTED = 0, 1, 3


def fwd(h=P, W=P, t=P, N=4, H=64, V=1000, k=0, tf=None, logp=P, lse=P, ent=P, ids=None, words=None, st=None, ws=None,
        wb=0):
    return _lib.flce_score(h, W, t, N, H, V, k, -100, tf, logp, lse, ent, ids, words, st, ws, wb, 0)


def bwd(h=P, W=P, t=P, lse=P, ent=P, ga=P, ge=P, st=None, dH=P, dW=P, dt=D["f32"], N=4, H=64, V=1000, tf=None, ws=None,
        wb=0):
    return _lib.flce_score_backward(h, W, t, lse, ent, ga, ge, st, dH, dW, dt, N, H, V, 256, -100, tf, ws, wb, 0)


@pytest.mark.parametrize("kw,want", [
    (dict(h=None), INVALID), (dict(W=None), INVALID), (dict(N=-1), INVALID), (dict(N=1 << 31), INVALID),
    (dict(N=(1 << 31) - 65536), INVALID), (dict(H=0), INVALID), (dict(V=0), INVALID), (dict(k=-1), INVALID),
    (dict(k=1001, ids=P), INVALID), (dict(k=3), INVALID), (dict(ids=P), INVALID), (dict(words=P), INVALID),
    (dict(t=None), INVALID), (dict(logp=None, lse=None, ent=None), INVALID), (dict(tf={"temperature": 0.0}), INVALID),
    (dict(tf={"softcap": -1.0}), INVALID), (dict(ws=P, wb=64), INVALID), (dict(ws=P + 8, wb=1 << 40), INVALID),
    (dict(k=129, ids=P), UNSUPPORTED), (dict(H=60), UNSUPPORTED), (dict(h=P + 2), UNSUPPORTED),
    (dict(W=P + 8), UNSUPPORTED), (dict(t=P + 4), UNSUPPORTED), (dict(logp=P + 2), UNSUPPORTED),
    (dict(lse=P + 1), UNSUPPORTED), (dict(ent=P + 2), UNSUPPORTED), (dict(k=3, ids=P + 4), UNSUPPORTED),
    (dict(k=3, words=P + 2), UNSUPPORTED),
    (dict(st=P, k=3, ids=P), INVALID), (dict(st=P, t=None, logp=None), INVALID), (dict(st=P + 16), UNSUPPORTED),
    (dict(st=P, N=32769), UNSUPPORTED), (dict(st=P, ws=P, wb=64), INVALID),
    (dict(N=0), OK), (dict(N=0, h=None, W=None, t=None), OK), (dict(N=0, k=5, ids=P), OK),
])
def test_forward_refusals(kw, want):
    assert fwd(**kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(h=None), INVALID), (dict(W=None), INVALID), (dict(t=None), INVALID), (dict(lse=None), INVALID),
    (dict(ent=None), INVALID), (dict(dH=None, dW=None), INVALID), (dict(N=-1), INVALID), (dict(H=0), INVALID),
    (dict(dt=D["f16"]), INVALID), (dict(tf={"temperature": -1.0}), INVALID), (dict(ws=P, wb=64), INVALID),
    (dict(H=12), UNSUPPORTED), (dict(dW=P + 8), UNSUPPORTED), (dict(dH=P + 2), UNSUPPORTED),
    (dict(ga=P + 2), UNSUPPORTED), (dict(ge=P + 2), UNSUPPORTED), (dict(t=P + 4), UNSUPPORTED),
    (dict(st=P + 128), UNSUPPORTED), (dict(st=P, N=32769), UNSUPPORTED), (dict(st=P, ws=P, wb=64), INVALID),
    (dict(st=P, dH=None, dW=None), INVALID), (dict(N=0, dW=None), OK), (dict(N=0, dH=None, dW=None), OK),
])
def test_backward_refusals(kw, want):
    assert bwd(**kw) == want


def test_operators_check_what_the_kernels_rest_on():
    """torch.ops.flce refuses what its callers here would not pass on."""
    norm, score, top = _lib.torch_ops()
    x, t = torch.zeros(3, 64, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int64)
    for call in (lambda: score(x, x, t, 256, -100, [], False), lambda: top(x, x, 2, None, -100, []),
                 lambda: norm(x, x[0], None, None, 1e-5, 0.0), lambda: score(x[0], x, t, 256, -100, [], False),
                 lambda: norm(x[0], x[0], None, None, 1e-5, 0.0)):
        with pytest.raises(RuntimeError, match="flce: "):
            call()


def test_sizes():
    f = _lib.flce_score_workspace_bytes
    assert f(-1, 64, 1000, 4) == 0 and f(4, 64, 1000, 129) == 0 and f(4, 64, 100, 101) == 0 and f(4, 64, 100, -1) == 0
    # records or logits of at most 256 MB, whatever the rows, beside a few per row
    for N in (1, 5000, 1 << 20):
        for V, k in ((1000, 128), (32000, 128), (151936, 20), (1 << 20, 128)):
            assert f(N, 512, V, k) <= (256 << 20) + N * 64 + (64 << 20) + 4096 * 512 * 2
    # without words: partials and a few per row
    assert f(1 << 20, 512, 151936, 0) <= (1 << 20) * 64 + (32 << 20)
    b = _lib.flce_score_backward_workspace_bytes
    assert b(4096, 512, 20000, 4096, D["bf16"]) == b(4096, 512, 20000, 4096, D["f32"])
    assert b(8192, 512, 20000, 256, D["bf16"]) >= 20000 * 512 * 4
    # the kept logits: 2 bytes a column and 1/8 for the chunks' maxima, where the rows fit the budget
    s = _lib.flce_score_state_bytes
    assert 0 < s(4096, 1024, 20000, 4096) <= 4096 * (20256 * 2.25 + 16) + 4096
    assert s(4096, 1024, 20000, 3968) == 0 and s(4096, 64, 20000, 4096) == 0 and s(0, 1024, 20000, 4096) == 0
    assert s(128, 64, 20000, 128) > 0 and s(256, 64, 20000, 256) > 0 and s(257, 64, 20000, 512) == 0
    assert s(40000, 1024, 20000, 40000) == 0 and s(5, 1024, 20000, 1) > 0 and s(-1, 1024, 20000, 4096) == 0


def test_torch_checks():
    h, W = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(100, 64, dtype=torch.bfloat16)
    t = torch.zeros(4, dtype=torch.int64)
    for call in (lambda: flce.top_logprobs(h, W, 3), lambda: flce.selective_log_softmax_entropy(h, W, t)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


@pytest.mark.parametrize("tf", [None, {"softcap": 4.0, "temperature": 0.7, "scale_multiply": 1.5}])
def test_reference_gradient_matches_differences(tf):
    """The reference's D against central differences of its values, in 64 bits."""
    g = torch.Generator().manual_seed(3)
    N, V = 5, 23
    eye = torch.eye(V, dtype=torch.float64)
    z = 2 * torch.randn(N, V, generator=g, dtype=torch.float64)
    t = torch.randint(0, V, (N,), generator=g)
    t[2] = R.IGNORE
    ga, ge = torch.randn(N, generator=g, dtype=torch.float64), torch.randn(N, generator=g, dtype=torch.float64)
    D, _ = R.dlogits(R.reference(z, eye, t, 0, tf), t, ga, ge)

    def value(z):
        r = R.reference(z, eye, t, 0, tf)
        return r["logp"] * ga + r["entropy"] * ge

    e = 1e-6
    for _ in range(6):
        d = torch.randn(N, V, generator=g, dtype=torch.float64)
        diff = (value(z + e * d) - value(z - e * d)) / (2 * e)
        assert torch.allclose((D * d).sum(1), diff, rtol=1e-6, atol=1e-8)
