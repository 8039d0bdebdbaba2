"""The layer norm, the scores and the likeliest words as one program runs them: a
policy step (norm with the residual's addition -> log-probabilities and entropy ->
clipped objective with an entropy term -> gradients), and a teacher's lists for a
student's distillation.  Each link is checked in 64 bits on what the link before
it gave."""
import math

import pytest
import torch

import chunked_lm_head_gb300 as flce
from chunked_lm_head_gb300 import _lib

import layer_ref as L
import score_ref as S
import topk_ref as T

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
EPS = 1e-5


def batch(N, H, V, residual, seed):
    g = torch.Generator(device="cuda").manual_seed(100 * seed + N)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    t = torch.randint(0, V, (N,), generator=g, device="cuda")
    if N > 4:
        t[: N // 4] = S.IGNORE  # a prompt without loss
    return dict(x=rnd(N, H).bfloat16(), r=rnd(N, H).to(residual), w=(1 + 0.1 * rnd(H)).to(residual),
                b=(0.1 * rnd(H)).to(residual), W=(3 / math.sqrt(H) * rnd(V, H)).bfloat16(), t=t, adv=rnd(N),
                old=-math.log(V) + 0.3 * rnd(N))


def objective(logp, entropy, t, adv, old, c_entropy=0.02, clip=0.2):
    """The clipped ratio's and the entropy's mean over the counted rows."""
    on = (t != S.IGNORE).to(logp.dtype)
    ratio = (logp - old).clamp(max=20).exp()
    gain = torch.minimum(ratio * adv, ratio.clamp(1 - clip, 1 + clip) * adv) + c_entropy * entropy
    return -(gain * on).sum() / on.sum().clamp(min=1)


# one token, a few, a ragged batch with kept logits, one in row blocks without
@pytest.mark.parametrize("tf", [None, {"softcap": 20.0, "temperature": 0.8}], ids=["none", "softcap"])
@pytest.mark.parametrize("N,H,V,chunk,residual", [(1, 64, 1000, 256, F32), (3, 264, 2003, 256, BF16),
                                                  (150, 520, 3001, 256, F32), (421, 1000, 5003, 512, BF16),
                                                  (300, 256, 4096, 128, F32)])
def test_policy_step(N, H, V, chunk, residual, tf):
    c = batch(N, H, V, residual, 1)
    leaves = [c[k].clone().requires_grad_(True) for k in ("x", "r", "w", "b", "W")]
    for step in range(2):  # (twice: the weights change in place between)
        x, r, w, b, W = leaves
        h, s = flce.layer_norm(x, w, b, r, eps=EPS)
        logp, entropy = flce.selective_log_softmax_entropy(h, W, c["t"], chunk_rows=chunk, transform=tf)
        loss = objective(logp, entropy, c["t"], c["adv"], c["old"])
        for v in (h, logp, entropy):
            v.retain_grad()
        (loss + 1e-3 * s.float().square().sum() / N).backward()  # (the stream goes on, with a gradient of its own)
        assert _lib.flce_device_status() == 0

        with torch.no_grad():
            sd = L.stream(x, r)
            assert torch.equal(s, sd)
            y, _, _ = L.forward(sd, w, b, EPS, 0.0)
            err = (h.double() - y).abs()
            assert bool((err <= 1.01 * y.abs() * L.half_step(BF16) + 2 * L.forward_bound(sd, w, b, EPS, 0.0)).all())
            ref = S.reference(h, W, c["t"], 0, tf)
            S.check(dict(logp=logp, entropy=entropy), h, W, c["t"], ref, tf=tf)
            kept = _lib.flce_score_state_bytes(N, H, V, chunk) > 0
            S.check_grads(h.grad, W.grad, h, W, c["t"], ref, logp.grad, entropy.grad, tf, kept=kept)
            ds = (2e-3 / N * s.float()).to(residual)  # as autograd forms it, to its roundings (3 half steps)
            d, dw, db = L.backward(h.grad, ds, sd, w, EPS, 0.0)
            bd, bw, bb = L.backward_bounds(h.grad, ds, sd, w, EPS, 0.0)
            bd = bd + 3.03 * L.half_step(residual) * ds.double().abs()
            for name, got, want, bound in (("dx", x.grad, d, 2 * bd), ("dr", r.grad, d, 2 * bd), ("dw", w.grad, dw, bw),
                                           ("db", b.grad, db, bb)):
                err = (got.double() - want).abs()
                assert bool((err <= bound + 1.01 * L.half_step(got.dtype) * want.abs()).all()), (name, float(err.max()))
            assert not bool(h.grad[c["t"] == S.IGNORE].any())
            # the objective's own derivative: its value along a step of logp and entropy, in 64 bits
            lp, en = logp.double(), entropy.double()
            f = lambda e: objective(lp + e * logp.grad, en + e * entropy.grad, c["t"], c["adv"].double(),  # noqa: E731
                                    c["old"].double())
            norm = float(logp.grad.double().square().sum() + entropy.grad.double().square().sum())
            slope = float(f(1e-5) - f(-1e-5)) / 2e-5
            assert abs(slope - norm) <= 1e-3 * norm + 1e-9, (slope, norm)
            for v in (w, b, W):
                v -= 0.1 * v.grad
                v.grad = None
            x.grad = r.grad = None


@pytest.mark.parametrize("N,H,V,K", [(1, 64, 1000, 8), (150, 264, 3001, 33), (300, 512, 2000, 128)])
def test_a_teachers_lists_for_a_student(N, H, V, K):
    c = batch(N, H, V, F32, 2)
    g = torch.Generator(device="cuda").manual_seed(7)
    h, _ = flce.layer_norm(c["x"], c["w"], c["b"], c["r"])
    top = flce.top_logprobs(h, c["W"], K, c["t"])
    S.check(top, h, c["W"], c["t"], S.reference(h, c["W"], c["t"], K), K)
    hs = (0.8 * h.float() + 0.4 * torch.randn(N, H, generator=g, device="cuda")).bfloat16().requires_grad_(True)
    Ws = (c["W"].float() * 0.9).bfloat16().requires_grad_(True)
    zero = torch.zeros(N, device="cuda")
    loss, kl, n = flce.topk_distill_loss(hs, Ws, top["ids"], top["logprobs"], zero, c["t"], tail=True)
    dH, dW = torch.autograd.grad(loss, (hs, Ws))
    assert _lib.flce_device_status() == 0
    ref = T.reference(hs, Ws, top["ids"], top["logprobs"], zero, c["t"], tail=True)
    T.check(dict(loss=loss.detach(), kl=kl, n_valid=n, dH=dH, dW=dW), ref)
    assert int(n) == int((c["t"] != S.IGNORE).sum())  # a list is there for every counted row


def test_a_captured_policy_step():
    N, H, V = 200, 512, 3001
    c = batch(N, H, V, F32, 3)

    def step():
        x, r, w, b, W = (c[k].detach().requires_grad_(True) for k in ("x", "r", "w", "b", "W"))
        h, s = flce.layer_norm(x, w, b, r)
        logp, entropy = flce.selective_log_softmax_entropy(h, W, c["t"])
        loss = objective(logp, entropy, c["t"], c["adv"], c["old"])
        top = flce.top_logprobs(h.detach(), W.detach(), 5, c["t"])
        return [loss.detach(), top["ids"], top["logprobs"], *torch.autograd.grad(loss, (x, r, w, b, W))]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    # two graphs that take turns
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step())
        graphs.append(graph)
    for seed in (4, 5):
        new = batch(N, H, V, F32, seed)
        for k in c:
            c[k].copy_(new[k])
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        want = step()
        for got in outs:
            assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert _lib.flce_device_status() == 0
