"""One head's work between the residual stream and the loss, with the calls a
training program and a scoring program would make:

  * train: final RMS norm with the residual's addition -> student head ->
    distillation loss from a teacher's stored top logits -> gradients of the
    stream, the norm's gain, and the head;
  * score: the same norm with e4m3 rows and scales -> e4m3 head -> log-probs.

    python examples/distill_from_top_logits.py [--tokens N] [--hidden H] [--vocab V] [--steps S]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import chunked_lm_head_gb300 as flce  # noqa: E402
from chunked_lm_head_gb300 import _lib  # noqa: E402


def stored_teacher(x, W, k, generator):
    """(ids[N,k], logits[N,k] bf16, lse[N]) as a teacher's pass would have kept
    them: its best k words per token and the log-sum-exp of all of them."""
    h = 0.9 * x.float() + 0.5 * torch.randn(x.shape, generator=generator, device=x.device)
    z = 2.0 * (h @ W.float().t())
    logits, ids = z.topk(k, dim=1)
    return ids.int(), logits.bfloat16(), z.logsumexp(1)


def step_size(n_valid: int, hidden: int) -> float:
    """A gradient step the mean loss does not overshoot: one over its curvature
    in the head, at most 1/2 (softmax) times the largest eigenvalue of h h^T / n,
    near (1 + sqrt(hidden / n))^2 for n normed rows."""
    return 2.0 / (1.0 + (hidden / max(n_valid, 1)) ** 0.5) ** 2


def train(x, stream, W, teacher, targets, steps: int):
    """`steps` steps of plain gradient descent on the head and the gain; the
    losses, one per step."""
    ids, logits, lse = teacher
    lr = step_size(int((targets != flce.IGNORE_INDEX).sum()), x.shape[1])
    gain = torch.ones(x.shape[1], device=x.device, requires_grad=True)
    head = W.clone().requires_grad_(True)
    x, stream = x.clone().requires_grad_(True), stream.clone().requires_grad_(True)
    losses = []
    for _ in range(steps):
        h, _ = flce.rms_norm(x, gain, stream)
        loss, kl, n_valid = flce.topk_distill_loss(h, head, ids, logits, lse, targets, tail=True, chunk_rows=4096,
                                                   recompute=False)
        # x's and the stream's gradients would go on into the layers below
        d_x, d_stream, d_gain, d_head = torch.autograd.grad(loss, (x, stream, gain, head))
        with torch.no_grad():
            gain -= lr * d_gain
            head -= (lr * d_head.float()).bfloat16()
        losses.append(loss.detach())
    return torch.stack(losses), gain.detach(), head.detach()


def quantised_head(W):
    """(W8, scales) of the head, made once."""
    W8 = torch.empty(W.shape, dtype=torch.uint8, device=W.device)
    scale = torch.empty(W.shape[0], device=W.device)
    _lib.check("flce_quantize_e4m3_rows", _lib.flce_quantize_e4m3_rows(W, *W.shape, W8, scale))
    return W8, scale


def score(x, stream, gain, W8, W_scale, targets):
    """Log-probs of the targets [N] by the e4m3 head."""
    N, H = x.shape
    out = flce.rms_norm_e4m3(x, gain, stream)
    logp = torch.empty(N, device=x.device)
    _lib.check("flce_forward_e4m3", _lib.flce_forward_e4m3(out["q"], out["scale"], W8, W_scale, targets, None, N, H,
                                                           W8.shape[0], 256, flce.IGNORE_INDEX, None, logp, None, None,
                                                           None))
    return logp, out


def main(tokens: int = 1000, hidden: int = 512, vocab: int = 8000, k: int = 32, steps: int = 8, seed: int = 0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(tokens, hidden, generator=g, device="cuda").bfloat16()
    stream = torch.randn(tokens, hidden, generator=g, device="cuda").bfloat16()
    W = (0.05 * torch.randn(vocab, hidden, generator=g, device="cuda")).bfloat16()
    targets = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
    targets[: tokens // 4] = flce.IGNORE_INDEX  # a prompt without loss
    losses, gain, head = train(x, stream, W, stored_teacher(x, W, k, g), targets, steps)
    W8, W_scale = quantised_head(head)
    logp, normed = score(x, stream, gain, W8, W_scale, targets)
    return {"losses": losses, "logp": logp, "normed": normed, "W8": W8, "W_scale": W_scale, "targets": targets}


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=1000)
    ap.add_argument("--hidden", type=int, default=512)
    ap.add_argument("--vocab", type=int, default=8000)
    ap.add_argument("--steps", type=int, default=8)
    a = ap.parse_args()
    r = main(a.tokens, a.hidden, a.vocab, steps=a.steps)
    print("distillation loss per step:", " ".join(f"{v:.4f}" for v in r["losses"].tolist()))
    kept = r["targets"] != flce.IGNORE_INDEX
    print(f"mean log-prob of {int(kept.sum())} targets by the e4m3 head: {float(r['logp'][kept].mean()):.4f}")
