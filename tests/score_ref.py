"""The scores' definition in 64 bits: log-probability, entropy, likeliest words
and their gradients, and how far 32-bit kernels can be off."""
import math

import torch

IGNORE = -100


def transformed(z, tf):
    """(f(z), f'(z))"""
    tf = tf or {}
    s = (tf.get("scale_multiply") or 1.0) / (tf.get("scale_divide") or 1.0)
    cap, T = tf.get("softcap") or 0.0, tf.get("temperature", 1.0)
    if not cap:
        return z * s / T, torch.full_like(z, s / T)
    t = torch.tanh(z * s / cap)
    return t * cap / T, (1 - t * t) * s / T


def live(h, targets):
    n = torch.ones(h.shape[0], dtype=torch.bool, device=h.device)
    return n if targets is None else targets != IGNORE


def reference(h, W, targets=None, k=0, tf=None):
    """dict of 64-bit values; "z", "u", "slope", "logq" are [N, V]."""
    z = h.double() @ W.double().t()
    u, slope = transformed(z, tf)
    lse = u.logsumexp(1)
    logq = u - lse[:, None]
    q = logq.exp()
    on = live(h, targets)
    out = dict(z=z, u=u, slope=slope, logq=logq, q=q, on=on, entropy=torch.where(on, -(q * logq).sum(1), 0.0),
               lse=torch.where(on, lse, 0.0))
    if targets is not None:
        at = targets.clamp(min=0)[:, None]
        out["logp"] = torch.where(on, logq.gather(1, at)[:, 0], 0.0)
    if k:
        best, ids = z.sort(dim=1, descending=True, stable=True)
        out["ids"] = torch.where(on[:, None], ids[:, :k], -1)
        out["logprobs"] = torch.where(on[:, None], logq.gather(1, ids[:, :k]), 0.0)
    return out


def logit_error(h, r, tf=None):
    """[N] how far a 32-bit u can be off.  z: every step of 16 products cuts the
    running sum, at most twice the row's largest logit, by less than 2^-23 of it
    (the few-row sums are rounded, which is less).  u: the two factors and tanh (2
    units in the last place) on top, at most 2^-20 of the largest."""
    steps = math.ceil(h.shape[1] / 16)
    return r["slope"].amax(1) * steps * 2.0 ** -22 * r["z"].abs().amax(1) + 2.0 ** -20 * r["u"].abs().amax(1)


def bounds(h, r, tf=None):
    """dict(lse, logp, logprobs [N,1], entropy): u's error, and of the sums (2^-22 an
    exponential, and the sums' and logarithm's roundings) 2^-19 of 1 and of the
    result.  The entropy's slope in u is p |log p + entropy|."""
    e = logit_error(h, r, tf)
    lse = e + 2.0 ** -19 * (1 + r["lse"].abs())
    slope = (r["q"] * (r["logq"] + r["entropy"][:, None]).abs()).sum(1)
    return dict(lse=lse, logp=lse + e, logprobs=(lse + e)[:, None],
                entropy=(e + 2.0 ** -20) * slope + 2.0 ** -19 * (1 + r["entropy"]))


def dlogits(r, targets, ga, ge):
    """D [N, V]: the gradient of sum ga logp + ge entropy in z."""
    on = r["on"]
    zero = torch.zeros(r["q"].shape[0], dtype=torch.float64, device=r["q"].device)
    ga = (zero if ga is None else torch.where(on, ga.double(), 0.0))[:, None]
    ge = (zero if ge is None else torch.where(on, ge.double(), 0.0))[:, None]
    V = r["q"].shape[1]
    inside = (targets >= 0) & (targets < V)
    onehot = torch.zeros_like(r["q"]).scatter_(1, targets.clamp(0, V - 1)[:, None], 1.0) * inside[:, None]
    D = ga * (onehot - r["q"]) - ge * r["q"] * (r["logq"] + r["entropy"][:, None])
    return D * r["slope"], onehot


def check(out, h, W, targets, r, k=0, tf=None, what=""):
    b = bounds(h, r, tf)
    for name in ("lse", "logp", "logprobs", "entropy"):
        if out.get(name) is None:
            continue
        on = r["on"] if out[name].dim() == 1 else r["on"][:, None]
        err = (out[name].double() - r[name]).abs()
        assert bool((err <= torch.where(on, b[name], 0.0)).all()), (what, name, float(err.max()))
    if k:
        same = out["ids"] == r["ids"]
        assert bool(same.all()), (what, "ids", int((~same).sum()))


def chunk_distance(u):
    """[N, V] how far each u is below the largest of its 32 columns."""
    N, V = u.shape
    pad = torch.nn.functional.pad(u, (0, -V % 32), value=-math.inf).view(N, -1, 32)
    return (pad.amax(2, keepdim=True) - pad).view(N, -1)[:, :V]


def check_grads(dH, dW, h, W, targets, r, ga, ge, tf=None, what="", kept=False):
    """Against D W and D^T h: D rounded to bf16 once (2^-8 of each value, half a
    step) after the errors of p and log p, the sums' cuts, the outputs' rounding.
    kept: logits in fp16 relative to the largest of their 32 columns (2^-11 of that
    distance, and 2^-25 where it is below fp16's range), and the dlogits of at
    most 128 rows in two parts (2^-16)."""
    D, onehot = dlogits(r, targets, ga, ge)
    on = r["on"][:, None]
    e = logit_error(h, r, tf)[:, None]
    mag = lambda g: 0.0 if g is None else torch.where(on, g.double().abs()[:, None], 0.0)  # noqa: E731
    # p's relative error: that of u and lse, and 2^-19 as above; log p's: the same, absolute
    rel = 2 * e + 2.0 ** -18
    half_d = 2.0 ** -8
    if kept:
        rel = rel + 2.0 ** -11 * chunk_distance(r["u"]) + 2.0 ** -24
        half_d = 2.0 ** -16 if h.shape[0] <= 128 else half_d
    terms = r["q"] * (mag(ga) + mag(ge) * ((r["logq"] + r["entropy"][:, None]).abs() + 1)) * r["slope"]
    # (a soft-cap's slope, 1 - tanh^2, loses bits where tanh is near 1: 2^-21 of 1)
    if tf and tf.get("softcap"):
        terms = terms + (r["q"] * mag(ge) * (r["logq"].abs() + 1) + (r["q"] + onehot) * mag(ga)) * 2.0 ** -2 / tf.get(
            "temperature", 1.0)
    dD = 1.01 * half_d * D.abs() + rel * terms
    for name, got, want, err, absolute in (
            ("dH", dH, D @ W.double(), dD @ W.double().abs(), D.abs() @ W.double().abs()),
            ("dW", dW, D.t() @ h.double(), dD.t() @ h.double().abs(), D.t().abs() @ h.double().abs())):
        if got is None:
            continue
        steps = math.ceil((D.shape[1] if name == "dH" else D.shape[0]) / 16)
        half = torch.finfo(got.dtype).eps / 2
        bound = err + steps * 2.0 ** -23 * absolute + 1.01 * half * want.abs() + 1e-30
        bad = ~((got.double() - want).abs() <= bound)
        assert not bool(bad.any()), (what, name, int(bad.sum()), float((got.double() - want).abs().max()))
