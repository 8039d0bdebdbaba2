"""The distillation from top logits in 64 bits, from the teacher's distribution
over the whole vocabulary, and the error bounds its tests use."""
import math

import torch


def transform(z, tf):
    """(u, du/dz) of the logit transform."""
    if tf is None:
        return z, torch.ones_like(z)
    s = (tf.get("scale_multiply") or 1.0) / (tf.get("scale_divide") or 1.0)
    T, cap = tf.get("temperature", 1.0), tf.get("softcap", 0.0)
    if cap:
        t = torch.tanh(s * z / cap)
        return cap * t / T, s / T * (1 - t * t)
    return s * z / T, torch.full_like(z, s / T)


def teacher(ids, logits, lse_t, V):
    """(q[N,V], listed[N,V], counted[N]): the teacher's mass per word."""
    N, K = ids.shape
    ids, t = ids.long(), logits.double()
    keep = (ids >= 0) & (ids < V)
    t = torch.where(keep, t, -math.inf)
    lt = t.logsumexp(1) if lse_t is None else lse_t.double()
    p = torch.where(keep, (t - lt[:, None]).exp(), 0.0).nan_to_num(0.0)
    at = torch.where(keep, ids, V)
    q = torch.zeros(N, V + 1, dtype=torch.float64, device=ids.device).scatter_add_(1, at, p)
    seen = torch.zeros(N, V + 1, dtype=torch.float64, device=ids.device).scatter_add_(1, at, torch.ones_like(p))
    counted = keep.any(1) if lse_t is not None else keep.any(1) & (t.amax(1) > -math.inf)
    return q[:, :V], seen[:, :V] > 0, counted


def loss_terms(z, q, listed, tail, tf):
    """(kl, lse, D before weights, parts) per row from the logits z in 64 bits."""
    u, du = transform(z, tf)
    lse = u.logsumexp(1)
    p = (u - lse[:, None]).exp()
    P = q.sum(1)
    rest_lse = torch.where(listed, -math.inf, u).logsumexp(1)
    R = (rest_lse - lse).exp()
    T = torch.where(R > 0, (1 - P).clamp(min=0), 0.0) if tail else torch.zeros_like(P)
    kl = (torch.special.xlogy(q, q) - torch.where(q > 0, q * (u - lse[:, None]), 0.0)).sum(1)
    kl = kl + torch.where(T > 0, torch.special.xlogy(T, T) - T * (rest_lse - lse), 0.0)
    M = P + T
    inside = M[:, None] * p - q
    outside = torch.where(R > 0, M * R - T, 0.0)[:, None] * (u - rest_lse[:, None]).exp().nan_to_num(0.0)
    D = torch.where(listed, inside, outside) * du
    size = torch.where(listed, M[:, None] * p + q, (M * R + T)[:, None] * (u - rest_lse[:, None]).exp().nan_to_num(0.0))
    return kl, lse, D, size * du


def reference(h, W, ids, logits, lse_t=None, targets=None, weights=None, tail=False, tf=None, ignore=-100):
    h, W = h.detach().double(), W.detach().double()
    N, V = h.shape[0], W.shape[0]
    z = h @ W.t()
    q, listed, counted = teacher(ids, logits, lse_t, V)
    kl, lse, D, size = loss_terms(z, q, listed, tail, tf)
    m = counted if targets is None else counted & (targets != ignore)
    w = torch.ones(N, dtype=torch.float64, device=h.device) if weights is None else weights.double()
    n = int(m.sum())
    kl = torch.where(m, kl, 0.0)
    g = torch.where(m, w / max(n, 1), 0.0)[:, None]
    # rounding of a logit: H products summed in fp32, 16 to a step, each step
    # cut to 24 bits of the running sum
    H = h.shape[1]
    mag = (h.abs() @ W.abs().t()).amax(1)
    slope = 1.0 if tf is None else (tf.get("scale_multiply") or 1.0) / (tf.get("scale_divide") or 1.0) / tf.get("temperature", 1.0)
    zerr = (H / 16 + 4) * 2.0 ** -23 * mag * slope
    # of a log-sum-exp on top: exp2 to 2^-22, V terms added 32 at a time, one
    # rounding of the 32-bit result
    lerr = zerr + 2.0 ** -22 + (V / 32 + 64) * 2.0 ** -24 + 2.0 ** -23 * (1 + lse.abs())
    if tf is not None and tf.get("softcap"):
        lerr = lerr + 2.0 ** -21 * tf["softcap"] / tf.get("temperature", 1.0)  # tanhf
    return dict(kl=kl, lse=lse, loss=float((kl * w).sum() / max(n, 1)), n_valid=n, D=D * g, dH=(D * g) @ W,
                dW=(D * g).t() @ h, size=size * g.abs(), lerr=lerr, h=h, W=W, w=w)


def check(got, ref, roundings=1, what=""):
    """got: kl, lse (or None), loss, n_valid, dH, dW (each may be missing)."""
    def within(x, want, bound, name):
        x = x.double()
        bad = ~((x - want).abs() <= bound)
        assert not bool(bad.any()), (what, name, int(bad.sum()), float((x - want).abs().max()), float(bound.max()))

    # a kl takes mass of at most two from logits and two log-sum-exps, its
    # masses to 2^-22 of logs of at most 2^7
    klerr = 4 * ref["lerr"] + 2.0 ** -14 * 2.0 ** -7 + 2.0 ** -20 * ref["kl"].abs()
    if got.get("lse") is not None:
        within(got["lse"], ref["lse"], ref["lerr"], "lse")
    if got.get("kl") is not None:
        within(got["kl"], ref["kl"], klerr, "kl")
    if got.get("n_valid") is not None:
        assert int(got["n_valid"]) == ref["n_valid"], what
    if got.get("loss") is not None:
        bound = float((klerr * ref["w"].abs()).sum()) / max(ref["n_valid"], 1)
        assert abs(float(got["loss"]) - ref["loss"]) <= bound, (what, float(got["loss"]), ref["loss"], bound)
    # D: `roundings` half steps of bf16 (2^-8; the one-call step stores its
    # exponentials in bf16 first), its masses to the log-sum-exps' errors
    B = ref["D"].abs() * (roundings * 2.0 ** -8) + ref["size"] * (3 * ref["lerr"][:, None] + 2.0 ** -20)
    V, N = ref["D"].shape[1], ref["D"].shape[0]
    for name, sums, want in (("dH", lambda x: x @ ref["W"].abs(), ref["dH"]),
                             ("dW", lambda x: x.t() @ ref["h"].abs(), ref["dW"])):
        if got.get(name) is None:
            continue
        terms = V if name == "dH" else N
        bound = sums(B) + sums(ref["D"].abs()) * (terms / 16 + 32) * 2.0 ** -23
        step = 2.0 ** -8 if got[name].dtype == torch.bfloat16 else 2.0 ** -24
        within(got[name], want, 1.02 * bound + step * (want.abs() + bound) + 1e-30, name)
        # and in all, where the roundings do not all point one way: the
        # gradient tolerance of the other losses' tests
        norm = float(want.norm())
        if norm > 0:
            assert float((got[name].double() - want).norm()) <= 1e-2 * norm, (what, name)
