"""Measured cases of the LM head's norm and of the distillation from a teacher's top logits.

Three operators, the steps between a model's residual stream and its loss:

  norm       root-mean-square norm of x, or of the residual stream with x added to it: forward, or forward and backward
  norm_e4m3  the same with an 8-bit (e4m3) output and one scale per row, the operand form of the e4m3 head
  distill    loss of the student head h W^T against a teacher's stored top logits: forward, or forward and backward

``own`` selects the side of ``run``: False computes the operators from elementary torch operations in 32 bits, True
calls this package.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
IGNORE = -100


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the final norm of one decoded token: nothing but latency
        dict(name="norm_token", op="norm", train=False, N=1, H=4096, residual="bf16", weight="bf16", offset=0.0),
        # the final norm of a 16,384-token training step at hidden size 4,096
        dict(name="norm_train_16k", op="norm", train=True, N=16384, H=4096, residual="bf16", weight="bf16", offset=0.0),
        # a ragged batch, a residual stream and gain held in 32 bits, the gain stored as its distance from one
        dict(name="norm_train_odd_f32", op="norm", train=True, N=1003, H=1000, residual="f32", weight="f32", offset=1.0),
        # the long-context step, 131,072 tokens at hidden size 2,560, no residual to add
        dict(name="norm_train_131k", op="norm", train=True, N=131072, H=2560, residual="none", weight="bf16", offset=0.0),
        # scoring a few sampled tokens with the e4m3 head
        dict(name="norm_e4m3_few", op="norm_e4m3", N=8, H=2048, residual="bf16", weight="bf16", offset=0.0, strided=False),
        # scoring 32,768 rollout tokens at hidden size 4,096 (old-policy or reference log-probs)
        dict(name="norm_e4m3_32k", op="norm_e4m3", N=32768, H=4096, residual="bf16", weight="bf16", offset=0.0, strided=False),
        # rows taken out of a wider buffer, an odd count of them
        dict(name="norm_e4m3_odd", op="norm_e4m3", N=777, H=2064, residual="f32", weight="f32", offset=0.0, strided=True),
        # the smallest training step of the test workloads
        dict(name="distill_tiny", op="distill", train=True, N=64, H=64, V=1000, K=16, tail=False, masked=False,
             logits="f32", ids="i64", temperature=1.0),
        # one token scored against the teacher's stored logits
        dict(name="distill_token", op="distill", train=False, N=1, H=4096, V=151936, K=64, tail=False, masked=False,
             logits="f32", ids="i64", temperature=1.0),
        # one 256-row chunk over a 248,320-word vocabulary
        dict(name="distill_chunk_256", op="distill", train=True, N=256, H=2048, V=248320, K=128, tail=False, masked=False,
             logits="bf16", ids="i32", temperature=1.0),
        # packed prompts without loss, per-token weights, stored lists of unequal length, the rest of the teacher's
        # mass as one more outcome
        dict(name="distill_masked_odd", op="distill", train=True, N=1501, H=1096, V=32003, K=37, tail=True, masked=True,
             logits="f32", ids="i64", temperature=2.0),
        # a training step of 4,096 tokens at hidden size 4,096 and 151,936 words
        dict(name="distill_train_4k", op="distill", train=True, N=4096, H=4096, V=151936, K=64, tail=False, masked=False,
             logits="bf16", ids="i32", temperature=1.0),
    ]


def _log_between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_e4m3", "distill", "distill"])
    if op != "distill":
        H = 16 * _log_between(rng, 4, 512)
        N = min(_log_between(rng, 1, 32768), 131072 * 2560 // H)
        case = dict(op=op, N=N, H=H, residual=rng.choice(["none", "bf16", "f32"]), weight=rng.choice(["bf16", "f32"]),
                    offset=rng.choice([0.0, 1.0]))
        if op == "norm":
            return dict(case, train=rng.random() < 0.6)
        return dict(case, strided=rng.random() < 0.3)
    V = _log_between(rng, 1000, 151936)
    return dict(op=op, train=rng.random() < 0.7, N=_log_between(rng, 1, 4096), H=8 * _log_between(rng, 8, 512), V=V,
                K=_log_between(rng, 1, 128), tail=rng.random() < 0.5, masked=rng.random() < 0.5,
                logits=rng.choice(["bf16", "f32"]), ids=rng.choice(["i32", "i64"]),
                temperature=rng.choice([1.0, 1.0, 2.0]))


def _prompt_rows(case):
    return case["N"] // 4 if case["masked"] else 0


def _has(case):
    return case["residual"] != "none"


def work(case):
    """The bytes and operations of one pass: each input read once, each output written once."""
    N, H = case["N"], case["H"]
    if case["op"] == "distill":
        V, K, rows = case["V"], case["K"], case["N"] - _prompt_rows(case)
        entry = (2 if case["logits"] == "bf16" else 4) + (4 if case["ids"] == "i32" else 8)
        head = 2 * V * H
        if not case["train"]:
            return {"bytes": head + 2 * rows * H + rows * K * entry + 8 * N, "flops": 2 * rows * V * H}
        return {"bytes": 2 * head + 2 * (rows + N) * H + rows * K * entry + 8 * N, "flops": 6 * rows * V * H}
    r = {"none": 0, "bf16": 2, "f32": 4}[case["residual"]]
    w = 2 if case["weight"] == "bf16" else 4
    forward = N * H * (2 + 2 * r) + w * H
    if case["op"] == "norm_e4m3":
        return {"bytes": forward + N * H + 4 * N, "flops": 6 * N * H}
    forward += 2 * N * H
    if not case["train"]:
        return {"bytes": forward, "flops": 5 * N * H}
    s = r or 2
    # dy and the stream are read, and the stream's own gradient where there is one; dx is written, and the residual's
    # gradient where its type is another than dx's
    back = N * H * (2 + s + r + 2 + (4 if r == 4 else 0)) + 2 * w * H
    return {"bytes": forward + back, "flops": 14 * N * H}


# ----------------------------------------------------------------- inputs

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "i32": torch.int32, "i64": torch.int64}


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _stream(g, N, H, kind):
    """A residual stream: unit scale, a few channels far larger than the others."""
    x = _normal(g, N, H)
    x[:, :: max(1, H // 4)] *= 20.0
    return x.to(DTYPES[kind])


def _prepare_norm(case, g):
    N, H = case["N"], case["H"]
    st = dict(case=case)
    if case["op"] == "norm_e4m3" and case["strided"]:
        st["x"] = _normal(g, N, H + 48).bfloat16()[:, 16:16 + H]
    else:
        st["x"] = _normal(g, N, H).bfloat16()
    st["residual"] = _stream(g, N, H, case["residual"]) if _has(case) else None
    st["weight"] = (1.0 - case["offset"] + 0.1 * _normal(g, H)).to(DTYPES[case["weight"]])
    if case.get("train"):
        st["dy"] = (0.01 * _normal(g, N, H)).bfloat16()
        st["ds"] = (0.01 * _normal(g, N, H)).to(DTYPES[case["residual"]]) if _has(case) else None
        for k in ("x", "residual", "weight"):
            if st[k] is not None:
                st[k].requires_grad_(True)
    return st


def _prepare_distill(case, g):
    N, H, V, K = case["N"], case["H"], case["V"], case["K"]
    h = _normal(g, N, H).bfloat16()
    W = (0.02 * _normal(g, V, H)).bfloat16()
    # the teacher agrees with the student in part and is surer of its words
    ht = (0.7 * h.float() + 0.7 * _normal(g, N, H)).bfloat16()
    ids = torch.empty(N, K, dtype=torch.int64, device="cuda")
    logits = torch.empty(N, K, device="cuda")
    lse_t = torch.empty(N, device="cuda")
    for a in range(0, N, 1024):
        z = (ht[a:a + 1024] @ W.t()).float()
        z = 2.0 * z / z.std() + 1e-3 * torch.rand(z.shape, generator=g, device="cuda")
        logits[a:a + 1024], ids[a:a + 1024] = z.topk(K, dim=1)
        lse_t[a:a + 1024] = z.logsumexp(1)
    targets = weights = None
    if case["masked"]:
        targets = torch.zeros(N, dtype=torch.int64, device="cuda")
        targets[: _prompt_rows(case)] = IGNORE
        weights = torch.rand(N, generator=g, device="cuda") + 0.5
        kept = torch.randint(0, K + 1, (N, 1), generator=g, device="cuda")  # some rows keep nothing
        kept[N - 1] = K
        ids[torch.arange(K, device="cuda")[None, :] >= kept] = -1
    st = dict(case=case, h=h, W=W, ids=ids.to(DTYPES[case["ids"]]), logits=logits.to(DTYPES[case["logits"]]),
              lse_t=lse_t if case["tail"] else None, targets=targets, weights=weights)
    if case["train"]:
        h.requires_grad_(True)
        W.requires_grad_(True)
    return st


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return _prepare_distill(case, g) if case["op"] == "distill" else _prepare_norm(case, g)


# ------------------------------------------------- the framework's kernels

def _run_own(st):
    import chunked_lm_head_gb300 as flce
    c = st["case"]
    if c["op"] == "distill":
        tf = {"temperature": c["temperature"]} if c["temperature"] != 1.0 else None
        args = dict(lse_t=st["lse_t"], targets=st["targets"], weights=st["weights"], tail=c["tail"], transform=tf)
        if not c["train"]:
            out = flce.topk_kd_forward(st["h"], st["W"], st["ids"], st["logits"], **args)
            return {"loss": out["loss"], "kl": out["kl"], "lse": out["lse"], "n_valid": out["n_valid"]}
        loss, kl, n_valid = flce.topk_distill_loss(st["h"], st["W"], st["ids"], st["logits"], chunk_rows=4096,
                                                   recompute=False, **args)
        dh, dW = torch.autograd.grad(loss, (st["h"], st["W"]))
        return {"loss": loss, "kl": kl, "n_valid": n_valid, "dh": dh, "dW": dW}
    if c["op"] == "norm_e4m3":
        out = flce.rms_norm_e4m3(st["x"], st["weight"], st["residual"], weight_offset=c["offset"])
        q = {"q": out["q"], "scale": out["scale"]}
        return dict(q, residual=out["residual"]) if _has(c) else q
    if not _has(c):
        y = flce.rms_norm(st["x"], st["weight"], weight_offset=c["offset"])
        if not c["train"]:
            return {"y": y}
        dx, dw = torch.autograd.grad(y, (st["x"], st["weight"]), st["dy"])
        return {"y": y, "dx": dx, "dw": dw}
    y, s = flce.rms_norm(st["x"], st["weight"], st["residual"], weight_offset=c["offset"])
    if not c["train"]:
        return {"y": y, "residual": s}
    dx, dr, dw = torch.autograd.grad((y, s), (st["x"], st["residual"], st["weight"]), (st["dy"], st["ds"]))
    return {"y": y, "residual": s, "dx": dx, "dr": dr, "dw": dw}


# ----------------------------------------------------------- the plain form

EPS = 1e-6


def _plain_norm(st):
    c = st["case"]
    x, w = st["x"].detach(), st["weight"].detach().float() + c["offset"]
    if _has(c):
        # the norm sees the stream as it is stored
        s = (x.float() + st["residual"].detach().float()).to(st["residual"].dtype)
    else:
        s = x
    sf = s.float()
    rstd = torch.rsqrt((sf * sf).mean(1, keepdim=True) + EPS)
    xhat = sf * rstd
    y = xhat * w
    if c["op"] == "norm_e4m3":
        scale = y.abs().amax(1) / E4M3_MAX
        scale = torch.where(scale > 0, scale, torch.ones_like(scale))
        q = {"q": (y / scale[:, None]).to(torch.float8_e4m3fn), "scale": scale}
        return dict(q, residual=s) if _has(c) else q
    out = {"y": y.to(x.dtype)}
    if _has(c):
        out["residual"] = s
    if not c["train"]:
        return out
    dy = st["dy"].float()
    g = dy * w
    ds = rstd * (g - xhat * (g * xhat).mean(1, keepdim=True))
    if _has(c):
        ds = ds + st["ds"].float()
        out["dr"] = ds.to(st["residual"].dtype)
    out["dx"] = ds.to(x.dtype)
    out["dw"] = (dy * xhat).sum(0).to(st["weight"].dtype)
    return out


def _plain_distill(st):
    c = st["case"]
    h, W = st["h"].detach(), st["W"].detach()
    hf, Wf = h.float(), W.float()
    ids, N = st["ids"].long(), c["N"]
    keep = ids >= 0
    at = ids.clamp(min=0)
    m = keep.any(1)
    if st["targets"] is not None:
        m = m & (st["targets"] != IGNORE)
    # the teacher's few numbers in 64 bits: the rest of its mass is one less their sum
    t = torch.where(keep, st["logits"].double(), -math.inf)
    lt = st["lse_t"].double() if st["lse_t"] is not None else torch.where(m, t.logsumexp(1), 0.0)
    logpt = t - lt[:, None]
    pt = logpt.exp()
    P = pt.sum(1)
    T = (1.0 - P).clamp(min=0.0) if c["tail"] else torch.zeros_like(P)
    u = hf @ Wf.t()
    if c["temperature"] != 1.0:
        u = u / c["temperature"]
    uk = u.gather(1, at)
    lse = u.logsumexp(1)
    # the student's mass outside the list, summed by itself
    inside = torch.zeros_like(u, dtype=torch.uint8).scatter_add_(1, at, keep.to(torch.uint8)) > 0
    lse_rest = u.masked_fill(inside, -math.inf).logsumexp(1)
    cross = torch.where(pt > 0, pt * (logpt - (uk - lse[:, None]).double()), 0.0).sum(1)
    rest = torch.where(T > 0, T * (T.log() - (lse_rest - lse).double()), 0.0)
    kl = torch.where(m, cross + rest, 0.0)
    n_valid = m.sum()
    w = st["weights"] if st["weights"] is not None else torch.ones(N, device=h.device)
    out = {"kl": kl.float(), "loss": ((kl * w).sum() / n_valid.clamp(min=1)).float(), "n_valid": n_valid}
    if not c["train"]:
        return dict(out, lse=lse)
    scale = torch.where(m, w / n_valid.clamp(min=1), 0.0) / c["temperature"]
    D = (u - lse[:, None]).exp() * (P + T).float()[:, None]
    if c["tail"]:
        D -= torch.where(inside, 0.0, (u - lse_rest[:, None]).exp() * T.float()[:, None])
    D.scatter_add_(1, at, -torch.where(keep, pt, 0.0).float())
    D *= scale[:, None]
    out["dh"] = (D @ Wf).to(h.dtype)
    out["dW"] = (D.t() @ hf).to(W.dtype)
    return out


def run(st):
    if own:
        return _run_own(st)
    return _plain_distill(st) if st["case"]["op"] == "distill" else _plain_norm(st)


# ---------------------------------------------------- the values in 64 bits

def _exact_norm(st):
    c = st["case"]
    x, gain = st["x"].detach().double(), st["weight"].detach().double() + c["offset"]
    s = x
    if _has(c):
        kind = st["residual"].dtype
        s = (x + st["residual"].detach().double()).to(kind).double()
    H = c["H"]
    sq = torch.einsum("nh,nh->n", s, s) / H + EPS
    inv = sq.pow(-0.5)
    y = torch.einsum("nh,n,h->nh", s, inv, gain)
    out = {"residual": s} if _has(c) else {}
    if c["op"] == "norm_e4m3":
        top = y.abs().max(1).values
        scale = torch.where(top == 0, 1.0, top / E4M3_MAX)
        return dict(out, q=y / scale[:, None], scale=scale)
    out["y"] = y
    if not c["train"]:
        return out
    dy = st["dy"].double()
    # d/ds of y = s (|s|^2 / H + eps)^(-1/2) gain
    along = torch.einsum("nh,nh,h->n", dy, s, gain) * inv.pow(3) / H
    ds = torch.einsum("nh,h,n->nh", dy, gain, inv) - s * along[:, None]
    if _has(c):
        ds = ds + st["ds"].double()
        out["dr"] = ds
    out["dx"] = ds
    out["dw"] = torch.einsum("nh,nh,n->h", dy, s, inv)
    return out


def _exact_distill(st):
    c = st["case"]
    N, V, K = c["N"], c["V"], c["K"]
    h, W = st["h"].detach().double(), st["W"].detach().double()
    ids = st["ids"].long()
    live = torch.ones(N, dtype=torch.bool, device="cuda") if st["targets"] is None else st["targets"].ne(IGNORE)
    live = live & (ids.max(1).values >= 0)
    count = int(live.sum())
    w = torch.ones(N, dtype=torch.float64, device="cuda") if st["weights"] is None else st["weights"].double()
    kl = torch.zeros(N, dtype=torch.float64, device="cuda")
    lse = torch.zeros(N, dtype=torch.float64, device="cuda")
    dh, dW = torch.zeros_like(h), torch.zeros_like(W) if c["train"] else None
    for a in range(0, N, 512):
        b = slice(a, min(N, a + 512))
        u = h[b] @ W.t() / c["temperature"]
        top = u.max(1, keepdim=True).values
        e = (u - top).exp()
        mass = e.sum(1, keepdim=True)
        lse[b] = (top + mass.log())[:, 0]
        p = e / mass
        # the teacher's distribution over all words; a column past the last takes the entries that are none
        q = torch.zeros(p.shape[0], V + 1, dtype=torch.float64, device="cuda")
        seen = torch.zeros_like(q)
        where = torch.where(ids[b] < 0, V, ids[b])
        x = st["logits"][b].double()
        if st["lse_t"] is not None:
            val = (x - st["lse_t"][b].double()[:, None]).exp()
        else:
            xm = torch.where(ids[b] < 0, -1e300, x)
            val = (xm - xm.max(1, keepdim=True).values).exp()
            val = val / val.sum(1, keepdim=True)
        q.scatter_add_(1, where, val)
        seen.scatter_add_(1, where, torch.ones_like(val))
        q, listed_ = q[:, :V], seen[:, :V] > 0
        rest_t = (1.0 - q.sum(1)).clamp(min=0.0) if c["tail"] else torch.zeros(p.shape[0], dtype=torch.float64, device="cuda")
        rest_s = torch.where(listed_, 0.0, p).sum(1)
        logp = u - lse[b][:, None]
        row = (torch.special.xlogy(q, q) - torch.where(q > 0, q * logp, 0.0)).sum(1)
        row = row + torch.special.xlogy(rest_t, rest_t) - torch.special.xlogy(rest_t, rest_s)
        kl[b] = torch.where(live[b], row, 0.0)
        if c["train"]:
            D = p * (q.sum(1) + rest_t)[:, None] - q
            D = D - torch.where(listed_, 0.0, p) * torch.where(rest_t > 0, rest_t / rest_s, 0.0)[:, None]
            D = torch.where(live[b][:, None], D * (w[b] / max(1, count) / c["temperature"])[:, None], 0.0)
            dh[b] = D @ W
            dW += D.t() @ h[b]
    out = {"kl": kl, "loss": (kl * w).sum() / max(1, count), "n_valid": None}
    return dict(out, dh=dh, dW=dW) if c["train"] else dict(out, lse=lse)


def exact(case, seed):
    if case["op"] == "distill" and work(case)["flops"] > 6e12:
        return None  # the products in 64 bits take a quarter of a minute and more
    st = prepare(case, seed)
    return _exact_distill(st) if case["op"] == "distill" else _exact_norm(st)
