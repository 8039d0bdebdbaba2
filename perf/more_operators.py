"""Measured cases of the layer norm in front of the head and of what the head's distribution is read for.

Three operators, the steps between a model's residual stream and its words:

  layer    layer norm of x, or of the residual stream with x added to it: forward, or forward and backward
  entropy  log-probability of given tokens and entropy of the head's distribution softmax(f(h W^T)): forward, or forward
           and backward (policy losses with an entropy term)
  top      the K likeliest words of the head with their log-probabilities, beside log-sum-exp and entropy (alternatives
           shown to a user, lists stored of a teacher)

``own`` selects the side of ``run``: False computes the operators from elementary torch operations, True calls this
package.
"""
import math

import torch

own = False

IGNORE = -100
EPS = 1e-5


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the final norm of one decoded token: nothing but latency
        dict(name="layer_token", op="layer", train=False, N=1, H=4096, residual="bf16", weight="bf16", bias=True),
        # the final norm of a 16,384-token training step at hidden size 4,096
        dict(name="layer_train_16k", op="layer", train=True, N=16384, H=4096, residual="bf16", weight="bf16", bias=True),
        # a ragged batch, the residual stream and the parameters held in 32 bits
        dict(name="layer_train_odd_f32", op="layer", train=True, N=1003, H=1000, residual="f32", weight="f32", bias=True),
        # the long-context step, 131,072 tokens at hidden size 2,560, no residual to add, a norm without a bias
        dict(name="layer_train_131k", op="layer", train=True, N=131072, H=2560, residual="none", weight="bf16", bias=False),
        # the smallest training step of the test workloads
        dict(name="entropy_tiny", op="entropy", train=True, N=64, H=64, V=1000, masked=False, softcap=0.0, temperature=1.0),
        # one 256-row chunk over a 248,320-word vocabulary
        dict(name="entropy_chunk_256", op="entropy", train=True, N=256, H=2048, V=248320, masked=False, softcap=0.0,
             temperature=1.0),
        # packed prompts without loss, a soft-cap and a temperature
        dict(name="entropy_masked_odd", op="entropy", train=True, N=1501, H=1096, V=32003, masked=True, softcap=30.0,
             temperature=0.7),
        # a policy step of 4,096 tokens at hidden size 4,096 and 151,936 words
        dict(name="entropy_train_4k", op="entropy", train=True, N=4096, H=4096, V=151936, masked=False, softcap=0.0,
             temperature=1.0),
        # the alternatives of one decoded token
        dict(name="top_token", op="top", N=1, H=4096, V=151936, K=20, masked=False, softcap=0.0, temperature=1.0),
        # the alternatives of a small batch that decodes
        dict(name="top_decode_33", op="top", N=33, H=2048, V=248320, K=5, masked=False, softcap=0.0, temperature=0.7),
        # a scored conversation whose prompt needs no alternatives
        dict(name="top_masked_odd", op="top", N=777, H=1096, V=32003, K=37, masked=True, softcap=30.0, temperature=1.0),
        # a teacher's lists for 4,096 tokens
        dict(name="top_teacher_4k", op="top", N=4096, H=4096, V=151936, K=64, masked=False, softcap=0.0, temperature=1.0),
    ]


def _log_between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["layer", "entropy", "top"])
    if op == "layer":
        H = 8 * _log_between(rng, 8, 1024)
        N = min(_log_between(rng, 1, 32768), 131072 * 2560 // H)
        return dict(op=op, train=rng.random() < 0.6, N=N, H=H, residual=rng.choice(["none", "bf16", "f32"]),
                    weight=rng.choice(["bf16", "f32"]), bias=rng.random() < 0.7)
    V = _log_between(rng, 1000, 151936)
    case = dict(op=op, N=_log_between(rng, 1, 4096), H=8 * _log_between(rng, 8, 512), V=V, masked=rng.random() < 0.5,
                softcap=rng.choice([0.0, 0.0, 30.0]), temperature=rng.choice([1.0, 1.0, 0.7]))
    if op == "entropy":
        return dict(case, train=rng.random() < 0.7)
    return dict(case, K=_log_between(rng, 1, 128))


def _prompt_rows(case):
    return case["N"] // 4 if case["masked"] else 0


def _has(case):
    return case["residual"] != "none"


def work(case):
    """The bytes and operations of one pass: each input read once, each output written once."""
    N, H = case["N"], case["H"]
    if case["op"] != "layer":
        V, rows = case["V"], case["N"] - _prompt_rows(case)
        head = 2 * V * H
        if case["op"] == "top":
            return {"bytes": head + 2 * rows * H + 12 * N * case["K"] + (20 if case["masked"] else 8) * N,
                    "flops": 2 * rows * V * H}
        if not case["train"]:
            return {"bytes": head + 2 * rows * H + 16 * N, "flops": 2 * rows * V * H}
        return {"bytes": 2 * head + 2 * (rows + N) * H + 24 * N, "flops": 6 * rows * V * H}
    r = {"none": 0, "bf16": 2, "f32": 4}[case["residual"]]
    w = (2 if case["weight"] == "bf16" else 4) * (2 if case["bias"] else 1)
    forward = N * H * (4 + 2 * r) + w * H
    if not case["train"]:
        return {"bytes": forward, "flops": 8 * N * H}
    s = r or 2
    # dy and the stream are read, and the stream's own gradient where there is one; dx is written, and the residual's
    # gradient where its type is another than dx's
    back = N * H * (2 + s + r + 2 + (4 if r == 4 else 0)) + 2 * w * H
    return {"bytes": forward + back, "flops": 20 * N * H}


# ----------------------------------------------------------------- inputs

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _prepare_layer(case, g):
    N, H = case["N"], case["H"]
    kind = DTYPES[case["weight"]]
    st = dict(case=case, x=_normal(g, N, H).bfloat16(), residual=None, bias=None, ds=None)
    if _has(case):
        # a residual stream: unit scale about a mean, a few channels far larger than the others
        r = _normal(g, N, H) + 0.5
        r[:, :: max(1, H // 4)] *= 20.0
        st["residual"] = r.to(DTYPES[case["residual"]])
    st["weight"] = (1.0 + 0.1 * _normal(g, H)).to(kind)
    if case["bias"]:
        st["bias"] = (0.1 * _normal(g, H)).to(kind)
    if case["train"]:
        st["dy"] = (0.01 * _normal(g, N, H)).bfloat16()
        if _has(case):
            st["ds"] = (0.01 * _normal(g, N, H)).to(DTYPES[case["residual"]])
        for k in ("x", "residual", "weight", "bias"):
            if st[k] is not None:
                st[k].requires_grad_(True)
    return st


def _prepare_head(case, g):
    N, H, V = case["N"], case["H"], case["V"]
    # normed hidden states; logits of standard deviation 3, a distribution sure of some words
    h = _normal(g, N, H).bfloat16()
    W = (3.0 / math.sqrt(H) * _normal(g, V, H)).bfloat16()
    st = dict(case=case, h=h, W=W, targets=None, transform=None)
    if case["softcap"] or case["temperature"] != 1.0:
        st["transform"] = dict(softcap=case["softcap"], temperature=case["temperature"])
    if case["masked"] or case["op"] == "entropy":
        st["targets"] = torch.randint(0, V, (N,), generator=g, device="cuda")
        st["targets"][: _prompt_rows(case)] = IGNORE
    if case.get("train"):
        # gradients of a loss averaged over the tokens: an advantage per token, and the entropy's coefficient
        st["dlogp"] = _normal(g, N) / N
        st["dentropy"] = -0.5 * torch.rand(N, generator=g, device="cuda") / N
        h.requires_grad_(True)
        W.requires_grad_(True)
    return st


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return _prepare_layer(case, g) if case["op"] == "layer" else _prepare_head(case, g)


# ------------------------------------------------- the framework's kernels

def _run_own(st):
    import chunked_lm_head_gb300 as flce
    c = st["case"]
    if c["op"] == "top":
        out = flce.top_logprobs(st["h"], st["W"], c["K"], targets=st["targets"], transform=st["transform"])
        keys = ("ids", "logprobs", "lse", "entropy") + (("logp",) if c["masked"] else ())
        return {k: out[k] for k in keys}
    if c["op"] == "entropy":
        logp, entropy = flce.selective_log_softmax_entropy(st["h"], st["W"], st["targets"], chunk_rows=4096,
                                                           transform=st["transform"])
        out = {"logp": logp, "entropy": entropy}
        if c["train"]:
            out["dh"], out["dW"] = torch.autograd.grad((logp, entropy), (st["h"], st["W"]), (st["dlogp"], st["dentropy"]))
        return out
    y = flce.layer_norm(st["x"], st["weight"], st["bias"], st["residual"], eps=EPS)
    out = {"y": y}
    if _has(c):
        out = {"y": y[0], "residual": y[1]}
    if c["train"]:
        names = [k for k in ("x", "residual", "weight", "bias") if st[k] is not None]
        grads = torch.autograd.grad(y, [st[k] for k in names], (st["dy"], st["ds"]) if _has(c) else st["dy"])
        out.update({"d" + k: d for k, d in zip(names, grads)})
    return out


# ----------------------------------------------------------- the plain form

def _plain_layer(st):
    c = st["case"]
    x, w = st["x"].detach(), st["weight"].detach().float()
    s = x
    if _has(c):
        # the norm sees the stream as it is stored
        s = (x.float() + st["residual"].detach().float()).to(st["residual"].dtype)
    sf = s.float()
    centred = sf - sf.mean(1, keepdim=True)
    rstd = torch.rsqrt((centred * centred).mean(1, keepdim=True) + EPS)
    xhat = centred * rstd
    y = xhat * w
    if c["bias"]:
        y = y + st["bias"].detach().float()
    out = {"y": y.to(x.dtype)}
    if _has(c):
        out["residual"] = s
    if not c["train"]:
        return out
    dy = st["dy"].float()
    g = dy * w
    d = rstd * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    if _has(c):
        d = d + st["ds"].float()
    out["dx"] = d.to(x.dtype)
    if _has(c):
        out["dresidual"] = d.to(st["residual"].dtype)
    out["dweight"] = (dy * xhat).sum(0).to(st["weight"].dtype)
    if c["bias"]:
        out["dbias"] = dy.sum(0).to(st["bias"].dtype)
    return out


def _transformed(c, z):
    """(f(z), f'(z)) of raw logits z."""
    if c["softcap"]:
        t = torch.tanh(z / c["softcap"])
        return c["softcap"] / c["temperature"] * t, (1.0 - t * t) / c["temperature"]
    return z / c["temperature"], 1.0 / c["temperature"]


def _plain_head(st):
    c = st["case"]
    h, W, N = st["h"].detach(), st["W"].detach(), c["N"]
    hf, Wf = h.float(), W.float()
    z = hf @ Wf.t()
    u, slope = _transformed(c, z)
    lse = u.logsumexp(1)
    logq = u - lse[:, None]
    q = logq.exp()
    entropy = -(q * logq).sum(1)
    live = torch.ones(N, dtype=torch.bool, device=h.device)
    if st["targets"] is not None:
        live = st["targets"] != IGNORE
        at = st["targets"].clamp(min=0)[:, None]
        logp = torch.where(live, logq.gather(1, at)[:, 0], 0.0)
    if c["op"] == "entropy":
        out = {"logp": logp, "entropy": torch.where(live, entropy, 0.0)}
        if c["train"]:
            a = torch.where(live, st["dlogp"], 0.0)[:, None]
            b = torch.where(live, st["dentropy"], 0.0)[:, None]
            # logp: onehot - q; entropy: -q (log q + entropy)
            D = -q * (a + b * (logq + entropy[:, None]))
            D.scatter_add_(1, at, a)
            D *= slope
            out["dh"] = (D @ Wf).to(h.dtype)
            out["dW"] = (D.t() @ hf).to(W.dtype)
        return out
    # the order of words whose logits lie next to one another, in 64 bits: of a few more than K of them
    K = c["K"]
    near = z.topk(min(K + 16, c["V"]), dim=1).indices.sort(dim=1).values
    exact_z = torch.bmm(W[near].double(), h.double()[:, :, None])[:, :, 0]
    best, place = exact_z.sort(dim=1, descending=True, stable=True)
    ids = near.gather(1, place[:, :K])
    logprobs = (_transformed(c, best[:, :K])[0] - lse.double()[:, None]).float()
    out = {"ids": torch.where(live[:, None], ids, -1), "logprobs": torch.where(live[:, None], logprobs, 0.0),
           "lse": torch.where(live, lse, 0.0), "entropy": torch.where(live, entropy, 0.0)}
    return dict(out, logp=logp) if c["masked"] else out


def run(st):
    if own:
        return _run_own(st)
    return _plain_layer(st) if st["case"]["op"] == "layer" else _plain_head(st)


# ---------------------------------------------------- the values in 64 bits

def _exact_layer(st):
    c = st["case"]
    x, gain = st["x"].detach().double(), st["weight"].detach().double()
    s = x
    if _has(c):
        s = (x + st["residual"].detach().double()).to(st["residual"].dtype).double()
    H = c["H"]
    var, mean = torch.var_mean(s, dim=1, unbiased=False)
    inv = (var + EPS).pow(-0.5)
    n = torch.einsum("nh,n->nh", s, inv) - (mean * inv)[:, None]
    y = torch.einsum("nh,h->nh", n, gain)
    if c["bias"]:
        y = y + st["bias"].detach().double()
    out = {"y": y}
    if _has(c):
        out["residual"] = s
    if not c["train"]:
        return out
    dy = st["dy"].double()
    # the projection of dy gain off the constants and off the normed row
    along_one = torch.einsum("nh,h->n", dy, gain) / H
    along_n = torch.einsum("nh,h,nh->n", dy, gain, n) / H
    d = torch.einsum("nh,h,n->nh", dy, gain, inv) - (along_one * inv)[:, None] - torch.einsum("nh,n,n->nh", n, along_n, inv)
    if _has(c):
        d = d + st["ds"].double()
    out["dx"] = d
    if _has(c):
        out["dresidual"] = d
    out["dweight"] = torch.einsum("nh,nh->h", dy, n)
    if c["bias"]:
        out["dbias"] = dy.sum(0)
    return out


def _exact_head(st):
    c = st["case"]
    N, V = c["N"], c["V"]
    h, W = st["h"].detach().double(), st["W"].detach().double()
    cap, T = c["softcap"], c["temperature"]
    live = torch.ones(N, dtype=torch.bool, device="cuda") if st["targets"] is None else st["targets"].ne(IGNORE)
    keys = ["lse", "entropy"] if c["op"] == "top" else ["entropy"]
    out = {k: torch.zeros(N, dtype=torch.float64, device="cuda") for k in keys}
    if st["targets"] is not None:
        out["logp"] = torch.zeros(N, dtype=torch.float64, device="cuda")
    if c["op"] == "top":
        out["ids"] = torch.full((N, c["K"]), -1, dtype=torch.int64, device="cuda")
        out["logprobs"] = torch.zeros(N, c["K"], dtype=torch.float64, device="cuda")
    if c.get("train"):
        out["dh"], out["dW"] = torch.zeros_like(h), torch.zeros_like(W)
    for a in range(0, N, 512):
        b = slice(a, min(N, a + 512))
        z = h[b] @ W.t()
        u = cap * torch.tanh(z / cap) / T if cap else z / T
        top = u.max(1, keepdim=True).values
        e = (u - top).exp()
        mass = e.sum(1, keepdim=True)
        p = e / mass
        # log(mass) + sum p (top - u): every term is positive
        entropy = mass.log()[:, 0] + (p * (top - u)).sum(1)
        lse = (top + mass.log())[:, 0]
        on = live[b]
        out["entropy"][b] = torch.where(on, entropy, 0.0)
        if c["op"] == "top":
            out["lse"][b] = torch.where(on, lse, 0.0)
            near = z.topk(min(c["K"] + 16, V), dim=1).indices.sort(dim=1).values
            best, place = z.gather(1, near).sort(dim=1, descending=True, stable=True)
            ids = near.gather(1, place)[:, : c["K"]]
            out["ids"][b] = torch.where(on[:, None], ids, -1)
            out["logprobs"][b] = torch.where(on[:, None], u.gather(1, ids) - lse[:, None], 0.0)
        if st["targets"] is None:
            continue
        t = st["targets"][b].clamp(min=0)[:, None]
        out["logp"][b] = torch.where(on, u.gather(1, t)[:, 0] - lse, 0.0)
        if c.get("train"):
            da, de = (torch.where(on, st[k][b].double(), 0.0)[:, None] for k in ("dlogp", "dentropy"))
            onehot = torch.zeros_like(p).scatter_(1, t, 1.0)
            D = da * (onehot - p) + de * p * (lse[:, None] - u - entropy[:, None])
            D = D * ((1.0 - (u * T / cap).square()) / T if cap else 1.0 / T)
            out["dh"][b] = D @ W
            out["dW"] += D.t() @ h[b]
    return {k: out[k] for k in ("ids", "logprobs", "lse", "logp", "entropy", "dh", "dW") if k in out}


def exact(case, seed):
    if case["op"] != "layer" and work(case)["flops"] > 6e12:
        return None  # the products in 64 bits take a quarter of a minute and more
    st = prepare(case, seed)
    return _exact_layer(st) if case["op"] == "layer" else _exact_head(st)
