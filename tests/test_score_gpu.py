"""Log-probability with entropy and the likeliest words against the definition
in 64 bits, at the sizes, masks and ties where a kernel can go wrong."""
import math

import pytest
import torch

import chunked_lm_head_gb300 as flce
from chunked_lm_head_gb300 import _lib

import score_ref as R

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
TFS = [None, {"temperature": 0.7}, {"softcap": 20.0, "temperature": 1.5, "scale_multiply": 1.25},
       {"scale_divide": 2.0}]


def make(N, H, V, seed=0, std=3.0, mask=0.0):
    g = torch.Generator(device="cuda").manual_seed(977 * seed + 31 * N + 7 * H + V)
    h = torch.randn(N, H, generator=g, device="cuda").bfloat16()
    W = (std / math.sqrt(H) * torch.randn(V, H, generator=g, device="cuda")).bfloat16()
    t = torch.randint(0, V, (N,), generator=g, device="cuda")
    if mask:
        t[torch.rand(N, generator=g, device="cuda") < mask] = R.IGNORE
    ga = torch.randn(N, generator=g, device="cuda")
    ge = torch.randn(N, generator=g, device="cuda")
    return h, W, t, ga, ge


# rows on both sides of the few-row forward and of a tile; vocabularies that end
# inside a chunk, a tile and a record pair; hidden sizes down to 8
FORWARD = [(1, 8, 7), (1, 64, 1000), (2, 72, 33001), (3, 4096, 5000), (4, 264, 40003), (5, 64, 1000), (33, 200, 8225),
           (128, 64, 255), (129, 72, 257), (257, 256, 20011), (300, 1096, 32003)]


@pytest.mark.parametrize("tf", TFS, ids=["none", "temperature", "softcap", "divide"])
@pytest.mark.parametrize("N,H,V", FORWARD)
def test_forward_matches_the_definition(N, H, V, tf):
    h, W, t, _, _ = make(N, H, V)
    r = R.reference(h, W, t, 0, tf)
    out = flce.score_forward(h, W, t, transform=tf)
    assert _lib.flce_device_status() == 0
    assert out["ids"] is None and out["logprobs"] is None
    R.check(out, h, W, t, r, tf=tf)


TOP = [(1, 64, 1000, 1), (1, 64, 1000, 128), (1, 256, 60000, 20), (2, 8, 9, 9), (3, 128, 40001, 128), (4, 72, 33000, 5),
       (5, 64, 40, 40), (5, 64, 128, 128), (70, 64, 300, 100), (130, 72, 33025, 37), (257, 256, 20011, 20),
       (300, 1096, 32003, 64), (64, 40, 70001, 128)]


@pytest.mark.parametrize("tf", TFS[:3], ids=["none", "temperature", "softcap"])
@pytest.mark.parametrize("N,H,V,K", TOP)
def test_words_match_the_definition(N, H, V, K, tf):
    h, W, t, _, _ = make(N, H, V, seed=1)
    r = R.reference(h, W, t, K, tf)
    out = flce.top_logprobs(h, W, K, t, transform=tf)
    assert _lib.flce_device_status() == 0
    R.check(out, h, W, t, r, K, tf)
    bare = flce.top_logprobs(h, W, K, transform=tf)
    assert bare["logp"] is None
    for k in ("ids", "logprobs", "lse", "entropy"):
        assert torch.equal(bare[k], out[k]), k


@pytest.mark.parametrize("cg", [1, 2])
@pytest.mark.parametrize("N,V,K", [(1, 5000, 20), (150, 5000, 4), (150, 5000, 60), (2500, 3001, 9)])
def test_ignored_rows(flce_opts, N, V, K, cg):
    """Below and above the row count from which they are left out of the product."""
    flce_opts.set("cta_group", cg)
    h, W, t, _, _ = make(N, 64, V, seed=2, mask=0.4)
    r = R.reference(h, W, t, K)
    out = flce.top_logprobs(h, W, K, t)
    R.check(out, h, W, t, r, K)
    gone = t == R.IGNORE
    assert bool((out["ids"][gone] == -1).all())
    for k in ("lse", "entropy", "logp", "logprobs"):
        assert not bool(out[k][gone].any()), k
    e = flce.score_forward(h, W, t)
    R.check(e, h, W, t, r)
    assert not bool(e["lse"][gone].any())
    every = torch.full_like(t, R.IGNORE)
    none = flce.top_logprobs(h, W, K, every)
    assert bool((none["ids"] == -1).all()) and not bool(none["lse"].any())
    assert _lib.flce_device_status() == 0


@pytest.mark.parametrize("N", [1, 4, 5, 200])
@pytest.mark.parametrize("V,K", [(50001, 40), (4000, 40)])
def test_near_ties_are_told_apart(N, V, K):
    """Words whose logits differ by less than a 32-bit sum's rounding: copies of one
    word's weights with one element moved by one step, in index order shuffled."""
    H = 512
    h, W, _, _, _ = make(N, H, V, seed=3)
    base = (0.1 * h[0]).bfloat16()  # its logit is far above the others
    small = int(h[0].float().abs().argmin())
    where = torch.randperm(V, generator=torch.Generator().manual_seed(5))[:60].cuda()
    W[where] = base
    W[where[:30], small] = torch.linspace(-0.01, 0.01, 30, device="cuda").bfloat16()
    r = R.reference(h, W, None, K)
    gaps = r["z"][0].sort(descending=True).values[:31].diff().abs()
    assert float(gaps[gaps > 0].min()) < 2.0 ** -24 * float(r["z"][0].max())  # below fp32's steps
    out = flce.top_logprobs(h, W, K)
    R.check(out, h, W, None, r, K)


@pytest.mark.parametrize("N", [2, 130])
@pytest.mark.parametrize("V,K", [(40000, 9), (3000, 40), (1000, 128)])
def test_equal_logits_go_to_the_lowest_index(N, V, K):
    """Rows of zeros, and a head whose words are all alike: more candidates than the list holds."""
    h, W, _, _, _ = make(N, 64, V, seed=4)
    h[1] = 0
    out = flce.top_logprobs(h, W, K)
    assert torch.equal(out["ids"][1], torch.arange(K, device="cuda"))
    assert torch.allclose(out["logprobs"][1], torch.full((K,), -math.log(V), device="cuda"), rtol=1e-6)
    assert abs(float(out["entropy"][1]) - math.log(V)) <= 2e-6 * math.log(V)
    W[:] = W[7].clone()
    out = flce.top_logprobs(h, W, K)
    assert torch.equal(out["ids"], torch.arange(K, device="cuda").expand(N, K))
    assert _lib.flce_device_status() == 0


@pytest.mark.parametrize("N,V,K", [(700, 120000, 20), (3, 120000, 20), (700, 2500, 128)])
def test_rows_of_padding(N, V, K):
    """Most rows zero (also with -0): their words are the first, and they cost no sums."""
    h, W, t, _, _ = make(N, 256, V, seed=26)
    h[1:] = 0
    h[2, 5] = -0.0
    r = R.reference(h, W, t, K)
    out = flce.top_logprobs(h, W, K, t)
    R.check(out, h, W, t, r, K)
    assert torch.equal(out["ids"][1:], torch.arange(K, device="cuda").expand(N - 1, K))


@pytest.mark.parametrize("N", [1, 3, 140])
@pytest.mark.parametrize("V,K", [(40000, 50), (2000, 50)])
def test_words_that_are_neighbours(N, V, K):
    """The best words in one run of indices: whole chunks are candidates."""
    h, W, _, _, _ = make(N, 128, V, seed=5)
    W[1003:1003 + 77] += (0.2 * h[0].float()).bfloat16()
    r = R.reference(h, W, None, K)
    assert bool(((r["ids"][0] >= 1003) & (r["ids"][0] < 1080)).all())
    R.check(flce.top_logprobs(h, W, K), h, W, None, r, K)


@pytest.mark.parametrize("N", [1, 4, 129])
@pytest.mark.parametrize("V,K", [(9000, 5), (900, 100)])
def test_not_a_number_and_infinity(N, V, K):
    h, W, t, _, _ = make(N, 64, V, seed=6)
    clean = flce.top_logprobs(h, W, K, t)
    for bad in (float("nan"), float("inf"), -float("inf")):
        b = h.clone()
        b[0, 3] = bad
        for out in (flce.top_logprobs(b, W, K, t), flce.score_forward(b, W, t)):
            # an infinity times weights of both signs: a row with +infinity or NaN
            for k in ("lse", "entropy", "logp", "logprobs"):
                if out[k] is not None:
                    assert bool(out[k][0].isnan().all()), (k, bad)
                    assert torch.equal(out[k][1:], clean[k][1:]) or out["ids"] is None, (k, bad)
        out = flce.top_logprobs(b, W, K, t, transform={"softcap": 5.0})
        assert bool((out["ids"][0] == -1).all()) and bool(out["lse"][0].isnan())
    # words that no row can take: their logit is -infinity everywhere
    b, Wb = h.abs() + 0.1, W.clone()
    Wb[5:40] = -float("inf")
    keep = torch.ones(V, dtype=torch.bool, device="cuda")
    keep[5:40] = False
    z = (b.double() @ W.double().t()).masked_fill(~keep, -float("inf"))
    lse = z.logsumexp(1)
    p = (z - lse[:, None]).exp()
    ent = -torch.where(p > 0, p * (z - lse[:, None]), 0.0).sum(1)
    out = flce.top_logprobs(b, Wb, K)
    e = 4 * 2.0 ** -22 * z[:, keep].abs().amax(1) * 2
    assert bool(((out["lse"].double() - lse).abs() <= e + 2.0 ** -18 * (1 + lse.abs())).all())
    assert bool(((out["entropy"].double() - ent).abs() <= 40 * e + 2.0 ** -18 * (1 + ent)).all())
    assert torch.equal(out["ids"], z.sort(dim=1, descending=True, stable=True).indices[:, :K])
    assert _lib.flce_device_status() == 0


def test_confident_and_uniform_rows():
    """Entropy near 0 and near log V, where lse - sum p x would cancel or drift."""
    V, H = 30000, 64
    h, W, t, _, _ = make(6, H, V, seed=7)
    W[123] = (0.9 * h[0]).bfloat16()  # row 0: one word with logit about 58
    h[1] = 0
    r = R.reference(h, W, t, 3)
    out = flce.top_logprobs(h, W, 3, t)
    R.check(out, h, W, t, r, 3)
    small = float(r["entropy"][0])
    assert small < 1e-8 and abs(float(out["entropy"][0]) - small) <= 2.0 ** -22
    assert float(out["entropy"].min()) >= 0.0


def test_targets_outside_the_vocabulary(flce_opts):
    h, W, t, ga, ge = make(140, 64, 1000, seed=8)
    t[2], t[3] = 1000, -5
    for out in (flce.score_forward(h, W, t), flce.top_logprobs(h, W, 4, t), flce.score_forward(h[:4], W, t[:4])):
        assert out["logp"][2:4].isnan().all() and not out["logp"][4:].isnan().any() and not out["lse"].isnan().any()
    r = R.reference(h, W, t.clamp(0, 999), 0)
    dH, dW = flce.score_backward(h, W, t, r["lse"].float(), r["entropy"].float(), ga, ge)
    R.check_grads(dH, dW, h, W, t, r, ga, ge)
    flce_opts.set("validate", 1)
    with pytest.raises(_lib.FlceError, match="BAD_TARGET"):
        flce.score_forward(h, W, t)


# ------------------------------------------------------------------ gradients

GRADS = [(1, 64, 1000, 256), (4, 72, 5003, 256), (64, 64, 1000, 256), (129, 256, 3000, 128), (300, 136, 5001, 4096),
         (700, 64, 9000, 128), (513, 72, 20001, 256)]


@pytest.mark.parametrize("which", ["both", "logp", "entropy"])
@pytest.mark.parametrize("tf", TFS[:3], ids=["none", "temperature", "softcap"])
@pytest.mark.parametrize("N,H,V,chunk", GRADS)
def test_gradients_match_the_definition(N, H, V, chunk, tf, which):
    """One row block, several, and several slabs of the vocabulary (few chunk rows)."""
    h, W, t, ga, ge = make(N, H, V, seed=9, mask=0.2)
    ga = None if which == "entropy" else ga
    ge = None if which == "logp" else ge
    h.requires_grad_(True)
    W.requires_grad_(True)
    logp, entropy = flce.selective_log_softmax_entropy(h, W, t, chunk_rows=chunk, transform=tf)
    outs = [(o, g) for o, g in ((logp, ga), (entropy, ge)) if g is not None]
    dH, dW = torch.autograd.grad([o for o, _ in outs], (h, W), [g for _, g in outs])
    assert dH.dtype == BF16 and dW.dtype == BF16
    with torch.no_grad():
        r = R.reference(h, W, t, 0, tf)
        R.check(dict(logp=logp, entropy=entropy), h, W, t, r, tf=tf)
        R.check_grads(dH, dW, h, W, t, r, ga, ge, tf, kept=N <= 128)
        out = flce.score_forward(h, W, t, transform=tf)
        dH32, dW32 = flce.score_backward(h, W, t, out["lse"], out["entropy"], ga, ge, chunk, transform=tf)
        if N > 128:  # (else the first were from kept logits)
            assert torch.equal(dH32, dH)
            assert torch.equal(dW32.bfloat16(), dW)
        R.check_grads(dH32, dW32, h, W, t, r, ga, ge, tf)
    assert _lib.flce_device_status() == 0


KEPT = [(1, 512, 1000), (3, 64, 1000), (128, 72, 5003), (4, 520, 5003), (64, 512, 3001), (65, 1096, 2000), (128, 512, 9000), (129, 512, 3000),
        (300, 1000, 9001), (700, 512, 20001), (2049, 512, 1000)]


@pytest.mark.parametrize("which", ["both", "logp", "entropy"])
@pytest.mark.parametrize("tf", TFS[:3], ids=["none", "temperature", "softcap"])
@pytest.mark.parametrize("N,H,V", KEPT)
def test_gradients_from_kept_logits(N, H, V, tf, which):
    """Rows on both sides of the two-part dlogits and of the row compaction."""
    h, W, t, ga, ge = make(N, H, V, seed=22, mask=0.2)
    ga = None if which == "entropy" else ga
    ge = None if which == "logp" else ge
    out = flce.score_forward(h, W, t, transform=tf, keep_rows=N)
    assert out["state"] is not None
    before = out["state"].clone()
    r = R.reference(h, W, t, 0, tf)
    R.check(out, h, W, t, r, tf=tf)
    for dt in (torch.float32, BF16):
        dH, dW = flce.score_backward(h, W, t, out["lse"], out["entropy"], ga, ge, transform=tf, state=out["state"],
                                     dW_dtype=dt)
        assert _lib.flce_device_status() == 0
        R.check_grads(dH, dW, h, W, t, r, ga, ge, tf, kept=True)
    one = flce.score_backward(h, W, t, out["lse"], out["entropy"], ga, ge, transform=tf, state=out["state"],
                              need_dW=False)
    assert one[1] is None and torch.equal(one[0], dH)
    assert torch.equal(out["state"], before)  # it can be read again


def test_kept_and_recomputed_through_autograd():
    N, H, V = 200, 512, 9001
    h, W, t, ga, ge = make(N, H, V, seed=23, mask=0.2)
    h.requires_grad_(True)
    W.requires_grad_(True)
    with torch.no_grad():
        r = R.reference(h, W, t)
    for kw, kept in ((dict(chunk_rows=256), True), (dict(chunk_rows=256, recompute=True), False),
                     (dict(chunk_rows=128), False)):
        logp, entropy = flce.selective_log_softmax_entropy(h, W, t, **kw)
        grads = torch.autograd.grad((logp, entropy), (h, W), (ga, ge), retain_graph=True)
        again = torch.autograd.grad((logp, entropy), (h, W), (ga, ge))
        with torch.no_grad():
            R.check_grads(*grads, h, W, t, r, ga, ge, kept=kept)
        assert all(torch.equal(a, b) for a, b in zip(grads, again))


@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("N,H", [(2, 64), (20, 512), (128, 64), (129, 64), (200, 512), (256, 1096), (300, 64), (700, 512)])
def test_what_ignored_rows_hold_goes_nowhere(N, H, value):
    h, W, t, ga, ge = make(N, H, 3001, seed=29, mask=0.3)
    t[N // 2] = R.IGNORE
    h2 = h.clone()
    h2[t == R.IGNORE] = value

    def step(x, chunk, recompute):
        x, y = x.detach().requires_grad_(True), W.detach().requires_grad_(True)
        out = flce.selective_log_softmax_entropy(x, y, t, chunk_rows=chunk, recompute=recompute)
        top = flce.top_logprobs(x.detach(), y.detach(), 5, t)
        return [o.detach() for o in out] + [top[k] for k in ("ids", "logprobs", "lse", "entropy", "logp")] + list(
            torch.autograd.grad(out, (x, y), (ga, ge)))

    for chunk, recompute in ((128, True), (256, False), (256, True), (1024, False)):
        for a, b in zip(step(h, chunk, recompute), step(h2, chunk, recompute)):
            assert torch.equal(a, b), (chunk, recompute)
    assert _lib.flce_device_status() == 0


@pytest.mark.parametrize("N,H,chunk", [(20, 64, 256), (200, 512, 256), (300, 64, 128), (400, 512, 128)])
def test_no_counted_row_has_no_gradient(N, H, chunk):
    h, W, t, ga, ge = make(N, H, 3001, seed=27)
    t[:] = R.IGNORE
    h.requires_grad_(True)
    W.requires_grad_(True)
    logp, entropy = flce.selective_log_softmax_entropy(h, W, t, chunk_rows=chunk)
    assert not bool(logp.any()) and not bool(entropy.any())
    dH, dW = torch.autograd.grad((logp, entropy), (h, W), (ga, ge))
    assert not bool(dH.any()) and not bool(dW.any())
    assert _lib.flce_device_status() == 0


def test_likely_targets_keep_their_gradient():
    """1 - p of a target with p = 0.999: 16-bit logits alone would be off by a tenth of it."""
    N, H, V = 32, 512, 3000
    h, W, t, ga, ge = make(N, H, V, seed=24)
    t[:] = torch.arange(N, device="cuda") * 90 + 7
    W[t] = (0.04 * h.float()).bfloat16()  # logits about 20 against a log-sum-exp of 12.5 of the others
    r = R.reference(h, W, t)
    assert bool(((1 - r["logp"].exp()) < 0.02).all())
    out = flce.score_forward(h, W, t, keep_rows=N)
    dH, dW = flce.score_backward(h, W, t, out["lse"], out["entropy"], ga, None, state=out["state"])
    R.check_grads(dH, dW, h, W, t, r, ga, None, kept=True)
    D, _ = R.dlogits(r, t, ga, None)
    for got, want in ((dH, D @ W.double()), (dW, D.t() @ h.double())):
        assert float((got.double() - want).norm() / want.norm()) < 5e-3


@pytest.mark.parametrize("option,value", [("cta_group", 1), ("compact", 0), ("fwd_splits", 3), ("dh_splits", 2)])
def test_options_leave_kept_logits_right(flce_opts, option, value):
    h, W, t, ga, ge = make(400, 512, 9001, seed=25, mask=0.3)
    r = R.reference(h, W, t)
    out = flce.score_forward(h, W, t, keep_rows=512)
    flce_opts.set(option, value)  # between forward and backward, and then for both
    for o in (out, flce.score_forward(h, W, t, keep_rows=512)):
        dH, dW = flce.score_backward(h, W, t, o["lse"], o["entropy"], ga, ge, state=o["state"])
        R.check_grads(dH, dW, h, W, t, r, ga, ge, kept=True)
    assert _lib.flce_device_status() == 0


@pytest.mark.parametrize("option,value", [("cta_group", 1), ("pipeline", 0), ("compact", 0), ("d_tma", 0),
                                          ("fwd_splits", 3), ("grid_workers", 7), ("fwd_block_rows", 256)])
def test_options_change_the_schedule_only(flce_opts, option, value):
    N, H, V = 600, 72, 9001
    h, W, t, ga, ge = make(N, H, V, seed=10, mask=0.3)
    flce_opts.set("skip_min_rows", 100)
    r = R.reference(h, W, t, 11)
    flce_opts.set(option, value)
    out = flce.top_logprobs(h, W, 11, t)
    R.check(out, h, W, t, r, 11)
    e = flce.score_forward(h, W, t)
    R.check(e, h, W, t, r)
    dH, dW = flce.score_backward(h, W, t, e["lse"], e["entropy"], ga, ge, 128)
    R.check_grads(dH, dW, h, W, t, r, ga, ge)
    assert _lib.flce_device_status() == 0


def test_only_the_wanted_gradients_and_expanded_ones():
    h, W, t, ga, ge = make(200, 64, 3000, seed=11)
    for a, b in ((True, False), (False, True)):
        x, y = h.clone().requires_grad_(a), W.clone().requires_grad_(b)
        logp, entropy = flce.selective_log_softmax_entropy(x, y, t)
        (logp.sum() - 0.125 * entropy.sum()).backward()  # expanded gradients
        with torch.no_grad():
            r = R.reference(h, W, t)
            one = torch.ones(200, device="cuda")
            R.check_grads(x.grad, y.grad, h, W, t, r, one, -0.125 * one)
    with torch.no_grad():
        logp, entropy = flce.selective_log_softmax_entropy(h, W, t)
    assert not logp.requires_grad
    assert torch.equal(logp, flce.score_forward(h, W, t)["logp"])


# ------------------------------------------------------------------- use

def test_same_bits_each_time_and_on_another_stream():
    h, W, t, ga, ge = make(300, 136, 9001, seed=13, mask=0.2)

    def step(**kw):
        o = flce.top_logprobs(h, W, 20, t, **kw)
        return [o[k] for k in ("ids", "logprobs", "lse", "entropy", "logp")] + list(
            flce.score_backward(h, W, t, o["lse"], o["entropy"], ga, ge, **kw))

    first = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = step()
    side.synchronize()
    third = step(stream=side)
    side.synchronize()
    for a, b, c in zip(first, second, third):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_two_calls_at_once():
    h, W, t, _, _ = make(3, 256, 40001, seed=14)
    h2, W2, t2, _, _ = make(200, 256, 20001, seed=15)
    want = flce.top_logprobs(h, W, 7, t), flce.top_logprobs(h2, W2, 7, t2)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(4):
        with torch.cuda.stream(a):
            x = flce.top_logprobs(h, W, 7, t)
        with torch.cuda.stream(b):
            y = flce.top_logprobs(h2, W2, 7, t2)
        got.append((x, y))
    torch.cuda.synchronize()
    for pair in got:
        for o, w in zip(pair, want):
            for k in ("ids", "logprobs", "lse", "entropy", "logp"):
                assert torch.equal(o[k], w[k]), k


@pytest.mark.parametrize("N,H", [(2, 64), (150, 64), (2100, 64), (2, 512), (300, 512)])
def test_capture_and_replay(N, H):
    h, W, t, ga, ge = make(N, H, 9001, seed=16, mask=0.2)

    def step():
        x, y = h.detach().requires_grad_(True), W.detach().requires_grad_(True)  # leaves of this step's own
        o = flce.top_logprobs(h, W, 6, t)
        logp, entropy = flce.selective_log_softmax_entropy(x, y, t, chunk_rows=512)
        return [o[k] for k in ("ids", "logprobs", "lse", "entropy", "logp")] + [logp.detach(), entropy.detach()] + list(
            torch.autograd.grad((logp, entropy), (x, y), (ga, ge)))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    h.copy_(make(N, H, 9001, seed=17)[0])
    t.copy_(make(N, H, 9001, seed=18, mask=0.5)[2])
    graph.replay()
    torch.cuda.synchronize()
    captured = [c.clone() for c in captured]
    for a, b in zip(captured, step()):
        assert torch.equal(a, b)
    assert _lib.flce_device_status() == 0


def test_a_capture_beside_a_live_eager_graph_is_refused():
    h, W, t, ga, ge = make(150, 64, 5001, seed=28)
    h.requires_grad_(True)
    W.requires_grad_(True)
    w = torch.ones(64, device="cuda", dtype=BF16, requires_grad=True)

    def step():
        logp, entropy = flce.selective_log_softmax_entropy(flce.layer_norm(h, w), W, t)
        return torch.autograd.grad((logp, entropy), (h, W, w), (ga, ge))

    want = step()
    for alive in (lambda: flce.layer_norm(h, w.detach()), lambda: flce.layer_norm(h.detach(), w),
                  lambda: flce.selective_log_softmax_entropy(h.detach(), W, t)):
        held = alive()
        graph = torch.cuda.CUDAGraph()
        with pytest.raises(RuntimeError, match="eager graph of a leaf"):
            with torch.cuda.graph(graph):
                step()
        del held, graph
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert _lib.flce_device_status() == 0


def test_a_callers_workspace():
    h, W, t, ga, ge = make(200, 64, 9001, seed=19)
    ws = torch.full((_lib.flce_score_workspace_bytes(200, 64, 9001, 5),), 255, dtype=torch.uint8, device="cuda")
    a, b = flce.top_logprobs(h, W, 5, t, workspace=ws), flce.top_logprobs(h, W, 5, t)
    for k in ("ids", "logprobs", "lse", "entropy", "logp"):
        assert torch.equal(a[k], b[k]), k
    wb = torch.full((_lib.flce_score_backward_workspace_bytes(200, 64, 9001, 256, _lib.DTYPES["bf16"]),), 255,
                    dtype=torch.uint8, device="cuda")
    for dt in (torch.float32, BF16):
        p = flce.score_backward(h, W, t, a["lse"], a["entropy"], ga, ge, workspace=wb, dW_dtype=dt)
        q = flce.score_backward(h, W, t, a["lse"], a["entropy"], ga, ge, dW_dtype=dt)
        assert torch.equal(p[0], q[0]) and torch.equal(p[1], q[1])
    with pytest.raises(ValueError, match="CUDA"):
        flce.top_logprobs(h, W, 5, t, workspace=ws.cpu())


def test_no_rows():
    W = torch.randn(100, 64, device="cuda").bfloat16().requires_grad_(True)
    h = torch.empty(0, 64, device="cuda", dtype=BF16, requires_grad=True)
    t = torch.empty(0, dtype=torch.int64, device="cuda")
    out = flce.top_logprobs(h, W, 3)
    assert out["ids"].shape == (0, 3) and out["lse"].shape == (0,)
    logp, entropy = flce.selective_log_softmax_entropy(h, W, t)
    dH, dW = torch.autograd.grad(logp.sum() + entropy.sum(), (h, W))
    assert dH.shape == (0, 64) and not bool(dW.any())
    logp, entropy = flce.selective_log_softmax_entropy(h, W.detach(), t)
    assert torch.autograd.grad(logp.sum() + entropy.sum(), h)[0].shape == (0, 64)


def test_a_second_derivative_is_refused():
    h, W, t, _, _ = make(8, 64, 100, seed=20)
    h.requires_grad_(True)
    logp, entropy = flce.selective_log_softmax_entropy(h, W, t)
    (dh,) = torch.autograd.grad(logp.sum() + entropy.sum(), h, create_graph=True)
    with pytest.raises(RuntimeError, match="second derivative"):
        dh.float().sum().backward()


def test_refusals_of_the_torch_checks():
    h, W, t, ga, ge = make(8, 64, 100, seed=21)
    o = flce.score_forward(h, W, t)
    for call in (lambda: flce.top_logprobs(h.float(), W, 3), lambda: flce.top_logprobs(h, W.t(), 3),
                 lambda: flce.top_logprobs(h, W, 0), lambda: flce.top_logprobs(h, W, 101),
                 lambda: flce.top_logprobs(h, W, 3, t.int()), lambda: flce.top_logprobs(h, W, 3, t[:4]),
                 lambda: flce.top_logprobs(h, W, 3, t.cpu()), lambda: flce.top_logprobs(h[:, ::2], W[:, :32], 3),
                 lambda: flce.selective_log_softmax_entropy(h, W, None),
                 lambda: flce.score_backward(h, W, t, o["lse"].double(), o["entropy"], ga, ge),
                 lambda: flce.score_backward(h, W, t, o["lse"], o["entropy"], ga[:3], ge),
                 lambda: flce.score_backward(h, W, None, o["lse"], o["entropy"], ga, ge),
                 lambda: flce.score_backward(h, W, t, o["lse"], o["entropy"], ga, ge, state=ga),
                 lambda: flce.score_forward(h, W, keep_rows=8), lambda: flce.score_forward(h, W, t, 3, keep_rows=8),
                 lambda: flce.score_backward(h, W, t, o["lse"], o["entropy"], ga, ge, dW_dtype=torch.float16)):
        with pytest.raises(ValueError):
            call()
    W2 = torch.zeros(1000, 64, device="cuda", dtype=BF16)
    with pytest.raises(_lib.FlceError, match="UNSUPPORTED"):
        flce.top_logprobs(h, W2, 129)


def test_a_head_past_32_bit_offsets():
    """V H beyond 2^31: words at the vocabulary's end."""
    N, H, V = 6, 4096, 530001
    g = torch.Generator(device="cuda").manual_seed(3)
    h = torch.randn(N, H, generator=g, device="cuda").bfloat16()
    W = torch.empty(V, H, device="cuda", dtype=BF16)
    for a in range(0, V, 65536):
        W[a:a + 65536] = 0.02 * torch.randn(min(65536, V - a), H, generator=g, device="cuda")
    W[V - 40:] *= 4
    z = torch.cat([h.double() @ W[a:a + 65536].double().t() for a in range(0, V, 65536)], 1)
    want = z.sort(dim=1, descending=True, stable=True).indices[:, :16]
    assert int((want >= V - 40).sum()) > 6
    for n in (6, 2):
        out = flce.top_logprobs(h[:n].contiguous(), W, 16)
        assert torch.equal(out["ids"], want[:n])
        assert float((out["lse"].double() - z[:n].logsumexp(1)).abs().max()) < 1e-4


@pytest.mark.parametrize("recompute", [False, True])
def test_kept_logits_past_32_bit_offsets(recompute):
    """N V beyond 2^31, gradients of the last rows alone."""
    N, H, V, n = 16400, 512, 131104, 200
    h, W, t, ga, ge = make(N, H, V, seed=30)
    ga[:-n] = 0
    ge[:-n] = 0
    h.requires_grad_(True)
    W.requires_grad_(True)
    out = flce.selective_log_softmax_entropy(h, W, t, chunk_rows=N, recompute=recompute)
    dH, dW = torch.autograd.grad(out, (h, W), (ga, ge))
    assert _lib.flce_device_status() == 0
    with torch.no_grad():
        end = [x[-n:].contiguous() for x in (h, t, out[0], out[1], ga, ge, dH)]
        r = R.reference(end[0], W, end[1])
        R.check(dict(logp=end[2], entropy=end[3]), end[0], W, end[1], r)
        R.check_grads(end[6], dW, end[0], W, end[1], r, end[4], end[5], kept=not recompute)
        assert not bool(dH[:-n].any())


@pytest.mark.parametrize("tf", [None, TFS[2]], ids=["none", "softcap"])
@pytest.mark.parametrize("N,H,V", [(300, 512, 20011), (384, 512, 20000), (270, 1024, 33001)])
def test_a_third_row_tile(N, H, V, tf):
    """Rows that fill one tile of a pair and little of the next, some of them ignored:
    forward, words, and gradients from kept and recomputed logits."""
    h, W, t, ga, ge = make(N, H, V, seed=31, mask=0.1)
    r = R.reference(h, W, t, 20, tf)
    R.check(flce.score_forward(h, W, t, transform=tf), h, W, t, r, tf=tf)
    R.check(flce.top_logprobs(h, W, 20, t, transform=tf), h, W, t, r, 20, tf=tf)
    for keep in (0, 512):
        o = flce.score_forward(h, W, t, transform=tf, keep_rows=keep)
        assert (o["state"] is not None) == (keep > 0)
        R.check(o, h, W, t, r, tf=tf)
        dH, dW = flce.score_backward(h, W, t, o["lse"], o["entropy"], ga, ge, chunk_rows=512, transform=tf,
                                     dW_dtype=BF16, state=o["state"])
        R.check_grads(dH, dW, h, W, t, r, ga, ge, tf, kept=keep > 0)
    assert _lib.flce_device_status() == 0
