"""Distillation from a teacher's top logits against the definition in 64 bits:
forward, recomputing backward and the one-call step, over list lengths,
masks, transforms, types and tilings."""
import math

import pytest
import torch

import chunked_lm_head_gb300 as flce
from chunked_lm_head_gb300 import _lib

import topk_ref as R

pytestmark = pytest.mark.gpu


def make(N, H, V, K, seed=0, std=0.1, mask=False, pad=False, whole=False, ids_dtype=torch.int64,
         logits_dtype=torch.float32, weights=False):
    g = torch.Generator(device="cuda").manual_seed(1000 + seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    h, W = rnd(N, H).bfloat16(), (std * rnd(V, H)).bfloat16()
    z = 1.5 * ((0.7 * h.float() + 0.7 * rnd(N, H)) @ W.float().t())
    logits, ids = z.topk(K, dim=1)
    order = torch.rand(N, K, generator=g, device="cuda").argsort(1)  # lists in any order
    logits, ids = logits.gather(1, order), ids.gather(1, order)
    if pad:
        ids[torch.rand(N, K, generator=g, device="cuda") < 0.3] = -1
        if N > 3:
            ids[1] = -7
    targets = w = None
    if mask:
        targets = torch.zeros(N, dtype=torch.int64, device="cuda")
        targets[torch.rand(N, generator=g, device="cuda") < 0.3] = -100
    if weights:
        w = torch.randn(N, generator=g, device="cuda")
    return dict(h=h, W=W, ids=ids.to(ids_dtype), logits=logits.to(logits_dtype),
                lse_t=z.logsumexp(1) if whole else None, targets=targets, weights=w)


def run_all(c, tail=False, tf=None, chunk=256, one_call_chunk=4096, what=""):
    """Forward, recomputing backward and one-call step of a case, checked."""
    ref = R.reference(**c, tail=tail, tf=tf)
    args = (c["h"], c["W"], c["ids"], c["logits"], c["lse_t"], c["targets"], c["weights"], tail)
    K = c["ids"].shape[1]
    out = flce.topk_kd_forward(*args, chunk_rows=chunk, transform=tf, for_backward=True)
    dH, dW = flce.topk_kd_backward(c["h"], c["W"], out["state"], K, 1.0, chunk, tf, count=out["n_valid"])
    assert _lib.flce_device_status() == 0
    R.check(dict(out, dH=dH, dW=dW), ref, what=what + "forward, backward")
    one = flce.topk_kd_forward_backward(*args, chunk_rows=one_call_chunk, transform=tf)
    assert _lib.flce_device_status() == 0
    R.check(one, ref, roundings=2, what=what + "one call")
    lean = flce.topk_kd_forward_backward(*args, chunk_rows=one_call_chunk, transform=tf, need_lse=False)
    R.check(lean, ref, roundings=2, what=what + "one call without lse")
    assert lean["lse"] is None
    # dW in bf16: straight from the GEMM, or from sums over row blocks
    half = flce.topk_kd_forward_backward(*args, chunk_rows=one_call_chunk, transform=tf, dW_dtype=torch.bfloat16)
    R.check(half, ref, roundings=2, what=what + "one call, bf16 dW")
    dH16, dW16 = flce.topk_kd_backward(c["h"], c["W"], out["state"], K, 1.0, chunk, tf, count=out["n_valid"],
                                       dW_dtype=torch.bfloat16)
    assert torch.equal(dW16, dW.bfloat16()) and torch.equal(dH16, dH)
    _, only = flce.topk_kd_backward(c["h"], c["W"], out["state"], K, 1.0, chunk, tf, count=out["n_valid"],
                                    dW_dtype=torch.bfloat16, need_dH=False)
    assert float((only.double() - dW.double()).norm()) <= 1e-2 * float(dW.double().norm())
    assert _lib.flce_device_status() == 0
    return ref, out, one


SHAPES = [(1, 64, 1000, 1), (2, 8, 40, 40), (5, 72, 257, 7), (64, 64, 1000, 16), (130, 128, 3001, 33),
          (300, 256, 5003, 100), (600, 192, 2048, 64), (33, 64, 4096, 128)]


@pytest.mark.parametrize("mode", ["scaled", "given", "tail"])
@pytest.mark.parametrize("N,H,V,K", SHAPES)
def test_matches_the_definition(N, H, V, K, mode):
    c = make(N, H, V, K, whole=mode != "scaled")
    run_all(c, tail=mode == "tail")


@pytest.mark.parametrize("mode", ["scaled", "given", "tail"])
@pytest.mark.parametrize("N,H,V,K", [(5, 72, 257, 7), (301, 128, 3001, 33), (700, 64, 1500, 20)])
def test_masks_padding_weights(N, H, V, K, mode):
    c = make(N, H, V, K, seed=1, mask=True, pad=True, whole=mode != "scaled", weights=True)
    run_all(c, tail=mode == "tail")


@pytest.mark.parametrize("tf", [{"temperature": 2.0}, {"scale_multiply": 0.5, "softcap": 5.0, "temperature": 0.8}])
@pytest.mark.parametrize("tail", [False, True])
def test_transforms(tf, tail):
    c = make(200, 128, 1203, 24, seed=2, mask=True, whole=tail)
    run_all(c, tail=tail, tf=tf)


@pytest.mark.parametrize("ids", [torch.int32, torch.int64])
@pytest.mark.parametrize("logits", [torch.float32, torch.bfloat16, torch.float16])
def test_types_and_row_strides(ids, logits):
    c = make(70, 64, 900, 12, seed=3, ids_dtype=ids, logits_dtype=logits)
    run_all(c)
    a = flce.topk_kd_forward(c["h"], c["W"], c["ids"], c["logits"])
    wide_i = torch.full((70, 31), -1, dtype=ids, device="cuda")
    wide_t = torch.full((70, 17), float("nan"), dtype=logits, device="cuda")
    wide_i[:, 5:17], wide_t[:, 3:15] = c["ids"], c["logits"]
    b = flce.topk_kd_forward(c["h"], c["W"], wide_i[:, 5:17], wide_t[:, 3:15])
    assert torch.equal(a["kl"], b["kl"]) and torch.equal(a["lse"], b["lse"])
    with pytest.raises(ValueError, match="contiguous"):
        flce.topk_kd_forward(c["h"], c["W"], wide_i[:, 4:28:2], wide_t[:, 3:15])


@pytest.mark.parametrize("options", [{"cta_group": 1}, {"compact": 0}, {"bwd_rows": 128}, {"bwd_rows": 256, "d_tma": 0},
                                     {"fwd_splits": 1}, {"fwd_block_rows": 256, "skip_min_rows": 0}, {"pdl": 0},
                                     {"cta_group": 1, "bwd_rows": 256, "fuse_dh_dw": 0}, {"grid_workers": 3}],
                         ids=lambda o: "-".join(f"{k}{v}" for k, v in o.items()))
def test_every_tiling_gives_the_definition(options):
    c = make(700, 128, 3000, 30, seed=4, mask=True, pad=True, whole=True, weights=True)
    with _lib.options(**options):
        for chunk in (128, 256):
            run_all(c, tail=True, chunk=chunk, one_call_chunk=128, what="fallback: ")
        run_all(c, tail=False, chunk=1024)
        out = flce.topk_kd_forward(c["h"], c["W"], c["ids"], c["logits"], c["lse_t"], c["targets"], c["weights"],
                                   skip_ignored=True)
    ref = R.reference(**c)
    R.check({k: out[k] for k in ("kl", "loss", "n_valid")}, ref, what="skip")


@pytest.mark.parametrize("N", [1, 2, 3, 4])
@pytest.mark.parametrize("H,V,K", [(8, 3, 3), (264, 1001, 5), (1000, 2500, 64), (4096, 5000, 16), (24576, 300, 7)])
def test_a_few_rows(N, H, V, K):
    """The forward of up to 4 rows reads W by warps instead of tiles (but for
    rows too long for its shared memory)."""
    tf = {"softcap": 6.0, "temperature": 0.9} if V % 2 else None
    c = make(N, H, V, K, seed=16, std=1.2 / H ** 0.5, pad=N > 2 and V > 5, whole=True, weights=True)
    c["ids"][0, 0] = c["ids"][0, 1]  # listed twice
    for tail in (False, True):
        ref = R.reference(**c, tail=tail, tf=tf)
        out = flce.topk_kd_forward(c["h"], c["W"], c["ids"], c["logits"], c["lse_t"], None, c["weights"], tail,
                                   transform=tf, for_backward=True)
        dH, dW = flce.topk_kd_backward(c["h"], c["W"], out["state"], K, 1.0, transform=tf, count=out["n_valid"])
        R.check(dict(out, dH=dH, dW=dW), ref)
    assert _lib.flce_device_status() == 0


def test_several_row_blocks_of_the_one_call_step():
    c = make(5000, 64, 700, 9, seed=5, mask=True, whole=True)
    run_all(c, tail=True, one_call_chunk=2048)


def test_the_list_holds_the_student_s_mass():
    """R near e^-35: the mass outside the list survives, since the listed
    columns never enter its sum."""
    N, H, V, K = 40, 64, 800, 4
    c = make(N, H, V, K, seed=6, std=0.05, whole=True)
    words = torch.tensor([700, 3, 255, 256], device="cuda")
    c["ids"] = words.expand(N, K).contiguous()
    c["W"][:, :K] = 0
    c["W"][words] = 0
    c["W"][words, torch.arange(K, device="cuda")] = 1
    c["h"][:, :K] = (40 + c["h"][:, :K].float()).bfloat16()
    c["lse_t"] = c["logits"].logsumexp(1) + 1e-3
    ref, out, one = run_all(c, tail=True)
    rest = torch.where(R.teacher(c["ids"], c["logits"], c["lse_t"], V)[1], -math.inf,
                       c["h"].double() @ c["W"].double().t()).logsumexp(1) - ref["lse"]
    assert float(rest.max()) < -20
    run_all(c, tail=False)


def test_an_id_listed_twice_adds_up():
    c = make(50, 64, 500, 10, seed=7, whole=True)
    c["ids"][:, 4] = c["ids"][:, 2]
    c["ids"][::2, 9] = c["ids"][::2, 2]
    c["lse_t"] += 0.5
    run_all(c, tail=True)
    c["lse_t"] = None
    run_all(c)


def test_impossible_words_and_empty_lists():
    c = make(20, 64, 500, 6, seed=8)
    c["logits"][3, 2] = -math.inf  # a listed word without mass
    c["logits"][4] = -math.inf     # none has
    c["ids"][5] = -1
    c["logits"][6, 1] = float("nan")
    c["ids"][6, 1] = -1            # what stands beside no entry does not matter
    ref, out, one = run_all(c)
    assert ref["n_valid"] == 18 and float(out["kl"][4]) == 0 and float(out["kl"][5]) == 0
    assert not one["dH"][4].any() and not one["dH"][5].any()
    # every list empty
    c["ids"][:] = -1
    one = flce.topk_kd_forward_backward(c["h"], c["W"], c["ids"], c["logits"])
    assert int(one["n_valid"]) == 0 and float(one["loss"]) == 0 and not one["dH"].any() and not one["dW"].any()
    out = flce.topk_kd_forward(c["h"], c["W"], c["ids"], c["logits"], for_backward=True)
    dH, dW = flce.topk_kd_backward(c["h"], c["W"], out["state"], 6, 1.0, count=out["n_valid"])
    assert not dH.any() and not dW.any()


def test_an_id_outside_the_vocabulary():
    c = make(20, 64, 500, 6, seed=9)
    ids = c["ids"].clone()
    ids[2, 1], ids[7] = 500, 1 << 40
    out = flce.topk_kd_forward(c["h"], c["W"], ids, c["logits"])
    bad = torch.isnan(out["kl"])
    assert bad[[2, 7]].all() and int(bad.sum()) == 2 and torch.isnan(out["loss"])
    one = flce.topk_kd_forward_backward(c["h"], c["W"], ids, c["logits"])
    assert torch.isfinite(one["dH"].float()).all() and torch.isfinite(one["dW"]).all()
    assert _lib.flce_device_status() == 0


def test_no_rows():
    c = make(4, 64, 500, 6)
    e = {k: (v[:0].contiguous() if k != "W" and v is not None else v) for k, v in c.items()}
    out = flce.topk_kd_forward(e["h"], e["W"], e["ids"], e["logits"], for_backward=True)
    assert float(out["loss"]) == 0 and int(out["n_valid"]) == 0
    one = flce.topk_kd_forward_backward(e["h"], e["W"], e["ids"], e["logits"])
    assert float(one["loss"]) == 0 and not one["dW"].any() and one["dH"].shape == (0, 64)
    _, dW = flce.topk_kd_backward(e["h"], e["W"], out["state"], 6, 1.0)
    assert not dW.any()


@pytest.mark.parametrize("recompute", [True, False])
def test_autograd(recompute):
    c = make(150, 128, 1000, 12, seed=10, mask=True, weights=True, whole=True)
    h, W = c["h"].requires_grad_(True), c["W"].requires_grad_(True)
    ref = R.reference(**c, tail=True)
    args = (c["ids"], c["logits"], c["lse_t"], c["targets"], c["weights"], True)
    loss, kl, n = flce.topk_distill_loss(h, W, *args, recompute=recompute)
    (3.0 * loss).backward()
    assert h.grad.dtype == W.grad.dtype == torch.bfloat16
    assert float((h.grad.double() / 3 - ref["dH"]).norm() / ref["dH"].norm()) < 1e-2
    assert float((W.grad.double() / 3 - ref["dW"]).norm() / ref["dW"].norm()) < 1e-2
    R.check(dict(loss=loss.detach(), kl=kl, n_valid=n), ref)
    # one gradient only; none; without gradients
    Wc = W.detach()
    loss, _, _ = flce.topk_distill_loss(h, Wc, *args, recompute=recompute)
    g, = torch.autograd.grad(loss, h)
    assert float((g.double() - ref["dH"]).norm() / ref["dH"].norm()) < 1e-2
    with torch.no_grad():
        loss2, _, _ = flce.topk_distill_loss(h, W, *args, recompute=recompute)
    assert not loss2.requires_grad and float(loss2) == pytest.approx(ref["loss"], rel=1e-4)


def test_the_loss_falls_along_its_gradient():
    """A difference of the kernels' own loss along the kernels' own gradient."""
    c = make(64, 128, 800, 16, seed=11, whole=True)
    args = (c["ids"], c["logits"], c["lse_t"], None, None, True)
    one = flce.topk_kd_forward_backward(c["h"], c["W"], *args)
    d = one["dW"] / one["dW"].norm()
    step = 0.25
    Wp, Wm = (c["W"].float() + s * step * d for s in (1, -1))
    # bf16 heads on either side: the step that was really taken
    taken = (Wp.bfloat16().double() - Wm.bfloat16().double())
    up, dn = (float(flce.topk_kd_forward(c["h"], w.bfloat16(), *args)["loss"]) for w in (Wp, Wm))
    want = float((one["dW"].double() * taken).sum())
    assert up - dn == pytest.approx(want, rel=0.05)


def test_repeatable_and_on_another_stream():
    c = make(600, 128, 2000, 20, seed=12, mask=True, whole=True)
    args = (c["h"], c["W"], c["ids"], c["logits"], c["lse_t"], c["targets"], None, True)
    a = flce.topk_kd_forward_backward(*args)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        b = flce.topk_kd_forward_backward(*args)
    d = flce.topk_kd_forward_backward(*args, stream=side)  # the library's own workspace on that stream
    side.synchronize()
    for x in (b, d):
        assert all(torch.equal(a[k], x[k]) for k in ("kl", "lse", "loss", "n_valid", "dH", "dW"))


def test_graph_capture():
    c = make(300, 128, 2000, 20, seed=13, mask=True, whole=True)
    args = (c["h"], c["W"], c["ids"], c["logits"], c["lse_t"], c["targets"], None, True)

    def step():
        one = flce.topk_kd_forward_backward(*args)
        out = flce.topk_kd_forward(*args, for_backward=True)
        dH, dW = flce.topk_kd_backward(c["h"], c["W"], out["state"], 20, 1.0, count=out["n_valid"])
        return [one[k] for k in ("kl", "loss", "dH", "dW")] + [out["kl"], out["loss"], dH, dW]

    eager = [t.clone() for t in step()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, eager))
    c["h"].copy_(c["h"].flip(0))
    c["ids"].copy_(c["ids"].flip(0))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, step()))


def test_past_32_bit_offsets():
    """N V past 2^31: the last rows against the definition."""
    N, H, V, K = 16500, 64, 131072, 4
    g = torch.Generator(device="cuda").manual_seed(14)
    h = torch.randn(N, H, generator=g, device="cuda").bfloat16()
    W = (0.1 * torch.randn(V, H, generator=g, device="cuda")).bfloat16()
    ids = torch.randint(0, V, (N, K), generator=g, device="cuda")
    logits = torch.randn(N, K, generator=g, device="cuda")
    targets = torch.zeros(N, dtype=torch.int64, device="cuda")
    out = flce.topk_kd_forward(h, W, ids, logits)
    s = slice(N - 40, N)
    ref = R.reference(h[s], W, ids[s], logits[s])
    R.check({k: out[k][s] for k in ("kl", "lse")}, ref)
    one = flce.topk_kd_forward_backward(h, W, ids, logits, targets=targets, need_dW=False)
    R.check({"kl": one["kl"][s], "dH": (one["dH"][s].double() * (N / 40)).bfloat16()}, ref, roundings=2)


def test_workspace_of_the_caller_is_enough():
    c = make(500, 64, 1500, 8, seed=15, whole=True)
    K = 8
    ws = torch.empty(_lib.flce_topk_kd_workspace_bytes(500, 64, 1500, K, 256), dtype=torch.uint8, device="cuda")
    a = flce.topk_kd_forward(c["h"], c["W"], c["ids"], c["logits"], workspace=ws, for_backward=True)
    b = flce.topk_kd_forward(c["h"], c["W"], c["ids"], c["logits"])
    assert torch.equal(a["kl"], b["kl"])
    bws = torch.empty(_lib.flce_topk_kd_backward_workspace_bytes(500, 64, 1500, 256, _lib.DTYPES["bf16"]),
                      dtype=torch.uint8, device="cuda")
    flce.topk_kd_backward(c["h"], c["W"], a["state"], K, 1.0, workspace=bws, dW_dtype=torch.bfloat16)
    with pytest.raises(_lib.FlceError):
        flce.topk_kd_backward(c["h"], c["W"], a["state"], K, 1.0, workspace=bws[:-256], dW_dtype=torch.bfloat16)
    with pytest.raises(_lib.FlceError):
        flce.topk_kd_forward(c["h"], c["W"], c["ids"], c["logits"], workspace=ws[:-256])
    with pytest.raises(ValueError, match="state"):
        flce.topk_kd_backward(c["h"], c["W"], a["state"], K - 1, 1.0)


@pytest.mark.parametrize("N,H,V", [(37, 64, 77825), (200, 264, 80003), (256, 520, 90112), (300, 264, 78001),
                                   (512, 136, 100003)])
@pytest.mark.parametrize("mask", [False, True])
def test_few_rows_of_a_wide_vocabulary(N, H, V, mask):
    """bf16 dW whose units are whole rows of tiles: one to eight K blocks of
    rows, ragged last tiles, rows left out on the device."""
    c = make(N, H, V, 19, seed=11, std=0.05, mask=mask, pad=mask, weights=mask)
    ref = R.reference(**c)
    args = (c["h"], c["W"], c["ids"], c["logits"], c["lse_t"], c["targets"], c["weights"])
    got = flce.topk_kd_forward_backward(*args, chunk_rows=4096, dW_dtype=torch.bfloat16)
    assert _lib.flce_device_status() == 0
    R.check(got, ref, roundings=2)
    again = flce.topk_kd_forward_backward(*args, chunk_rows=4096, dW_dtype=torch.bfloat16)
    assert torch.equal(got["dW"], again["dW"])


def test_no_counted_row_of_a_wide_vocabulary():
    c = make(130, 64, 78001, 5, seed=12)
    got = flce.topk_kd_forward_backward(c["h"], c["W"], c["ids"], c["logits"], None,
                                        torch.full((130,), -100, device="cuda"), chunk_rows=4096,
                                        dW_dtype=torch.bfloat16)
    assert _lib.flce_device_status() == 0
    assert not got["dW"].any() and not got["dH"].any() and int(got["n_valid"]) == 0


@pytest.mark.parametrize("options", [{}, {"cta_group": 1}])
@pytest.mark.parametrize("N,H,V,K,mask", [(1, 64, 1691, 1, False), (3, 760, 5003, 8, True), (64, 136, 3000, 16, False),
                                          (65, 264, 2049, 5, True), (128, 64, 4097, 40, False)])
def test_few_rows_take_their_dlogits_in_two_parts(N, H, V, K, mask, options):
    """dlogits of 16 bits and more: what is left is the rounding of the fp16
    exponentials, half a step of 2^-10 (a quarter of bf16's half step covers it
    and the fp32 sums), where one bf16 rounding is 2^-8."""
    c = make(N, H, V, K, seed=13, whole=True, mask=mask, weights=mask)
    ref = R.reference(**c, tail=True)
    args = (c["h"], c["W"], c["ids"], c["logits"], c["lse_t"], c["targets"], c["weights"], True)
    with _lib.options(**options):
        got = flce.topk_kd_forward_backward(*args, chunk_rows=4096)
        half = flce.topk_kd_forward_backward(*args, chunk_rows=4096, dW_dtype=torch.bfloat16)
    assert _lib.flce_device_status() == 0
    R.check(got, ref, roundings=0.25)
    R.check(half, ref, roundings=0.25)
