"""rms_norm, rms_norm_e4m3 and their backward against the definition in 64
bits, at the lengths and types where a kernel can go wrong."""
import pytest
import torch

import chunked_lm_head_gb300 as flce
from chunked_lm_head_gb300 import _lib

import norm_ref as R

pytestmark = pytest.mark.gpu

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
# fp32 roundings along one value of y: the sum of squares (at most 32 terms in
# a thread, then at most 11 joins), its mean, root and reciprocal, the three
# products: under 2^7 half steps
FP32 = 2 ** 7 * R.EPS24


def make(N, H, residual, weight, offset, seed=0, outlier=True):
    g = torch.Generator(device="cuda").manual_seed(seed + 7919 * N + H)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = rnd(N, H).bfloat16()
    r = None if residual is None else (3 * rnd(N, H)).to(residual)
    if r is not None and outlier and N:
        r[:, 0] = 500.0
    w = (1.0 - offset + 0.2 * rnd(H)).to(weight)
    return x, r, w, rnd


def assert_within(got, want, bound, what):
    bad = ~((got.double() - want).abs() <= bound)
    assert not bool(bad.any()), (what, int(bad.sum()), float((got.double() - want).abs().max()))


SHAPES = [(1, 8), (3, 16), (5, 256), (9, 264), (33, 1000), (8, 1024), (2, 1032), (7, 2048), (5, 2064), (257, 2560),
          (4, 4096), (3, 4112), (6, 8192), (2, 8208), (2, 16384), (3, 32768)]


@pytest.mark.parametrize("residual", [None, BF16, F32], ids=["none", "bf16", "f32"])
@pytest.mark.parametrize("N,H", SHAPES)
def test_forward_matches_the_definition(N, H, residual):
    weight, offset = ((F32, 1.0) if (N + H // 8) % 2 else (BF16, 0.0))
    x, r, w, _ = make(N, H, residual, weight, offset)
    out = flce.rms_norm_forward(x, w, r, eps=1e-5, weight_offset=offset)
    s = R.stream(x, r)
    if r is not None:
        assert torch.equal(out["residual"], s)
    y, rstd = R.forward(s, w, 1e-5, offset)
    assert_within(out["rstd"], rstd, rstd * FP32, "rstd")
    assert_within(out["y"], y, y.abs() * (R.half_step(BF16) + FP32), "y")
    assert _lib.flce_device_status() == 0


@pytest.mark.parametrize("residual", [None, BF16, F32], ids=["none", "bf16", "f32"])
@pytest.mark.parametrize("N,H", [s for s in SHAPES if s[1] % 16 == 0])
def test_e4m3_matches_the_definition(N, H, residual):
    weight, offset = ((F32, 1.0) if (N + H // 8) % 2 else (BF16, 0.0))
    x, r, w, _ = make(N, H, residual, weight, offset)
    out = flce.rms_norm_e4m3(x, w, r, eps=1e-5, weight_offset=offset, need_rstd=True)
    s = R.stream(x, r)
    if r is not None:
        assert torch.equal(out["residual"], s)
    y, rstd = R.forward(s, w, 1e-5, offset)
    assert_within(out["rstd"], rstd, rstd * FP32, "rstd")
    scale = y.abs().amax(1) / 448
    assert_within(out["scale"], scale, scale * FP32, "scale")
    assert out["q"].dtype == E4M3
    # half a step of e4m3, or half the step of its subnormals (2^-9)
    got = out["q"].float().double() * scale[:, None]
    assert_within(got, y, torch.maximum(y.abs() * R.half_step(E4M3), scale[:, None] * 2.0 ** -10)
                  + y.abs() * FP32, "q")
    assert float(out["q"].float().abs().amax(1).min()) == 448.0  # the row's largest value fills the range
    assert _lib.flce_device_status() == 0


def bwd_bound(dy, ds, s, w, offset, eps):
    """fp32 roundings of one d: FP32 of each term's magnitude."""
    sd = s.double()
    rstd = ((sd.square().mean(1) + eps) ** -0.5)[:, None]
    g = (dy.double() * (w.double() + offset)).abs()
    b = rstd * g + sd.abs() * rstd ** 3 * (g * sd.abs()).mean(1, keepdim=True)
    return FP32 * (b if ds is None else b + ds.double().abs())


@pytest.mark.parametrize("residual", [None, BF16, F32], ids=["none", "bf16", "f32"])
@pytest.mark.parametrize("N,H", SHAPES + [(1003, 1000), (2000, 64), (1500, 4096)])
def test_backward_matches_the_definition(N, H, residual):
    weight, offset = ((F32, 1.0) if (N + H // 8) % 2 else (BF16, 0.0))
    x, r, w, rnd = make(N, H, residual, weight, offset)
    for v in (x, r, w):
        if v is not None:
            v.requires_grad_(True)
    dy = rnd(N, H).bfloat16()
    s = R.stream(x.detach(), None if r is None else r.detach())
    if r is None:
        y = flce.rms_norm(x, w, eps=1e-5, weight_offset=offset)
        ds = None
        dx, dw = torch.autograd.grad(y, (x, w), dy)
        dr = None
    else:
        y, stream = flce.rms_norm(x, w, r, eps=1e-5, weight_offset=offset)
        assert torch.equal(stream, s)
        ds = rnd(N, H).to(residual)
        dx, dr, dw = torch.autograd.grad((y, stream), (x, r, w), (dy, ds))
    d, dweight = R.backward(dy, ds, s, w.detach(), 1e-5, offset)
    b = bwd_bound(dy, ds, s, w.detach(), offset, 1e-5)
    assert dx.dtype == BF16 and dw.dtype == weight
    assert_within(dx, d, d.abs() * R.half_step(BF16) + 1.01 * b, "dx")
    if r is not None:
        assert dr.dtype == residual
        assert_within(dr, d, d.abs() * R.half_step(residual) + 1.01 * b, "dr")
    # dweight: N terms of FP32-accurate value, summed in fp32 in some order
    sd = s.double()
    terms = (dy.double().abs() * sd.abs() * ((sd.square().mean(1) + 1e-5) ** -0.5)[:, None]).sum(0)
    assert_within(dw, dweight, dweight.abs() * R.half_step(weight) + 1.01 * terms * (FP32 + N * R.EPS24), "dweight")
    assert _lib.flce_device_status() == 0


def test_gradient_matches_differences():
    """The kernels' gradient along a random direction against the central
    difference of the definition in 64 bits."""
    N, H, eps, offset = 6, 264, 1e-5, 1.0
    x, r, w, rnd = make(N, H, F32, F32, offset, outlier=False)
    for v in (x, r, w):
        v.requires_grad_(True)
    dy, ds = rnd(N, H).bfloat16(), rnd(N, H)
    y, stream = flce.rms_norm(x, w, r, eps=eps, weight_offset=offset)
    dx, dr, dw = torch.autograd.grad((y, stream), (x, r, w), (dy, ds))
    ur, uw = rnd(N, H).double(), rnd(H).double()

    def loss(t):
        s = (x.detach().float() + r.detach()).double() + t * ur
        yy, _ = R.forward(s, w.detach().double() + t * uw, eps, offset)
        return (yy * dy.double()).sum() + (s * ds.double()).sum()

    step = 1e-5
    diff = float((loss(step) - loss(-step)) / (2 * step))
    got = float((dr.double() * ur).sum() + (dw.double() * uw).sum())
    # the difference's own error: step^2 of third derivatives of size one, and
    # 2^-52 of the loss's terms over the step
    size = float((dr.double() * ur).abs().sum() + (dw.double() * uw).abs().sum())
    assert abs(got - diff) <= 1e-5 * size, (got, diff)


def test_rows_out_of_a_wider_buffer_and_expanded_gradients():
    N, H = 37, 1040
    x, r, w, rnd = make(N, H, BF16, BF16, 0.0)
    wide = torch.zeros(N, H + 48, dtype=BF16, device="cuda")
    wide[:, 16:16 + H] = x
    wr = torch.zeros(2 * N, H, dtype=BF16, device="cuda")
    wr[::2] = r
    a = flce.rms_norm_forward(wide[:, 16:16 + H], w, wr[::2])
    b = flce.rms_norm_forward(x, w, r)
    assert torch.equal(a["y"], b["y"]) and torch.equal(a["residual"], b["residual"])
    qa, qb = flce.rms_norm_e4m3(wide[:, 16:16 + H], w, wr[::2]), flce.rms_norm_e4m3(x, w, r)
    assert torch.equal(qa["q"].view(torch.uint8), qb["q"].view(torch.uint8)) and torch.equal(qa["scale"], qb["scale"])
    # the stream as rows of a wider buffer, without a residual
    xs = wide[:, 16:16 + H].requires_grad_(True)
    one = torch.ones((), dtype=BF16, device="cuda").expand(N, H)  # an upstream gradient of stride 0
    g1, = torch.autograd.grad(flce.rms_norm(xs, w), xs, one)
    xc = x.clone().requires_grad_(True)
    g2, = torch.autograd.grad(flce.rms_norm(xc, w), xc, one.contiguous())
    assert torch.equal(g1, g2)
    with pytest.raises(ValueError, match="contiguous rows"):
        flce.rms_norm(x.t(), w)
    with pytest.raises(_lib.FlceError):  # rows that are not 16-byte aligned
        flce.rms_norm(wide[:, 1:1 + H], w)


def test_zero_rows_infinities_and_nan():
    H = 512
    x = torch.randn(5, H, device="cuda").bfloat16()
    w = torch.ones(H, dtype=BF16, device="cuda")
    x[1] = 0
    x[2, 7] = float("inf")
    x[3, 9] = float("nan")
    y = flce.rms_norm(x, w).float()
    assert torch.isfinite(y[[0, 1, 4]]).all() and not y[1].any()
    assert torch.isnan(y[2, 7]) and int(torch.isnan(y[2]).sum()) == 1 and not y[2].nan_to_num().any()
    assert torch.isnan(y[3]).all()
    out = flce.rms_norm_e4m3(x, w)
    q, scale = out["q"].float(), out["scale"]
    assert scale[1] == 1 and scale[2] == 1 and scale[3] == 1
    assert not q[1].any() and torch.isnan(q[2, 7]) and int(torch.isnan(q[2]).sum()) == 1
    assert torch.isnan(q[3]).all() and torch.isfinite(q[[0, 4]]).all()


def test_no_rows_and_partial_gradients():
    w = torch.ones(64, device="cuda").requires_grad_(True)
    x0 = torch.empty(0, 64, dtype=BF16, device="cuda").requires_grad_(True)
    y = flce.rms_norm(x0, w)
    gx, gw = torch.autograd.grad(y, (x0, w), torch.empty_like(y))
    assert gx.shape == (0, 64) and not gw.any()
    assert flce.rms_norm_e4m3(x0.detach(), w.detach())["scale"].shape == (0,)
    # only the stream's gradient; only the norm's; only the weight's
    x, r, w2, rnd = make(6, 64, F32, F32, 0.0)
    x.requires_grad_(True), r.requires_grad_(True)
    y, s = flce.rms_norm(x, w2, r)
    ds = rnd(6, 64)
    gx, gr = torch.autograd.grad(s, (x, r), ds)
    assert torch.equal(gr, ds) and torch.equal(gx, ds.bfloat16())
    w2.requires_grad_(True)
    y, s = flce.rms_norm(x.detach(), w2, r.detach())
    dy = rnd(6, 64).bfloat16()
    gw, = torch.autograd.grad(y, w2, dy)
    sd = s.detach().double()
    terms = (dy.double() * sd).abs().mul((sd.square().mean(1) + 1e-6)[:, None] ** -0.5).sum(0)
    assert_within(gw, R.backward(dy, None, s.detach(), w2.detach(), 1e-6, 0.0)[1], terms * (FP32 + 6 * R.EPS24),
                  "dweight alone")


def test_another_stream_and_repeatability():
    x, r, w, rnd = make(300, 2048, BF16, BF16, 0.0)
    dy = rnd(300, 2048).bfloat16()
    ref = flce.rms_norm_forward(x, w, r)
    g = flce.rms_norm_backward(dy, ref["residual"], w, ref["rstd"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out = flce.rms_norm_forward(x, w, r)
        g2 = flce.rms_norm_backward(dy, out["residual"], w, out["rstd"])
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out["y"], ref["y"]) and all(torch.equal(a, b) for a, b in zip(g, g2))


def test_graph_capture_of_forward_and_backward():
    x, r, w, rnd = make(200, 1024, BF16, F32, 0.0)
    dy, ds = rnd(200, 1024).bfloat16(), rnd(200, 1024).bfloat16()
    ws = torch.empty(_lib.flce_rms_norm_backward_workspace_bytes(200, 1024), dtype=torch.uint8, device="cuda")

    def step():
        out = flce.rms_norm_forward(x, w, r)
        return (out["y"],) + flce.rms_norm_backward(dy, out["residual"], w, out["rstd"], ds, workspace=ws)

    eager = [t.clone() for t in step()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, eager))
    x.copy_(x.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, step()))


def test_long_rows_past_32_bit_offsets():
    """Rows whose element offset passes 2^31."""
    N, H = 66000, 32768
    x = torch.zeros(N, H, dtype=BF16, device="cuda")
    x[-3:] = torch.randn(3, H, device="cuda").bfloat16()
    w = torch.ones(H, dtype=BF16, device="cuda")
    y = flce.rms_norm(x, w)
    want, _ = R.forward(x[-3:], w, 1e-6, 0.0)
    assert_within(y[-3:], want, want.abs() * (R.half_step(BF16) + FP32), "y")
    assert not y[: N - 3].any()
    del y
    q = flce.rms_norm_e4m3(x, w)["q"]
    assert float(q[-3:].float().abs().max()) == 448.0
