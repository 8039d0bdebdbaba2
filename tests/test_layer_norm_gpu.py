"""layer_norm and its backward against the definition in 64 bits, at the lengths
and types where a kernel can go wrong."""
import pytest
import torch

import chunked_lm_head_gb300 as flce
from chunked_lm_head_gb300 import _lib

import layer_ref as R

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
EPS = 1e-5


def make(N, H, residual, weight, offset, bias, seed=0, shift=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed + 7919 * N + H)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = (rnd(N, H) + shift).bfloat16()
    r = None if residual is None else (3 * rnd(N, H) + 1).to(residual)
    if r is not None and N:
        r[:, 0] = 500.0
    w = (1.0 - offset + 0.2 * rnd(H)).to(weight)
    b = (0.3 * rnd(H)).to(weight) if bias else None
    return x, r, w, b, rnd


def assert_within(got, want, bound, what):
    bad = ~((got.double() - want).abs() <= bound)
    assert not bool(bad.any()), (what, int(bad.sum()), float((got.double() - want).abs().max()))


def variant(N, H):
    """Type of the parameters, offset and bias: each met with each shape of kernel."""
    k = N + H // 8
    return (F32 if k % 2 else BF16), (1.0 if k % 3 == 0 else 0.0), k % 4 != 1


SHAPES = [(1, 8), (3, 16), (5, 256), (9, 264), (33, 1000), (8, 1024), (2, 1032), (7, 2048), (5, 2064), (257, 2560),
          (4, 4096), (3, 4112), (6, 8192), (2, 8208), (2, 16384), (1, 16392), (3, 32768)]


@pytest.mark.parametrize("residual", [None, BF16, F32], ids=["none", "bf16", "f32"])
@pytest.mark.parametrize("N,H", SHAPES)
def test_forward_matches_the_definition(N, H, residual):
    weight, offset, bias = variant(N, H)
    x, r, w, b, _ = make(N, H, residual, weight, offset, bias)
    out = flce.layer_norm_forward(x, w, b, r, eps=EPS, weight_offset=offset)
    s = R.stream(x, r)
    if r is not None:
        assert torch.equal(out["residual"], s)
    y, mean, rstd = R.forward(s, w, b, EPS, offset)
    assert_within(out["mean"], mean, R.FP32 * s.double().abs().mean(1), "mean")
    # the variance is about the mean found: its error is the mean's squared, below the other roundings
    assert_within(out["rstd"], rstd, rstd * 2 * R.FP32, "rstd")
    assert_within(out["y"], y, 1.01 * y.abs() * R.half_step(BF16) + 2 * R.forward_bound(s, w, b, EPS, offset), "y")
    assert _lib.flce_device_status() == 0


@pytest.mark.parametrize("residual", [None, BF16, F32], ids=["none", "bf16", "f32"])
@pytest.mark.parametrize("N,H", SHAPES + [(1003, 1000), (2000, 64), (1500, 4096)])
def test_backward_matches_the_definition(N, H, residual):
    weight, offset, bias = variant(N, H)
    x, r, w, b, rnd = make(N, H, residual, weight, offset, bias)
    for v in (x, r, w, b):
        if v is not None:
            v.requires_grad_(True)
    dy = rnd(N, H).bfloat16()
    s = R.stream(x.detach(), None if r is None else r.detach())
    out = flce.layer_norm(x, w, b, r, eps=EPS, weight_offset=offset)
    ds = None
    if r is not None:
        assert torch.equal(out[1], s)
        ds = rnd(N, H).to(residual)
    names = [k for k, v in (("x", x), ("r", r), ("w", w), ("b", b)) if v is not None]
    grads = dict(zip(names, torch.autograd.grad(out, [dict(x=x, r=r, w=w, b=b)[k] for k in names],
                                                dy if ds is None else (dy, ds))))
    d, dweight, dbias = R.backward(dy, ds, s, w.detach(), EPS, offset)
    bd, bw, bb = R.backward_bounds(dy, ds, s, w.detach(), EPS, offset)
    assert grads["x"].dtype == BF16 and grads["w"].dtype == weight
    assert_within(grads["x"], d, 1.01 * d.abs() * R.half_step(BF16) + 2 * bd, "dx")
    if r is not None:
        assert grads["r"].dtype == residual
        assert_within(grads["r"], d, 1.01 * d.abs() * R.half_step(residual) + 2 * bd, "dr")
    assert_within(grads["w"], dweight, 1.01 * dweight.abs() * R.half_step(weight) + bw, "dweight")
    if bias:
        assert_within(grads["b"], dbias, 1.01 * dbias.abs() * R.half_step(weight) + bb, "dbias")
    assert _lib.flce_device_status() == 0


def test_rows_far_from_zero_keep_their_variance():
    """Rows about 300 with a spread of 2: a sum of squares less a squared mean would lose the spread's bits."""
    N, H = 64, 2048
    x, r, w, b, rnd = make(N, H, F32, F32, 0.0, True)
    r = 300.0 + 2.0 * rnd(N, H)
    out = flce.layer_norm_forward(x, w, b, r, eps=EPS)
    s = R.stream(x, r)
    y, mean, rstd = R.forward(s, w, b, EPS, 0.0)
    assert_within(out["rstd"], rstd, rstd * 2 * R.FP32, "rstd")
    assert_within(out["y"], y, 1.01 * y.abs() * R.half_step(BF16) + 2 * R.forward_bound(s, w, b, EPS, 0.0), "y")


@pytest.mark.parametrize("residual", [None, BF16], ids=["none", "bf16"])
@pytest.mark.parametrize("N,H", [(3, 264), (5, 4096), (4, 8192)])
def test_constant_rows_give_the_bias(N, H, residual):
    """No variance: n is 0, y the bias, and the gradients are finite."""
    x = torch.full((N, H), 1.5, device="cuda", dtype=BF16, requires_grad=True)
    r = None if residual is None else torch.full((N, H), 0.25, device="cuda", dtype=residual)
    w = torch.ones(H, device="cuda")
    b = torch.randn(H, device="cuda")
    out = flce.layer_norm(x, w, b, r, eps=EPS)
    y = out if r is None else out[0]
    assert torch.equal(y, b.bfloat16().expand(N, H))
    (dx,) = torch.autograd.grad(y, (x,), torch.randn(N, H, device="cuda").bfloat16())
    assert bool(torch.isfinite(dx).all())


def test_rows_out_of_a_wider_buffer_and_a_single_row_of_any_stride():
    N, H = 37, 1000
    x, r, w, b, rnd = make(N, 2 * H, F32, BF16, 0.0, False)
    xs, rs, ws = x[:, 8:8 + H], r[:, 4:4 + H], w[:H].contiguous()
    got = flce.layer_norm_forward(xs, ws, None, rs, eps=EPS)
    want = flce.layer_norm_forward(xs.contiguous(), ws, None, rs.contiguous(), eps=EPS)
    for k in ("y", "residual", "mean", "rstd"):
        assert torch.equal(got[k], want[k]), k
    xs = xs.detach().requires_grad_(True)
    dy = rnd(N, H).bfloat16()
    a = torch.autograd.grad(flce.layer_norm(xs, ws), xs, dy)[0]
    c = xs.detach().contiguous().requires_grad_(True)
    assert torch.equal(a, torch.autograd.grad(flce.layer_norm(c, ws), c, dy)[0])
    with pytest.raises(ValueError):  # columns apart
        flce.layer_norm(x[:, ::2], ws)
    flce.layer_norm(x[:1, :H], ws)


@pytest.mark.parametrize("which", ["x", "w", "b", "r", "wb", "xr"])
def test_only_the_wanted_gradients(which):
    N, H = 50, 512
    x, r, w, b, rnd = make(N, H, F32, F32, 0.0, True)
    dy, ds = rnd(N, H).bfloat16(), rnd(N, H)
    t = dict(x=x, r=r, w=w, b=b)
    full = {k: v.clone().requires_grad_(True) for k, v in t.items()}
    grads = dict(zip("xrwb", torch.autograd.grad(flce.layer_norm(full["x"], full["w"], full["b"], full["r"]),
                                                 [full[k] for k in "xrwb"], (dy, ds))))
    some = {k: v.clone().requires_grad_(k in which) for k, v in t.items()}
    y, s = flce.layer_norm(some["x"], some["w"], some["b"], some["r"])
    got = torch.autograd.grad((y, s), [some[k] for k in which], (dy, ds))
    for k, g in zip(which, got):
        assert torch.equal(g, grads[k]), k


def test_gradients_that_reach_one_output_only():
    N, H = 20, 264
    x, r, w, b, rnd = make(N, H, BF16, F32, 0.0, True)
    for v in (x, r, w, b):
        v.requires_grad_(True)
    y, s = flce.layer_norm(x, w, b, r)
    ds = rnd(N, H).bfloat16()
    dx, dr = torch.autograd.grad(s, (x, r), ds, retain_graph=True)
    assert torch.equal(dx, ds) and torch.equal(dr, ds)
    dy = rnd(N, H).bfloat16()
    dx, dw = torch.autograd.grad(y, (x, w), dy)
    d, dweight, _ = R.backward(dy, None, s.detach(), w.detach(), EPS, 0.0)
    bd, bw, _ = R.backward_bounds(dy, None, s.detach(), w.detach(), EPS, 0.0)
    assert_within(dx, d, 1.01 * d.abs() * R.half_step(BF16) + 2 * bd, "dx")
    assert_within(dw, dweight, 1.01 * dweight.abs() * R.half_step(F32) + bw, "dw")


def test_gradients_as_expanded_and_unaligned_views():
    N, H = 9, 520
    x, _, w, b, rnd = make(N, H, None, BF16, 0.0, True)
    x.requires_grad_(True)
    row = rnd(H).bfloat16()
    a = torch.autograd.grad(flce.layer_norm(x, w, b), x, row.expand(N, H))[0]
    flat = torch.zeros(N * H + 1, device="cuda", dtype=BF16)
    flat[1:] = row.repeat(N)
    c = torch.autograd.grad(flce.layer_norm(x, w, b), x, flat[1:].view(N, H))[0]
    assert torch.equal(a, c)


def test_no_rows():
    x = torch.empty(0, 64, device="cuda", dtype=BF16, requires_grad=True)
    w = torch.ones(64, device="cuda", requires_grad=True)
    b = torch.zeros(64, device="cuda", requires_grad=True)
    y = flce.layer_norm(x, w, b)
    dx, dw, db = torch.autograd.grad(y, (x, w, b), torch.empty_like(y))
    assert y.shape == (0, 64) and dx.shape == (0, 64)
    assert not bool(dw.any()) and not bool(db.any())


def test_same_bits_each_time_and_on_another_stream():
    N, H = 3000, 1536
    x, r, w, b, rnd = make(N, H, BF16, F32, 0.0, True)
    dy = rnd(N, H).bfloat16()

    def step():
        f = flce.layer_norm_forward(x, w, b, r)
        return [f["y"]] + list(flce.layer_norm_backward(dy, f["residual"], w, f["mean"], f["rstd"]))

    first = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = step()
    side.synchronize()
    for a, c in zip(first, second):
        assert torch.equal(a, c)
    # a caller's stream and workspace
    ws = torch.empty(_lib.flce_layer_norm_backward_workspace_bytes(N, H), dtype=torch.uint8, device="cuda")
    f = flce.layer_norm_forward(x, w, b, r, stream=side)
    third = flce.layer_norm_backward(dy, f["residual"], w, f["mean"], f["rstd"], workspace=ws, stream=side)
    side.synchronize()
    for a, c in zip(first[1:], third):
        assert torch.equal(a, c)


def test_capture_and_replay():
    N, H = 700, 1000
    x, r, w, b, rnd = make(N, H, F32, BF16, 1.0, True)
    dy, ds = rnd(N, H).bfloat16(), rnd(N, H)

    def step():
        t = [v.detach().requires_grad_(True) for v in (x, r, w, b)]  # leaves of this step's own
        y, s = flce.layer_norm(t[0], t[2], t[3], t[1], weight_offset=1.0)
        grads = torch.autograd.grad((y, s), t, (dy, ds))
        return [y.detach(), s.detach(), *grads]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    x.copy_(rnd(N, H).bfloat16())
    graph.replay()
    torch.cuda.synchronize()
    for a, c in zip(captured, step()):
        assert torch.equal(a, c)


def test_a_second_derivative_is_refused():
    x = torch.randn(4, 64, device="cuda").bfloat16().requires_grad_(True)
    w = torch.ones(64, device="cuda", requires_grad=True)
    (dx,) = torch.autograd.grad(flce.layer_norm(x, w).float().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="second derivative"):
        dx.float().sum().backward()


def test_module():
    m = flce.LayerNorm(256, device="cuda")
    x = torch.randn(5, 256, device="cuda").bfloat16()
    y = m(x)
    y.float().sum().backward()
    assert m.weight.grad.shape == (256,) and torch.equal(m.bias.grad, torch.full_like(m.bias, 5.0))
    assert flce.LayerNorm(256, bias=False).bias is None


@pytest.mark.parametrize("residual", [None, BF16], ids=["none", "bf16"])
def test_rows_past_32_bit_offsets(residual):
    """N H beyond 2^31: the last rows as a call of their own gives them."""
    N, H, n = 1045000, 2064, 37
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(n, H, generator=g, device="cuda").bfloat16()
    dy = torch.randn(n, H, generator=g, device="cuda").bfloat16()
    w = torch.randn(H, generator=g, device="cuda")
    many = torch.zeros(N, H, device="cuda", dtype=BF16)
    many[-n:] = x
    dys = torch.zeros(N, H, device="cuda", dtype=BF16)
    dys[-n:] = dy
    r = None if residual is None else many.clone()
    a = flce.layer_norm_forward(many, w, None, r, eps=EPS)
    b = flce.layer_norm_forward(x, w, None, None if r is None else x, eps=EPS)
    for k in ("y", "residual", "mean", "rstd"):
        if a[k] is not None:
            assert torch.equal(a[k][-n:], b[k]), k
    assert not bool(a["y"][:1000].any())
    sa, sb = (many, x) if r is None else (a["residual"], b["residual"])
    ga = flce.layer_norm_backward(dys, sa, w, a["mean"], a["rstd"])
    gb = flce.layer_norm_backward(dy, sb, w, b["mean"], b["rstd"])
    assert torch.equal(ga[0][-n:], gb[0]) and not bool(ga[0][:1000].any())
    _, dweight, dbias = R.backward(dy, None, sb, w, EPS, 0.0)
    _, bw, bb = R.backward_bounds(dy, None, sb, w, EPS, 0.0)
    assert_within(ga[2], dweight, 1.01 * dweight.abs() * R.half_step(F32) + bw, "dw")
    assert_within(ga[3], dbias, 1.01 * dbias.abs() * R.half_step(F32) + bb, "db")
    assert _lib.flce_device_status() == 0
