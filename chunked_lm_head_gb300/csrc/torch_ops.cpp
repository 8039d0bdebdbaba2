// The layer norm and the scores as PyTorch operators (torch.ops.flce).  A call on few
// rows is bound by its host work: a training step of 1,003 x 1,000 took 248 us with
// its autograd node in Python, 100 of them on the engine's own thread, whose caches
// are cold, and takes 177 this way.  Marshalling only, as the ctypes binding: the arithmetic runs
// behind include/flce.h, whose entry points `bind` takes from the library that the
// binding has loaded.  The callers in Python check the tensors, and say what is wrong
// with them; here only what the kernels' reads and writes rest on is checked again.
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/custom_function.h>
#include <torch/csrc/autograd/variable.h>
#include <torch/library.h>

#include <string>
#include <vector>

#include "flce.h"

namespace {

using at::Tensor;
using torch::autograd::AutogradContext;
using torch::autograd::Function;
using torch::autograd::variable_list;

struct Api {
  decltype(&flce_layer_norm) layer_norm = nullptr;
  decltype(&flce_layer_norm_backward) layer_norm_backward = nullptr;
  decltype(&flce_layer_norm_backward_workspace_bytes) layer_norm_backward_workspace_bytes = nullptr;
  decltype(&flce_score) score = nullptr;
  decltype(&flce_score_workspace_bytes) score_workspace_bytes = nullptr;
  decltype(&flce_score_state_bytes) score_state_bytes = nullptr;
  decltype(&flce_score_backward) score_backward = nullptr;
  decltype(&flce_score_backward_workspace_bytes) score_backward_workspace_bytes = nullptr;
  decltype(&flce_status_string) status_string = nullptr;
};
Api g_api;

template <class F>
void take(F& f, int64_t address) {
  f = reinterpret_cast<F>(address);
}
void bind(at::IntArrayRef a) {
  TORCH_CHECK(a.size() == 9, "flce: nine entry points are expected");
  take(g_api.layer_norm, a[0]);
  take(g_api.layer_norm_backward, a[1]);
  take(g_api.layer_norm_backward_workspace_bytes, a[2]);
  take(g_api.score, a[3]);
  take(g_api.score_workspace_bytes, a[4]);
  take(g_api.score_state_bytes, a[5]);
  take(g_api.score_backward, a[6]);
  take(g_api.score_backward_workspace_bytes, a[7]);
  take(g_api.status_string, a[8]);
}

// Tensors whose addresses a kernel may take: of one type, on x's device, rows
// without gaps but for a row stride.
void expect(const Tensor& t, const Tensor& x, bool type, at::IntArrayRef shape, bool rows = false) {
  if (!t.defined()) return;
  TORCH_CHECK(t.is_cuda() && t.device() == x.device() && type && t.sizes() == shape &&
                  (t.is_contiguous() || (rows && t.stride(1) == 1 && t.stride(0) >= t.size(1))),
              "flce: an argument has another device, type, shape or layout than the operator takes");
}
bool is_bf16(const Tensor& t) { return t.defined() && t.scalar_type() == at::kBFloat16; }
bool is_parameter(const Tensor& t) { return t.defined() && (t.scalar_type() == at::kFloat || is_bf16(t)); }

void check(const char* fn, flce_status s) {
  TORCH_CHECK(s == FLCE_OK, fn, " failed: ", g_api.status_string(s));
}

int32_t kind(const Tensor& t) { return t.scalar_type() == at::kFloat ? FLCE_F32 : FLCE_BF16; }
void* data(const Tensor& t) { return t.defined() && t.numel() > 0 ? t.data_ptr() : nullptr; }
flce_bf16* bf16(const Tensor& t) { return static_cast<flce_bf16*>(data(t)); }
float* f32(const Tensor& t) { return static_cast<float*>(data(t)); }
// the current stream of the tensors' device, which is the current one
void* stream() { return c10::cuda::getCurrentCUDAStream().stream(); }
// (torch's allocator orders a workspace's reuse on the current stream)
Tensor bytes(size_t n, const Tensor& like) {
  return at::empty({static_cast<int64_t>(n)}, like.options().dtype(at::kByte));
}
// A gradient as the kernels read it: contiguous, from a 16-byte boundary on (a part
// of a flat buffer may start anywhere).
Tensor rows_of(const Tensor& g) {
  if (!g.defined()) return g;
  Tensor c = g.contiguous();
  return reinterpret_cast<uintptr_t>(c.data_ptr()) % 16 == 0 ? c : c.clone();
}

// Gradients that kernels formed without a graph, tied to the tensors they depend
// on: differentiating them again is refused, not taken for zero.
struct NoSecondDerivative : Function<NoSecondDerivative> {
  static variable_list forward(AutogradContext*, int64_t n, at::TensorList all) {
    variable_list out;
    for (int64_t i = 0; i < n; ++i) out.push_back(all[i].view_as(all[i]));
    return out;
  }
  static variable_list backward(AutogradContext*, variable_list) {
    TORCH_CHECK(false, "this gradient has no second derivative: it comes from a kernel, without a graph");
  }
};

// grads (each may be undefined) as a backward returns them: under create_graph
// tied to the inputs.
variable_list first_order(variable_list grads, const variable_list& inputs) {
  if (!at::GradMode::is_enabled()) return grads;
  std::vector<Tensor> all;
  for (const Tensor& g : grads)
    if (g.defined()) all.push_back(g);
  const int64_t n = static_cast<int64_t>(all.size());
  if (n == 0) return grads;
  for (const Tensor& x : inputs)
    if (x.defined()) all.push_back(x);
  variable_list tied = NoSecondDerivative::apply(n, at::TensorList(all));
  size_t k = 0;
  for (Tensor& g : grads)
    if (g.defined()) g = tied[k++];
  return grads;
}

// gradients of a node's inputs: as many as it may have (those past the last input
// are undefined, and dropped)
constexpr size_t kInputs = 16;

int64_t row_stride(const Tensor& x) { return x.size(0) > 1 ? x.stride(0) : x.size(1); }

// y, and with a residual the stream; stats [2,N] (mean, rstd) where they are wanted.
variable_list run_layer_norm(const Tensor& x, const Tensor& weight, const Tensor& b, const Tensor& r, double eps,
                             double weight_offset, Tensor* stats) {
  TORCH_CHECK(x.dim() == 2 && g_api.layer_norm, "flce: a matrix is expected, and bound entry points");
  const int64_t N = x.size(0), H = x.size(1);
  expect(x, x, is_bf16(x), {N, H}, true);
  expect(r, x, is_parameter(r), {N, H}, true);
  expect(weight, x, is_parameter(weight), {H});
  expect(b, x, b.defined() && b.scalar_type() == weight.scalar_type(), {H});
  Tensor y = at::empty({N, H}, x.options());
  Tensor s = r.defined() ? at::empty({N, H}, r.options()) : Tensor();
  if (stats) *stats = at::empty({2, N}, x.options().dtype(at::kFloat));
  float* mean = stats ? f32(*stats) : nullptr;
  check("flce_layer_norm",
        g_api.layer_norm(bf16(x), row_stride(x), data(r), r.defined() ? row_stride(r) : 0, r.defined() ? kind(r) : 0,
                         data(weight), data(b), kind(weight), static_cast<float>(weight_offset), static_cast<float>(eps),
                         N, H, bf16(y), data(s), mean, mean ? mean + N : nullptr, stream()));
  return r.defined() ? variable_list{y, s} : variable_list{y};
}

// Whether a graph is to be built.  A leaf that an eager graph still holds passes its
// gradient on the stream of that graph; where that is the default one and this call
// is being captured, the backward's wait between the two would end the capture and
// the process with it, so the call is refused while that can be told.
bool wanted(std::initializer_list<const Tensor*> inputs) {
  if (!at::GradMode::is_enabled()) return false;
  bool any = false;
  for (const Tensor* t : inputs) any |= t->defined() && t->requires_grad();
  if (!any || c10::cuda::currentStreamCaptureStatusMayInitCtx() == c10::cuda::CaptureStatus::None) return any;
  for (const Tensor* t : inputs) {
    if (!t->defined() || !t->requires_grad() || !t->is_leaf()) continue;
    const auto node = torch::autograd::impl::try_get_grad_accumulator(*t);
    const auto on = node ? node->stream() : std::nullopt;
    TORCH_CHECK(!on || *on != c10::cuda::getDefaultCUDAStream(on->device_index()).unwrap(),
                "an eager graph of a leaf of this call is alive: drop it (the losses and outputs made of it) before "
                "the call is captured");
  }
  return true;
}

struct LayerNorm : Function<LayerNorm> {
  static variable_list forward(AutogradContext* ctx, const Tensor& x, const Tensor& weight,
                               const std::optional<Tensor>& bias, const std::optional<Tensor>& residual, double eps,
                               double weight_offset) {
    ctx->set_materialize_grads(false);
    const Tensor b = bias.value_or(Tensor()), r = residual.value_or(Tensor());
    Tensor stats;
    variable_list out = run_layer_norm(x, weight, b, r, eps, weight_offset, &stats);
    ctx->save_for_backward({r.defined() ? out[1] : x, weight, stats});
    ctx->saved_data["offset"] = weight_offset;
    ctx->saved_data["bias"] = b.defined();
    ctx->saved_data["residual"] = r.defined();
    return out;
  }

  static variable_list backward(AutogradContext* ctx, variable_list grads) {
    const variable_list saved = ctx->get_saved_variables();
    const Tensor &s = saved[0], &weight = saved[1], &stats = saved[2];
    const bool has_b = ctx->saved_data["bias"].toBool(), has_r = ctx->saved_data["residual"].toBool();
    // (edges: the tensors that were there, in order)
    const bool need_x = ctx->needs_input_grad(0), need_w = ctx->needs_input_grad(1);
    const bool need_b = has_b && ctx->needs_input_grad(2), need_r = has_r && ctx->needs_input_grad(has_b ? 3 : 2);
    const Tensor ds0 = grads.size() > 1 ? grads[1] : Tensor();
    if (!grads[0].defined()) {  // only the stream was used
      if (!ds0.defined()) return variable_list(kInputs);
      variable_list out{need_x ? ds0.to(at::kBFloat16) : Tensor(), Tensor(), Tensor(), need_r ? ds0 : Tensor()};
      out.resize(kInputs);
      return out;
    }
    const Tensor dy = rows_of(grads[0]), ds = rows_of(ds0);
    const int64_t N = s.size(0), H = s.size(1);
    const bool wide = s.scalar_type() == at::kFloat;
    Tensor dx, dr, dw, db, ws;
    if (need_x || (need_r && !wide)) dx = at::empty({N, H}, dy.options());
    if (need_r && wide) dr = at::empty({N, H}, s.options());
    if (need_w) dw = at::empty({H}, weight.options());
    if (need_b) db = at::empty({H}, weight.options());
    if (need_w || need_b) ws = bytes(g_api.layer_norm_backward_workspace_bytes(N, H), s);
    const float* mean = f32(stats);
    if (dx.defined() || dr.defined() || dw.defined() || db.defined())
      check("flce_layer_norm_backward",
            g_api.layer_norm_backward(bf16(dy), data(s), row_stride(s), kind(s), data(ds), data(weight), kind(weight),
                                      static_cast<float>(ctx->saved_data["offset"].toDouble()), mean,
                                      mean ? mean + N : nullptr, N, H, bf16(dx), f32(dr), data(dw), data(db), data(ws),
                                      ws.defined() ? ws.numel() : 0, stream()));
    variable_list out{need_x ? dx : Tensor(), dw, db, need_r ? (wide ? dr : dx) : Tensor()};
    out = first_order(std::move(out), {s, weight, grads[0], ds0});
    out.resize(kInputs);
    return out;
  }
};

std::vector<Tensor> layer_norm(const Tensor& x, const Tensor& weight, const std::optional<Tensor>& bias,
                               const std::optional<Tensor>& residual, double eps, double weight_offset) {
  const Tensor b = bias.value_or(Tensor()), r = residual.value_or(Tensor());
  if (!wanted({&x, &weight, &b, &r})) return run_layer_norm(x, weight, b, r, eps, weight_offset, nullptr);
  return LayerNorm::apply(x, weight, bias, residual, eps, weight_offset);
}

// the four fields of a flce_logit_transform, or nothing
struct Transform {
  flce_logit_transform t{};
  bool given = false;
  explicit Transform(at::ArrayRef<double> v) : given(v.size() == 4) {
    if (given)
      t = {static_cast<float>(v[0]), static_cast<float>(v[1]), static_cast<float>(v[2]), static_cast<float>(v[3])};
  }
  const flce_logit_transform* get() const { return given ? &t : nullptr; }
};

// flce_score with k words; logp is undefined without targets, ids and words without
// words, state where none is kept (keep_rows 0, or it does not pay).
struct Scores {
  Tensor logp, lse, entropy, ids, words, state;
};
Scores run_score(const Tensor& h, const Tensor& W, const Tensor& targets, int64_t k, int64_t ignore_index,
                 at::ArrayRef<double> transform, int64_t keep_rows) {
  TORCH_CHECK(h.dim() == 2 && W.dim() == 2 && k >= 0 && g_api.score, "flce: matrices are expected, and bound entry points");
  const int64_t N = h.size(0), H = h.size(1), V = W.size(0);
  expect(h, h, is_bf16(h), {N, H});
  expect(W, h, is_bf16(W), {V, H});
  expect(targets, h, targets.defined() && targets.scalar_type() == at::kLong, {N});
  const auto f32_rows = h.options().dtype(at::kFloat);
  Scores o;
  o.lse = at::empty({N}, f32_rows);
  o.entropy = at::empty({N}, f32_rows);
  if (targets.defined()) o.logp = at::empty({N}, f32_rows);
  if (k > 0) {
    o.ids = at::empty({N, k}, h.options().dtype(at::kLong));
    o.words = at::empty({N, k}, f32_rows);
  }
  const size_t kept = keep_rows > 0 ? g_api.score_state_bytes(N, H, V, keep_rows) : 0;
  if (kept) o.state = bytes(kept, h);
  Tensor ws = bytes(g_api.score_workspace_bytes(N, H, V, k), h);
  const Transform tf(transform);
  check("flce_score", g_api.score(bf16(h), bf16(W), static_cast<const int64_t*>(data(targets)), N, H, V, k, ignore_index,
                                  tf.get(), f32(o.logp), f32(o.lse), f32(o.entropy),
                                  static_cast<int64_t*>(data(o.ids)), f32(o.words), data(o.state), data(ws), ws.numel(),
                                  stream()));
  return o;
}

struct Score : Function<Score> {
  static variable_list forward(AutogradContext* ctx, const Tensor& h, const Tensor& W, const Tensor& targets,
                               int64_t chunk_rows, int64_t ignore_index, std::vector<double> transform,
                               bool recompute) {
    ctx->set_materialize_grads(false);
    Scores o = run_score(h, W, targets, 0, ignore_index, transform, recompute ? 0 : chunk_rows);
    ctx->save_for_backward({h, W, targets, o.lse, o.entropy, o.state});
    ctx->saved_data["rows"] = chunk_rows;
    ctx->saved_data["ignore"] = ignore_index;
    ctx->saved_data["transform"] = std::move(transform);
    return {o.logp, o.entropy};
  }

  static variable_list backward(AutogradContext* ctx, variable_list grads) {
    const bool need_h = ctx->needs_input_grad(0), need_W = ctx->needs_input_grad(1);
    if ((!grads[0].defined() && !grads[1].defined()) || !(need_h || need_W)) return variable_list(kInputs);
    const variable_list saved = ctx->get_saved_variables();
    const Tensor &h = saved[0], &W = saved[1], &targets = saved[2], &lse = saved[3], &entropy = saved[4],
                 &state = saved[5];
    const int64_t N = h.size(0), H = h.size(1), V = W.size(0), rows = ctx->saved_data["rows"].toInt();
    auto vector = [](const Tensor& g) { return g.defined() ? g.to(at::kFloat).contiguous() : g; };
    const Tensor ga = vector(grads[0]), ge = vector(grads[1]);
    Tensor dH = need_h ? at::empty({N, H}, h.options()) : Tensor();
    Tensor dW = need_W ? at::empty({V, H}, W.options()) : Tensor();
    Tensor ws = bytes(g_api.score_backward_workspace_bytes(N, H, V, rows, FLCE_BF16), h);
    const std::vector<double> v = ctx->saved_data["transform"].toDoubleVector();
    const Transform tf(v);
    check("flce_score_backward",
          g_api.score_backward(bf16(h), bf16(W), static_cast<const int64_t*>(data(targets)), f32(lse), f32(entropy),
                               f32(ga), f32(ge), data(state), bf16(dH), data(dW), FLCE_BF16, N, H, V, rows,
                               ctx->saved_data["ignore"].toInt(), tf.get(), data(ws), ws.numel(), stream()));
    variable_list out = first_order({dH, dW}, {h, W, grads[0], grads[1]});
    out.resize(kInputs);
    return out;
  }
};

std::vector<Tensor> score(const Tensor& h, const Tensor& W, const Tensor& targets, int64_t chunk_rows,
                          int64_t ignore_index, at::ArrayRef<double> transform, bool recompute) {
  if (!wanted({&h, &W})) {
    Scores o = run_score(h, W, targets, 0, ignore_index, transform, 0);
    return {o.logp, o.entropy};
  }
  return Score::apply(h, W, targets, chunk_rows, ignore_index, transform.vec(), recompute);
}

// ids, words, lse, entropy, and with targets logp
std::vector<Tensor> top(const Tensor& h, const Tensor& W, int64_t k, const std::optional<Tensor>& targets,
                        int64_t ignore_index, at::ArrayRef<double> transform) {
  Scores o = run_score(h, W, targets.value_or(Tensor()), k, ignore_index, transform, 0);
  std::vector<Tensor> out{o.ids, o.words, o.lse, o.entropy};
  if (o.logp.defined()) out.push_back(o.logp);
  return out;
}

}  // namespace

TORCH_LIBRARY(flce, m) {
  m.def("bind(int[] entry_points) -> ()", &bind);
  m.def("layer_norm(Tensor x, Tensor weight, Tensor? bias, Tensor? residual, float eps, float weight_offset) -> Tensor[]",
        &layer_norm);
  m.def("score(Tensor h, Tensor W, Tensor targets, int chunk_rows, int ignore_index, float[] transform, bool recompute)"
        " -> Tensor[]", &score);
  m.def("top(Tensor h, Tensor W, int k, Tensor? targets, int ignore_index, float[] transform) -> Tensor[]", &top);
}
