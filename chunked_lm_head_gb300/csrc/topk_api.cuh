// libflce host side: the entry points of the distillation from a teacher's
// top logits (row kernels in topk.cuh; the forward, the one-call step and the
// tiled backward are those of the cross-entropy, in flce.cu, with the listed
// columns taken apart).
#pragma once

namespace {

bool topk_sizes_ok(int64_t N, int64_t H, int64_t V) { return sizes_ok(N, H, V) && N <= kMaxRows; }

bool topk_teacher_ok(const flce_top_logits* t) {
  if (t == nullptr || t->k < 1) return false;
  if (t->ids_type != FLCE_I32 && t->ids_type != FLCE_I64) return false;
  if (t->logits_type != FLCE_F32 && t->logits_type != FLCE_BF16 && t->logits_type != FLCE_F16) return false;
  if (t->tail != 0 && t->tail != 1) return false;
  return !(t->tail && t->lse == nullptr);  // the mass outside the list needs the teacher's whole sum
}

// The call's row arrays and block sums.  The first five are the state that
// the backward reads, laid out alike in a caller's state buffer.
struct TopkLayout {
  size_t ids = 0, val = 0, mark = 0, lse_rest = 0, coef = 0, state = 0;
  size_t mass = 0, stat = 0, bsum = 0, bcnt = 0, gemv = 0, total = 0;
};
TopkLayout topk_layout(int64_t N, int64_t K) {
  TopkLayout L;
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += align256(bytes);
    return at;
  };
  const size_t n = static_cast<size_t>(std::max<int64_t>(N, 1)), nk = n * static_cast<size_t>(K);
  L.ids = take(nk * 4);
  L.val = take(nk * 4);
  L.mark = take(n * 8);
  L.lse_rest = take(n * 4);
  L.coef = take(n * 4);
  L.state = o;
  L.mass = take(nk * 4);
  L.stat = take(n * 8);
  // one-call: ceil(N / R) segments of R / TOPK_ROWS block sums, R a multiple of
  // 128 and at most N rounded up to one
  const size_t blocks = (2 * n + 256) / TOPK_ROWS + 1;
  L.bsum = take(blocks * 8);
  L.bcnt = take(blocks * 8);
  L.gemv = take(n <= TOPK_GEMV_ROWS ? static_cast<size_t>(TOPK_GEMV_CTAS * device_sms()) * n * 8 : 0);
  L.total = o;
  return L;
}

TopkRows topk_rows_at(const TopkLayout& L, uint8_t* state, uint8_t* scratch) {
  TopkRows r{};
  r.ids = reinterpret_cast<int*>(state + L.ids);
  r.val = reinterpret_cast<float*>(state + L.val);
  r.mark = reinterpret_cast<long long*>(state + L.mark);
  r.lse_rest = reinterpret_cast<float*>(state + L.lse_rest);
  r.coef = reinterpret_cast<float*>(state + L.coef);
  r.mass = reinterpret_cast<float*>(scratch + L.mass);
  r.stat = reinterpret_cast<float2*>(scratch + L.stat);
  return r;
}

// The checks of a call that takes a teacher.
flce_status topk_check(const flce_top_logits* t, const int64_t* targets, const float* weights, int64_t N, int64_t H,
                       int64_t V) {
  if (!topk_sizes_ok(N, H, V) || !topk_teacher_ok(t)) return FLCE_ERR_INVALID_ARG;
  if (N > 0 && (!t->ids || !t->logits || t->ld_ids < t->k || t->ld_logits < t->k)) return FLCE_ERR_INVALID_ARG;
  if (t->k > TOPK_MAX_K) return FLCE_ERR_UNSUPPORTED;
  if (!aligned(t->ids, t->ids_type == FLCE_I64 ? 8 : 4) || !aligned(t->logits, t->logits_type == FLCE_F32 ? 4 : 2) ||
      !aligned(t->lse, 4) || !aligned(targets, 8) || !aligned(weights, 4))
    return FLCE_ERR_UNSUPPORTED;
  return FLCE_OK;
}

flce_status topk_lists(const flce_top_logits* t, const int64_t* targets, int64_t ignore_index, int64_t N, int64_t V,
                       const TopkRows& rows, cudaStream_t st) {
  if (N == 0) return FLCE_OK;
  const TopkTeacher d{t->ids,     t->logits,   t->lse,         t->ld_ids, t->ld_logits,
                      t->ids_type, t->logits_type, t->k, t->tail};
  ProfScope ps(K_TOPK, st);
  FLCE_CUDA_TRY(launch_dependent(topk_list_kernel, dim3(static_cast<unsigned>(ceil_div(N, TOPK_WARPS))),
                                 32 * TOPK_WARPS, static_cast<size_t>(TOPK_WARPS) * 2 * ((t->k + 3) & ~3) * 4, st, d,
                                 targets, ignore_index, static_cast<int>(N), static_cast<int>(V), rows));
  return FLCE_OK;
}

// dW in the caller's type.  bf16 comes straight from the dW GEMM where one row
// block holds every row; else it is summed over the blocks in fp32 scratch and
// rounded once at the end.
struct TopkGrad {
  bool scratch = false;
  size_t bytes = 0;  // of the scratch
};
TopkGrad topk_grad(int32_t dW_type, int64_t N, int64_t H, int64_t V, long long block_rows) {
  TopkGrad g;
  g.scratch = dW_type == FLCE_BF16 && N > block_rows;
  if (g.scratch) g.bytes = align256(static_cast<size_t>(V) * H * 4);
  return g;
}
// Rows of the tiled backward's block in its unpipelined plan, the one that a call
// of one block keeps.
long long topk_bwd_rows(int64_t N, int64_t H, int64_t V, int64_t chunk_rows) {
  const int cg = cta_group();
  return plan_backward(N, H, V, chunk_rows, device_workers(cg), BM * cg).R;
}
long long topk_one_call_rows(int64_t N, int64_t H, int64_t V, int64_t chunk_rows) {
  const long long R = N > 0 ? fused_rows(N, chunk_rows) : 0;
  return R > 0 ? R : topk_bwd_rows(N, H, V, chunk_rows);
}
bool topk_dw_ok(const void* dW, int32_t dW_type) { return dW == nullptr || dW_type == FLCE_BF16 || dW_type == FLCE_F32; }

flce_status topk_round_dw(const float* x, int64_t n, void* dW, const int* out_count, float grad_scale,
                          cudaStream_t st) {
  ProfScope ps(K_DH_REDUCE, st);
  round_bf16_kernel<<<8 * device_sms(), SMALL_THREADS, 0, st>>>(x, n, static_cast<uint16_t*>(dW), out_count, grad_scale);
  FLCE_CUDA_TRY(cudaGetLastError());
  return FLCE_OK;
}

}  // namespace

extern "C" {

flce_status flce_scale_grads_bf16(flce_bf16* dH, int64_t n_dH, flce_bf16* dW, int64_t n_dW, const float* scale,
                                  void* stream) {
  if (n_dH < 0 || n_dW < 0 || scale == nullptr || (n_dH > 0 && dH == nullptr) || (n_dW > 0 && dW == nullptr))
    return FLCE_ERR_INVALID_ARG;
  if (!aligned(dH, 16) || !aligned(dW, 16) || !aligned(scale, 4)) return FLCE_ERR_UNSUPPORTED;
  if (n_dH + n_dW == 0) return FLCE_OK;
  const long long blocks = std::min<long long>(8LL * device_sms(), ceil_div(n_dH + n_dW, 8LL * SMALL_THREADS));
  scale_bf16_pair_kernel<<<static_cast<unsigned>(blocks), SMALL_THREADS, 0, static_cast<cudaStream_t>(stream)>>>(
      reinterpret_cast<__nv_bfloat16*>(dH), n_dH, reinterpret_cast<__nv_bfloat16*>(dW), n_dW, scale);
  FLCE_CUDA_TRY(cudaGetLastError());
  return FLCE_OK;
}

size_t flce_topk_kd_state_bytes(int64_t N, int64_t k) {
  if (N < 0 || N > kMaxRows || k < 1 || k > TOPK_MAX_K) return 0;
  return topk_layout(N, k).state;
}

size_t flce_topk_kd_workspace_bytes(int64_t N, int64_t H, int64_t V, int64_t k, int64_t chunk_rows) {
  if (!topk_sizes_ok(N, H, V) || k < 1 || k > TOPK_MAX_K) return 0;
  return align256(flce_workspace_bytes(N, H, V, chunk_rows)) + topk_layout(N, k).total;
}

size_t flce_topk_kd_backward_workspace_bytes(int64_t N, int64_t H, int64_t V, int64_t chunk_rows, int32_t dW_type) {
  if (!topk_sizes_ok(N, H, V)) return 0;
  return align256(flce_workspace_bytes(N, H, V, chunk_rows)) +
         topk_grad(dW_type, N, H, V, topk_bwd_rows(N, H, V, chunk_rows)).bytes;
}

// Workspace of the one-call step inside: with a bf16 dW, or none, its fused
// form completes the dlogits' scale in fp32 (split_scale).
static size_t topk_one_call_inner(int64_t N, int64_t H, int64_t V, int64_t chunk_rows, bool split) {
  const int cg = cta_group();
  const int workers = device_workers(cg);
  const FusedPlan fp = plan_fused(N, H, V, chunk_rows, workers, BM * cg,
                                  split ? OneCall::kListedSplit : OneCall::kListed);
  return align256(fp.fused && N > 0 ? fused_layout(N, H, fp).total
                                    : fallback_workspace(N, H, V, chunk_rows, workers, BM * cg));
}

size_t flce_topk_kd_forward_backward_workspace_bytes(int64_t N, int64_t H, int64_t V, int64_t k, int64_t chunk_rows,
                                                     int32_t dW_type) {
  if (!topk_sizes_ok(N, H, V) || k < 1 || k > TOPK_MAX_K) return 0;
  // (a call without dW needs what one with a bf16 dW does)
  return std::max(topk_one_call_inner(N, H, V, chunk_rows, true),
                  dW_type == FLCE_F32 ? topk_one_call_inner(N, H, V, chunk_rows, false) : 0) +
         topk_layout(N, k).total + topk_grad(dW_type, N, H, V, topk_one_call_rows(N, H, V, chunk_rows)).bytes;
}

flce_status flce_topk_kd_forward(const flce_bf16* h, const flce_bf16* W, const flce_top_logits* teacher,
                                 const int64_t* targets, const float* weights, int64_t N, int64_t H, int64_t V,
                                 int64_t chunk_rows, int64_t ignore_index, const flce_logit_transform* transform,
                                 uint32_t flags, float* out_kl, float* out_lse, float* out_loss,
                                 int64_t* out_n_valid, void* state, void* workspace, size_t workspace_bytes,
                                 void* stream) {
  if ((flags & ~static_cast<uint32_t>(FLCE_FORWARD_SKIP_IGNORED)) != 0) return FLCE_ERR_INVALID_ARG;
  if (!out_kl && !out_lse && !out_loss && !out_n_valid && !state) return FLCE_ERR_INVALID_ARG;
  flce_status s = topk_check(teacher, targets, weights, N, H, V);
  if (s != FLCE_OK) return s;
  if (N > 0 && (!h || !W)) return FLCE_ERR_INVALID_ARG;
  if (!aligned(out_kl, 4) || !aligned(out_lse, 4) || !aligned(state, 256)) return FLCE_ERR_UNSUPPORTED;
  const TopkLayout L = topk_layout(N, teacher->k);
  const size_t inner = align256(flce_workspace_bytes(N, H, V, chunk_rows));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  GemmParams tfp{};
  if (!transform_params(transform, tfp)) return FLCE_ERR_INVALID_ARG;
  if (H % 8 != 0 || !aligned(h, 16) || !aligned(W, 16) || !aligned(out_loss, 4) || !aligned(out_n_valid, 8))
    return FLCE_ERR_UNSUPPORTED;
  Workspace ws;
  s = get_workspace(ws, workspace, workspace_bytes, inner + L.total, st);
  if (s != FLCE_OK) return s;
  uint8_t* wb = static_cast<uint8_t*>(ws.ptr);
  TopkCall c;
  c.rows = topk_rows_at(L, state ? static_cast<uint8_t*>(state) : wb + inner, wb + inner);
  c.K = teacher->k;
  c.tail = teacher->tail;
  c.weights = weights;
  c.out_kl = out_kl;
  c.out_lse = out_lse;
  c.bsum = reinterpret_cast<double*>(wb + inner + L.bsum);
  c.bcnt = reinterpret_cast<long long*>(wb + inner + L.bcnt);
  c.gemv = reinterpret_cast<float2*>(wb + inner + L.gemv);
  s = topk_lists(teacher, targets, ignore_index, N, V, c.rows, st);
  if (s != FLCE_OK) return s;
  const bool skip = (flags & FLCE_FORWARD_SKIP_IGNORED) != 0 && compact_on() && N >= skip_min_rows();
  return forward_impl(h, W, reinterpret_cast<const int64_t*>(c.rows.mark), nullptr, N, H, V, kMarkIgnored, transform,
                      nullptr, nullptr, out_loss, out_n_valid, wb, inner, stream, kFwdPartialsCap, skip, &c);
}

flce_status flce_topk_kd_backward(const flce_bf16* h, const flce_bf16* W, const void* state, float grad_scale,
                                  const flce_device_scale* device_scale, flce_bf16* dH, void* dW, int32_t dW_type,
                                  int64_t N, int64_t H, int64_t V, int64_t k, int64_t chunk_rows,
                                  const flce_logit_transform* transform, void* workspace, size_t workspace_bytes,
                                  void* stream) {
  if (!topk_sizes_ok(N, H, V) || k < 1 || (N > 0 && !state) || !topk_dw_ok(dW, dW_type)) return FLCE_ERR_INVALID_ARG;
  GemmParams tfp{};
  if (!transform_params(transform, tfp) || (!dH && !dW) || (N > 0 && (!h || !W))) return FLCE_ERR_INVALID_ARG;
  if (k > TOPK_MAX_K || H % 8 != 0 || !aligned(state, 256) || !aligned(dW, 16) || !aligned(dH, 16) || !aligned(h, 16) ||
      !aligned(W, 16))
    return FLCE_ERR_UNSUPPORTED;
  const TopkLayout L = topk_layout(N, k);
  TopkCall c;
  // read only by the tiled backward
  uint8_t* sb = static_cast<uint8_t*>(const_cast<void*>(state));
  c.rows = topk_rows_at(L, sb, sb);
  c.K = static_cast<int>(k);
  const long long* count = device_scale ? reinterpret_cast<const long long*>(device_scale->count) : nullptr;
  const float* scale = device_scale ? device_scale->scale : nullptr;
  const bool bf16 = dW != nullptr && dW_type == FLCE_BF16;
  const TopkGrad tg = topk_grad(dW ? dW_type : FLCE_F32, N, H, V, bf16 ? topk_bwd_rows(N, H, V, chunk_rows) : 0);
  if (bf16 && !tg.scratch) c.dW16 = static_cast<flce_bf16*>(dW);
  const size_t inner = align256(flce_workspace_bytes(N, H, V, chunk_rows));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  Workspace ws;
  flce_status s = get_workspace(ws, workspace, workspace_bytes, inner + tg.bytes, st);
  if (s != FLCE_OK) return s;
  float* sum = tg.scratch ? reinterpret_cast<float*>(static_cast<uint8_t*>(ws.ptr) + inner)
                          : bf16 ? nullptr : static_cast<float*>(dW);
  s = backward_impl(h, W, reinterpret_cast<const int64_t*>(c.rows.mark), c.rows.coef, c.rows.lse_rest, grad_scale, dH,
                    sum, N, H, V, chunk_rows, kMarkIgnored, transform, ws.ptr, inner, stream, count, scale, &c);
  if (s != FLCE_OK || !tg.scratch) return s;
  return topk_round_dw(sum, V * H, dW, nullptr, 1.f, st);
}

flce_status flce_topk_kd_forward_backward(const flce_bf16* h, const flce_bf16* W, const flce_top_logits* teacher,
                                          const int64_t* targets, const float* weights, int64_t N, int64_t H,
                                          int64_t V, int64_t chunk_rows, int64_t ignore_index,
                                          const flce_logit_transform* transform, float grad_scale, float* out_kl,
                                          float* out_lse, float* out_loss, int64_t* out_n_valid, flce_bf16* dH,
                                          void* dW, int32_t dW_type, void* workspace, size_t workspace_bytes,
                                          void* stream) {
  flce_status s = topk_check(teacher, targets, weights, N, H, V);
  if (s != FLCE_OK) return s;
  GemmParams tfp{};
  if (!transform_params(transform, tfp) || !std::isfinite(grad_scale)) return FLCE_ERR_INVALID_ARG;
  if ((!dH && !dW) || (N > 0 && (!h || !W)) || !topk_dw_ok(dW, dW_type)) return FLCE_ERR_INVALID_ARG;
  if (H % 8 != 0 || !aligned(h, 16) || !aligned(W, 16) || !aligned(dH, 16) || !aligned(dW, 16) ||
      !aligned(out_kl, 4) || !aligned(out_lse, 4) || !aligned(out_loss, 4) || !aligned(out_n_valid, 8))
    return FLCE_ERR_UNSUPPORTED;
  const TopkLayout L = topk_layout(N, teacher->k);
  const bool bf16 = dW != nullptr && dW_type == FLCE_BF16;
  const bool split = (bf16 || dW == nullptr) && N > 0 && fused_rows(N, chunk_rows) > 0;
  const size_t inner = topk_one_call_inner(N, H, V, chunk_rows, split);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  Workspace ws;
  const TopkGrad tg = topk_grad(dW ? dW_type : FLCE_F32, N, H, V, topk_one_call_rows(N, H, V, chunk_rows));
  s = get_workspace(ws, workspace, workspace_bytes, inner + L.total + tg.bytes, st);
  if (s != FLCE_OK) return s;
  uint8_t* wb = static_cast<uint8_t*>(ws.ptr);
  float* sum = tg.scratch ? reinterpret_cast<float*>(wb + inner + L.total) : bf16 ? nullptr : static_cast<float*>(dW);
  TopkCall c;
  if (bf16 && !tg.scratch) c.dW16 = static_cast<flce_bf16*>(dW);
  c.split_scale = split;
  c.rows = topk_rows_at(L, wb + inner, wb + inner);
  c.K = teacher->k;
  c.tail = teacher->tail;
  c.weights = weights;
  c.out_kl = out_kl;
  c.out_lse = out_lse;
  c.bsum = reinterpret_cast<double*>(wb + inner + L.bsum);
  c.bcnt = reinterpret_cast<long long*>(wb + inner + L.bcnt);
  c.gemv = reinterpret_cast<float2*>(wb + inner + L.gemv);
  s = topk_lists(teacher, targets, ignore_index, N, V, c.rows, st);
  if (s != FLCE_OK) return s;
  s = forward_backward_impl(h, W, reinterpret_cast<const int64_t*>(c.rows.mark), nullptr, N, H, V, chunk_rows,
                            kMarkIgnored, transform, grad_scale, nullptr, nullptr, out_loss, out_n_valid, dH, sum, wb,
                            inner, stream, nullptr, &c);
  if (s != FLCE_OK || !tg.scratch) return s;
  // the count that the step left in its workspace
  const int* count = nullptr;
  if (split) {
    const int cg = cta_group();
    const FusedPlan fp = plan_fused(N, H, V, chunk_rows, device_workers(cg), BM * cg, OneCall::kListedSplit);
    count = reinterpret_cast<const int*>(wb + fused_layout(N, H, fp).count);
  }
  return topk_round_dw(sum, V * H, dW, count, grad_scale, st);
}

}  // extern "C"
