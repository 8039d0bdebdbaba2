// libflce host side: the norm's entry points (kernels in norm.cuh).
#pragma once

#include "launch.cuh"
#include "norm.cuh"

namespace {

using namespace flce;

// Longest row: 4 vectors of 8 elements on each of 1,024 threads.
constexpr int64_t kNormMaxH = 32768;

bool norm_sizes_ok(int64_t N, int64_t H) { return N >= 0 && H > 0 && N < INT_MAX && H < INT_MAX; }
bool norm_dtype_ok(int32_t t) { return t == FLCE_BF16 || t == FLCE_F32; }

// Calls go(threads per row, vectors per thread) with the narrowest row that
// holds H: a warp up to 1,024 elements (no CTA barrier), then a CTA whose
// threads hold one or two vectors, so that several CTAs per SM keep loads in
// flight while others reduce.
template <class Go>
cudaError_t norm_shape(int64_t H, Go go) {
  using std::integral_constant;
  const int64_t nv = H / 8;
  if (nv <= 32) return go(integral_constant<int, 32>{}, integral_constant<int, 1>{});
  if (nv <= 128) return go(integral_constant<int, 32>{}, integral_constant<int, 4>{});
  if (nv <= 256) return go(integral_constant<int, 256>{}, integral_constant<int, 1>{});
  if (nv <= 512) return go(integral_constant<int, 256>{}, integral_constant<int, 2>{});
  if (nv <= 1024) return go(integral_constant<int, 512>{}, integral_constant<int, 2>{});
  return go(integral_constant<int, 1024>{}, integral_constant<int, 4>{});
}

template <bool kQ>
cudaError_t launch_norm(const NormParams& p, bool res, bool res_f32, cudaStream_t st) {
  return norm_shape(p.H, [&](auto tpr, auto vpt) -> cudaError_t {
    constexpr int TPR = decltype(tpr)::value, VPT = decltype(vpt)::value;
    constexpr int CTA = TPR < 256 ? 256 : TPR;
    const unsigned grid = static_cast<unsigned>(ceil_div(p.N, CTA / TPR));
    if (!res)
      rms_norm_kernel<NoResidual, kQ, TPR, VPT><<<grid, CTA, 0, st>>>(p);
    else if (res_f32)
      rms_norm_kernel<float, kQ, TPR, VPT><<<grid, CTA, 0, st>>>(p);
    else
      rms_norm_kernel<uint16_t, kQ, TPR, VPT><<<grid, CTA, 0, st>>>(p);
    return cudaGetLastError();
  });
}

// Row slots of the backward: rows in flight, each with a dweight partial.
int64_t norm_bwd_ctas(int64_t N, int64_t H, int* rows_per_cta) {
  *rows_per_cta = H / 8 <= 128 ? 8 : 1;
  return std::max<int64_t>(1, std::min<int64_t>(ceil_div(N, *rows_per_cta), 4LL * device_sms()));
}

}  // namespace

extern "C" {

static flce_status norm_forward(const flce_bf16* x, int64_t ldx, const void* residual, int64_t ldr,
                                int32_t residual_type, const void* weight, int32_t weight_type,
                                float weight_offset, float eps, int64_t N, int64_t H, flce_bf16* out_y,
                                uint8_t* out_q, float* out_scale, void* out_residual, float* out_rstd,
                                void* stream) {
  const bool q = out_q != nullptr;
  if (!norm_sizes_ok(N, H) || !std::isfinite(weight_offset) || !(std::isfinite(eps) && eps >= 0.f))
    return FLCE_ERR_INVALID_ARG;
  if (!norm_dtype_ok(weight_type) || (residual && !norm_dtype_ok(residual_type))) return FLCE_ERR_INVALID_ARG;
  if ((residual != nullptr) != (out_residual != nullptr)) return FLCE_ERR_INVALID_ARG;
  if (N > 0 && (!x || !weight || ldx < H || (residual && ldr < H))) return FLCE_ERR_INVALID_ARG;
  if (H % (q ? 16 : 8) != 0 || H > kNormMaxH) return FLCE_ERR_UNSUPPORTED;
  if (ldx % 8 != 0 || (residual && ldr % (residual_type == FLCE_F32 ? 4 : 8) != 0)) return FLCE_ERR_UNSUPPORTED;
  if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) || !aligned(out_y, 16) ||
      !aligned(out_q, 16) || !aligned(out_scale, 4) || !aligned(out_residual, 16) || !aligned(out_rstd, 4))
    return FLCE_ERR_UNSUPPORTED;
  if (N == 0) return FLCE_OK;
  NormParams p{};
  p.x = x;
  p.r = residual;
  p.weight = weight;
  p.ldx = ldx;
  p.ldr = ldr;
  p.N = static_cast<int>(N);
  p.H = static_cast<int>(H);
  p.w_f32 = weight_type == FLCE_F32;
  p.offset = weight_offset;
  p.eps = eps;
  p.y = out_y;
  p.q = out_q;
  p.scale = out_scale;
  p.s = out_residual;
  p.rstd = out_rstd;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  ProfScope ps(K_NORM, st);
  const bool f32 = residual_type == FLCE_F32;
  FLCE_CUDA_TRY(q ? launch_norm<true>(p, residual != nullptr, f32, st)
                  : launch_norm<false>(p, residual != nullptr, f32, st));
  return FLCE_OK;
}

flce_status flce_rms_norm(const flce_bf16* x, int64_t ldx, const void* residual, int64_t ldr,
                          int32_t residual_type, const void* weight, int32_t weight_type,
                          float weight_offset, float eps, int64_t N, int64_t H, flce_bf16* out_y,
                          void* out_residual, float* out_rstd, void* stream) {
  if (N != 0 && !out_y) return FLCE_ERR_INVALID_ARG;
  return norm_forward(x, ldx, residual, ldr, residual_type, weight, weight_type, weight_offset, eps, N, H,
                      out_y, nullptr, nullptr, out_residual, out_rstd, stream);
}

flce_status flce_rms_norm_e4m3(const flce_bf16* x, int64_t ldx, const void* residual, int64_t ldr,
                               int32_t residual_type, const void* weight, int32_t weight_type,
                               float weight_offset, float eps, int64_t N, int64_t H, uint8_t* out_q,
                               float* out_scale, void* out_residual, float* out_rstd, void* stream) {
  if (H > 0 && H % 16 != 0) return FLCE_ERR_UNSUPPORTED;
  if (N != 0 && (!out_q || !out_scale)) return FLCE_ERR_INVALID_ARG;
  return norm_forward(x, ldx, residual, ldr, residual_type, weight, weight_type, weight_offset, eps, N, H,
                      nullptr, out_q, out_scale, out_residual, out_rstd, stream);
}

size_t flce_rms_norm_backward_workspace_bytes(int64_t N, int64_t H) {
  if (!norm_sizes_ok(N, H)) return 0;
  int rows = 1;
  const int64_t ctas = norm_bwd_ctas(N, H, &rows);
  return align256(static_cast<size_t>(ctas) * rows * H * 4);
}

flce_status flce_rms_norm_backward(const flce_bf16* dy, const void* s, int64_t lds, int32_t s_type,
                                   const void* ds, const void* weight, int32_t weight_type,
                                   float weight_offset, const float* rstd, int64_t N, int64_t H,
                                   flce_bf16* dx, float* dr, void* dweight, void* workspace,
                                   size_t workspace_bytes, void* stream) {
  if (!norm_sizes_ok(N, H) || !std::isfinite(weight_offset)) return FLCE_ERR_INVALID_ARG;
  if (!norm_dtype_ok(weight_type) || !norm_dtype_ok(s_type)) return FLCE_ERR_INVALID_ARG;
  if (!dx && !dr && !dweight) return FLCE_ERR_INVALID_ARG;
  if (N > 0 && (!dy || !s || !weight || !rstd || lds < H)) return FLCE_ERR_INVALID_ARG;
  if (H % 8 != 0 || H > kNormMaxH || lds % (s_type == FLCE_F32 ? 4 : 8) != 0) return FLCE_ERR_UNSUPPORTED;
  if (!aligned(dy, 16) || !aligned(s, 16) || !aligned(ds, 16) || !aligned(weight, 16) || !aligned(rstd, 4) ||
      !aligned(dx, 16) || !aligned(dr, 16) || !aligned(dweight, 16))
    return FLCE_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (N == 0) {
    if (dweight) FLCE_CUDA_TRY(cudaMemsetAsync(dweight, 0, H * (weight_type == FLCE_F32 ? 4 : 2), st));
    return FLCE_OK;
  }
  int rows = 1;
  const int64_t ctas = norm_bwd_ctas(N, H, &rows);
  Workspace ws;
  if (dweight) {
    const flce_status g =
        get_workspace(ws, workspace, workspace_bytes, flce_rms_norm_backward_workspace_bytes(N, H), st);
    if (g != FLCE_OK) return g;
  }
  NormBwdParams p{};
  p.dy = dy;
  p.s = s;
  p.up = ds;
  p.weight = weight;
  p.rstd = rstd;
  p.lds = lds;
  p.N = static_cast<int>(N);
  p.H = static_cast<int>(H);
  p.w_f32 = weight_type == FLCE_F32;
  p.offset = weight_offset;
  p.dx = dx;
  p.dr = dr;
  p.part = dweight ? static_cast<float*>(ws.ptr) : nullptr;
  {
    ProfScope ps(K_NORM_BWD, st);
    FLCE_CUDA_TRY(norm_shape(H, [&](auto tpr, auto vpt) -> cudaError_t {
      constexpr int TPR = decltype(tpr)::value, VPT = decltype(vpt)::value;
      constexpr int CTA = TPR < 256 ? 256 : TPR;
      if (s_type == FLCE_F32)
        rms_norm_bwd_kernel<float, TPR, VPT><<<static_cast<unsigned>(ctas), CTA, 0, st>>>(p);
      else
        rms_norm_bwd_kernel<uint16_t, TPR, VPT><<<static_cast<unsigned>(ctas), CTA, 0, st>>>(p);
      return cudaGetLastError();
    }));
  }
  if (dweight) {
    ProfScope ps(K_NORM_BWD, st);
    const unsigned grid = static_cast<unsigned>(ceil_div(H, 32));
    const int slots = static_cast<int>(ctas * rows);
    if (weight_type == FLCE_F32)
      norm_dweight_kernel<<<grid, 256, 0, st>>>(p.part, slots, p.H, static_cast<float*>(dweight));
    else
      norm_dweight_kernel<<<grid, 256, 0, st>>>(p.part, slots, p.H, static_cast<uint16_t*>(dweight));
    FLCE_CUDA_TRY(cudaGetLastError());
  }
  return FLCE_OK;
}

}  // extern "C"
