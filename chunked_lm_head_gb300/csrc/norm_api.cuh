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

// Threads of a row's group for VPT vectors of 8 elements to a thread.
int norm_group(int64_t H, int vpt) { return static_cast<int>(round_up(ceil_div(H / 8, vpt), 32)); }
// Groups of a CTA of about `threads`.
int norm_groups(int T, int threads) { return std::max(1, std::min(kNormGroups, threads / T)); }

template <bool kQ, int VPT>
cudaError_t launch_norm_v(NormParams p, bool res, bool res_f32, int threads, cudaStream_t st) {
  p.T = norm_group(p.H, VPT);
  const int groups = norm_groups(p.T, threads);
  const unsigned grid = static_cast<unsigned>(ceil_div(p.N, groups));
  if (!res)
    rms_norm_kernel<NoResidual, kQ, VPT><<<grid, groups * p.T, 0, st>>>(p);
  else if (res_f32)
    rms_norm_kernel<float, kQ, VPT><<<grid, groups * p.T, 0, st>>>(p);
  else
    rms_norm_kernel<uint16_t, kQ, VPT><<<grid, groups * p.T, 0, st>>>(p);
  return cudaGetLastError();
}

// Two vectors to a thread in CTAs of about 512 threads (131,072 x 2,560 without
// a residual: 257 us, against 387 with one vector and 362 with four; CTAs of
// 256 threads 480); rows of a warp or less one vector in CTAs of 256 (262,144 x
// 256: 102 against 104 us); past 8,192 elements four, so that a row fits a CTA.
template <bool kQ>
cudaError_t launch_norm(const NormParams& p, bool res, bool res_f32, cudaStream_t st) {
  if (p.H <= 256) return launch_norm_v<kQ, 1>(p, res, res_f32, 256, st);
  if (p.H <= 8192) return launch_norm_v<kQ, 2>(p, res, res_f32, 512, st);
  return launch_norm_v<kQ, 4>(p, res, res_f32, 512, st);
}

// How the backward runs rows of H: vectors per thread, the group and the CTA.
struct NormBwdShape {
  int vpt, T, groups, ctas;
};
// One CTA of 512 threads to an SM, two vectors to a thread (16,384 x 4,096 bf16
// with the stream's gradient: 93 us, against 116 with one vector and 99 with
// four; two CTAs to an SM 96, their dweight partials twice as many).  Rows of
// a warp or less: one vector, three CTAs to an SM (262,144 x 256: 97 us
// against 166 with one CTA).
NormBwdShape norm_bwd_shape(int64_t N, int64_t H) {
  NormBwdShape b;
  b.vpt = H <= 256 ? 1 : H <= 8192 ? 2 : 4;
  b.T = norm_group(H, b.vpt);
  b.groups = norm_groups(b.T, 512);
  const int64_t most = static_cast<int64_t>(H <= 256 ? 3 : 1) * device_sms();
  b.ctas = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(ceil_div(N, b.groups), most)));
  return b;
}

template <class S>
cudaError_t launch_norm_bwd(const NormBwdParams& p, const NormBwdShape& b, cudaStream_t st) {
  // the groups' dweight to be joined: at most 7 x 2,048 floats
  const size_t smem = p.part ? static_cast<size_t>(b.groups - 1) * p.H * 4 : 0;
  auto go = [&](auto kern) -> cudaError_t {
    kern<<<b.ctas, b.groups * b.T, smem, st>>>(p);
    return cudaGetLastError();
  };
  if (b.vpt == 1) return go(rms_norm_bwd_kernel<S, 1, 512, true>);
  if (b.vpt == 2) return go(rms_norm_bwd_kernel<S, 2, 512, true>);
  if (b.T <= 512) return go(rms_norm_bwd_kernel<S, 4, 512, false>);
  return go(rms_norm_bwd_kernel<S, 4, 1024, false>);
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
  return align256(static_cast<size_t>(norm_bwd_shape(N, H).ctas) * H * 4);
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
  const NormBwdShape b = norm_bwd_shape(N, H);
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
    p.T = b.T;
    FLCE_CUDA_TRY(s_type == FLCE_F32 ? launch_norm_bwd<float>(p, b, st) : launch_norm_bwd<uint16_t>(p, b, st));
  }
  if (dweight) {
    ProfScope ps(K_NORM_BWD, st);
    const unsigned grid = static_cast<unsigned>(ceil_div(H, 32));
    if (weight_type == FLCE_F32)
      norm_dweight_kernel<<<grid, 1024, 0, st>>>(p.part, b.ctas, p.H, static_cast<float*>(dweight));
    else
      norm_dweight_kernel<<<grid, 1024, 0, st>>>(p.part, b.ctas, p.H, static_cast<uint16_t*>(dweight));
    FLCE_CUDA_TRY(cudaGetLastError());
  }
  return FLCE_OK;
}

}  // extern "C"
