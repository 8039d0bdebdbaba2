// libflce host side: the layer norm's entry points (kernels in layer_norm.cuh).
#pragma once

#include "layer_norm.cuh"
#include "norm_api.cuh"

namespace {

template <class R, int VPT, int MAXT, int CTAS>
cudaError_t launch_layer_groups(LayerParams p, cudaStream_t st) {
  p.T = norm_group(p.H, VPT);
  const int groups = norm_groups(p.T, MAXT);
  layer_norm_kernel<R, VPT, MAXT, CTAS><<<static_cast<unsigned>(ceil_div(p.N, groups)), groups * p.T, 0, st>>>(p);
  return cudaGetLastError();
}
template <bool kRes, int VPL, int CTAS>
cudaError_t launch_layer_warps(const LayerParams& p, cudaStream_t st) {
  layer_norm_warp_kernel<kRes, VPL, CTAS>
      <<<static_cast<unsigned>(ceil_div(p.N, NORM_WARP_ROWS)), 32 * NORM_WARP_ROWS, 0, st>>>(p);
  return cudaGetLastError();
}

// The shapes of launch_norm_as: a warp to a row where the row fits its
// registers, else groups of two vectors to a thread, past 8,192 elements four.
// Warps and groups (us): 65,536 x 256 23 / 29, x 1,024 53 / 70, x 2,560 113 / 164,
// 32,768 x 4,096 107 / 131; with a bf16 residual x 256 29 / 33, x 512 47 / 47, x
// 1,024 87 / 86.
// Three CTAs of 512 threads to an SM with a bf16 stream (16,384 x 4,096 with a
// residual 88 us, 16,384 x 6,144 126: two CTAs 105 and 135, four 90 and 131), two
// with fp32 (125 us; three 127, four 135).
template <class R>
cudaError_t launch_layer_as(const LayerParams& p, cudaStream_t st) {
  constexpr bool kRes = !std::is_same<R, NoResidual>::value;
  if constexpr (!std::is_same<R, float>::value) {
    if (p.H <= 256) return launch_layer_warps<kRes, 1, 6>(p, st);
    if (p.H <= 512) return launch_layer_warps<kRes, 2, 6>(p, st);
    if (p.H <= 1024) return launch_layer_warps<kRes, 4, 4>(p, st);
  }
  if constexpr (!kRes) {
    if (p.H <= 2048) return launch_layer_warps<false, 8, 3>(p, st);
    if (p.H <= 2560) return launch_layer_warps<false, 10, 3>(p, st);
    if (p.H <= 4096) return launch_layer_warps<false, 16, 2>(p, st);
  }
  if (p.H <= 8192) return launch_layer_groups<R, 2, 512, std::is_same<R, float>::value ? 2 : 3>(p, st);
  if (p.H <= 16384) return launch_layer_groups<R, 4, 512, 2>(p, st);
  return launch_layer_groups<R, 4, 1024, 1>(p, st);
}

// How the backward runs rows of H.  A row's latency (its loads, a reduction, its
// stores) sets the pace, so as many rows as fit are worked on at once, the next
// two's loads in flight.
//   bf16 stream, H <= 8,192: two vectors to a thread (a thread's dweight and dbias
//   take 32 registers), one CTA of up to 640 threads, three rows deep.  us with and
//   without the dbias (none: no residual):
//                          640 x 3   640 x 2   896 x 2   one vector, 1,024   two CTAs of 320
//     16,384 x 4,096       93 / 90   94 / 94   195 / 90      98 / 94             99 / 94
//     131,072 x 2,560 none 340 / 315 341 / 320 655 / 342     401 / 373           369 / 336
//     16,384 x 6,144       139       148       295           156                 152
//   fp32 stream: one vector, 1,024 threads, straight from global memory, whose
//   second read hits L1 (16,384 x 4,096: 197 us; two vectors 238).
//   Past 8,192 elements one row to a CTA (4,096 x 12,288: 111 us).
// Floors of these: 79, 297 (131,072 rows), 119, 158 (fp32) and 59 us.
NormBwdShape layer_bwd_shape(int64_t N, int64_t H, bool f32) {
  NormBwdShape b;
  b.vpt = f32 ? (H <= 8192 ? 1 : 4) : (H <= 8192 ? 2 : 4);
  b.T = norm_group(H, b.vpt);
  b.groups = norm_groups(b.T, b.vpt == 1 ? 1024 : b.vpt == 2 ? 640 : 512);
  b.ctas = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(ceil_div(N, b.groups), device_sms())));
  return b;
}

template <class S, bool kBias, int VPT, int DEPTH, int MAXT, int CTAS>
cudaError_t launch_layer_bwd_as(const LayerBwdParams& p, const NormBwdShape& b, cudaStream_t st) {
  const int threads = b.groups * b.T;
  const size_t stage = static_cast<size_t>(threads) * VPT * 8 * (2 + (p.up ? 2 : 1) * sizeof(S));
  const size_t smem =
      std::max(DEPTH * stage, p.part_w || p.part_b ? static_cast<size_t>(b.groups - 1) * p.H * 4 : 0);
  auto kern = layer_norm_bwd_kernel<S, kBias, VPT, DEPTH, MAXT, CTAS>;
  if (smem > 32768) {  // (the kernel has 8 KB of its own beside it)
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 204800);
    if (e != cudaSuccess) return e;
  }
  kern<<<b.ctas, threads, smem, st>>>(p);
  return cudaGetLastError();
}

template <class S, bool kBias>
cudaError_t launch_layer_bwd(const LayerBwdParams& p, const NormBwdShape& b, cudaStream_t st) {
  if constexpr (std::is_same<S, float>::value) {
    if (b.vpt == 1) return launch_layer_bwd_as<S, kBias, 1, 0, 1024, 1>(p, b, st);
    return launch_layer_bwd_as<S, kBias, 4, 0, 1024, 1>(p, b, st);
  } else {
    if (b.vpt == 2)
      return b.groups * b.T <= 512 ? launch_layer_bwd_as<S, kBias, 2, 3, 512, 1>(p, b, st)
                                   : launch_layer_bwd_as<S, kBias, 2, 3, 640, 1>(p, b, st);
    return b.T <= 512 ? launch_layer_bwd_as<S, kBias, 4, 1, 512, 1>(p, b, st)
                      : launch_layer_bwd_as<S, kBias, 4, 0, 1024, 1>(p, b, st);
  }
}

}  // namespace

extern "C" {

flce_status flce_layer_norm(const flce_bf16* x, int64_t ldx, const void* residual, int64_t ldr,
                            int32_t residual_type, const void* weight, const void* bias, int32_t weight_type,
                            float weight_offset, float eps, int64_t N, int64_t H, flce_bf16* out_y,
                            void* out_residual, float* out_mean, float* out_rstd, void* stream) {
  if (!norm_sizes_ok(N, H) || !std::isfinite(weight_offset) || !(std::isfinite(eps) && eps >= 0.f))
    return FLCE_ERR_INVALID_ARG;
  if (!norm_dtype_ok(weight_type) || (residual && !norm_dtype_ok(residual_type))) return FLCE_ERR_INVALID_ARG;
  if ((residual != nullptr) != (out_residual != nullptr)) return FLCE_ERR_INVALID_ARG;
  if (N > 0 && (!x || !weight || !out_y || ldx < H || (residual && ldr < H))) return FLCE_ERR_INVALID_ARG;
  if (H % 8 != 0 || H > kNormMaxH) return FLCE_ERR_UNSUPPORTED;
  if (ldx % 8 != 0 || (residual && ldr % (residual_type == FLCE_F32 ? 4 : 8) != 0)) return FLCE_ERR_UNSUPPORTED;
  if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) || !aligned(bias, 16) || !aligned(out_y, 16) ||
      !aligned(out_residual, 16) || !aligned(out_mean, 4) || !aligned(out_rstd, 4))
    return FLCE_ERR_UNSUPPORTED;
  if (N == 0) return FLCE_OK;
  LayerParams p{};
  p.x = x;
  p.r = residual;
  p.weight = weight;
  p.bias = bias;
  p.ldx = ldx;
  p.ldr = ldr;
  p.N = static_cast<int>(N);
  p.H = static_cast<int>(H);
  p.w_f32 = weight_type == FLCE_F32;
  p.offset = weight_offset;
  p.eps = eps;
  p.y = out_y;
  p.s = out_residual;
  p.mean = out_mean;
  p.rstd = out_rstd;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  ProfScope ps(K_LAYER_NORM, st);
  FLCE_CUDA_TRY(residual == nullptr           ? launch_layer_as<NoResidual>(p, st)
                : residual_type == FLCE_F32 ? launch_layer_as<float>(p, st)
                                              : launch_layer_as<uint16_t>(p, st));
  return FLCE_OK;
}

size_t flce_layer_norm_backward_workspace_bytes(int64_t N, int64_t H) {
  if (!norm_sizes_ok(N, H)) return 0;
  // of either stream type
  const int ctas = std::max(layer_bwd_shape(N, H, false).ctas, layer_bwd_shape(N, H, true).ctas);
  return 2 * align256(static_cast<size_t>(ctas) * H * 4);
}

flce_status flce_layer_norm_backward(const flce_bf16* dy, const void* s, int64_t lds, int32_t s_type,
                                     const void* ds, const void* weight, int32_t weight_type, float weight_offset,
                                     const float* mean, const float* rstd, int64_t N, int64_t H, flce_bf16* dx,
                                     float* dr, void* dweight, void* dbias, void* workspace, size_t workspace_bytes,
                                     void* stream) {
  if (!norm_sizes_ok(N, H) || !std::isfinite(weight_offset)) return FLCE_ERR_INVALID_ARG;
  if (!norm_dtype_ok(weight_type) || !norm_dtype_ok(s_type)) return FLCE_ERR_INVALID_ARG;
  if (N > 0 && !dx && !dr && !dweight && !dbias) return FLCE_ERR_INVALID_ARG;
  if (N > 0 && (!dy || !s || !weight || !mean || !rstd || lds < H)) return FLCE_ERR_INVALID_ARG;
  if (H % 8 != 0 || H > kNormMaxH || lds % (s_type == FLCE_F32 ? 4 : 8) != 0) return FLCE_ERR_UNSUPPORTED;
  if (!aligned(dy, 16) || !aligned(s, 16) || !aligned(ds, 16) || !aligned(weight, 16) || !aligned(mean, 4) ||
      !aligned(rstd, 4) || !aligned(dx, 16) || !aligned(dr, 16) || !aligned(dweight, 16) || !aligned(dbias, 16))
    return FLCE_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const size_t param = static_cast<size_t>(H) * (weight_type == FLCE_F32 ? 4 : 2);
  if (N == 0) {
    if (dweight) FLCE_CUDA_TRY(cudaMemsetAsync(dweight, 0, param, st));
    if (dbias) FLCE_CUDA_TRY(cudaMemsetAsync(dbias, 0, param, st));
    return FLCE_OK;
  }
  const NormBwdShape b = layer_bwd_shape(N, H, s_type == FLCE_F32);
  const size_t part = flce_layer_norm_backward_workspace_bytes(N, H) / 2;
  Workspace ws;
  if (dweight || dbias) {
    const flce_status g = get_workspace(ws, workspace, workspace_bytes, 2 * part, st);
    if (g != FLCE_OK) return g;
  }
  LayerBwdParams p{};
  p.dy = dy;
  p.s = s;
  p.up = ds;
  p.weight = weight;
  p.mean = mean;
  p.rstd = rstd;
  p.lds = lds;
  p.N = static_cast<int>(N);
  p.H = static_cast<int>(H);
  p.w_f32 = weight_type == FLCE_F32;
  p.T = b.T;
  p.offset = weight_offset;
  p.dx = dx;
  p.dr = dr;
  p.part_w = dweight ? static_cast<float*>(ws.ptr) : nullptr;
  p.part_b = dbias ? reinterpret_cast<float*>(static_cast<uint8_t*>(ws.ptr) + part) : nullptr;
  {
    ProfScope ps(K_LAYER_NORM_BWD, st);
    if (s_type == FLCE_F32)
      FLCE_CUDA_TRY((dbias ? launch_layer_bwd<float, true>(p, b, st) : launch_layer_bwd<float, false>(p, b, st)));
    else
      FLCE_CUDA_TRY((dbias ? launch_layer_bwd<uint16_t, true>(p, b, st) : launch_layer_bwd<uint16_t, false>(p, b, st)));
  }
  if (dweight || dbias) {
    ProfScope ps(K_LAYER_NORM_BWD, st);
    const dim3 grid(static_cast<unsigned>(ceil_div(H, 32)), dbias ? 2 : 1);
    if (weight_type == FLCE_F32)
      layer_dparam_kernel<<<grid, 1024, 0, st>>>(p.part_w, p.part_b, b.ctas, p.H, static_cast<float*>(dweight),
                                                 static_cast<float*>(dbias));
    else
      layer_dparam_kernel<<<grid, 1024, 0, st>>>(p.part_w, p.part_b, b.ctas, p.H, static_cast<uint16_t*>(dweight),
                                                 static_cast<uint16_t*>(dbias));
    FLCE_CUDA_TRY(cudaGetLastError());
  }
  return FLCE_OK;
}

}  // extern "C"
