// libflce host side: the norm's entry points (kernels in norm.cuh).
#pragma once

#include "launch.cuh"
#include "norm.cuh"

namespace {

using namespace flce;

// Longest row: 4 vectors of 8 elements on each of 1,024 threads.
constexpr int64_t kNormMaxH = 32768;

bool norm_sizes_ok(int64_t N, int64_t H) { return N >= 0 && H > 0 && N <= kMaxRows && H < INT_MAX; }
bool norm_dtype_ok(int32_t t) { return t == FLCE_BF16 || t == FLCE_F32; }

// Threads of a row's group for VPT vectors of 8 elements to a thread.
int norm_group(int64_t H, int vpt) { return static_cast<int>(round_up(ceil_div(H / 8, vpt), 32)); }
// Groups of a CTA of about `threads`.
int norm_groups(int T, int threads) { return std::max(1, std::min(kNormGroups, threads / T)); }

template <class R, bool kQ, int VPT, int MAXT, int CTAS>
cudaError_t launch_norm_groups(NormParams p, cudaStream_t st) {
  p.T = norm_group(p.H, VPT);
  const int groups = norm_groups(p.T, MAXT);
  rms_norm_kernel<R, kQ, VPT, MAXT, CTAS>
      <<<static_cast<unsigned>(ceil_div(p.N, groups)), groups * p.T, 0, st>>>(p);
  return cudaGetLastError();
}
template <bool kRes, bool kQ, int VPL, int CTAS>
cudaError_t launch_norm_warps(const NormParams& p, cudaStream_t st) {
  rms_norm_warp_kernel<kRes, kQ, VPL, CTAS>
      <<<static_cast<unsigned>(ceil_div(p.N, NORM_WARP_ROWS)), 32 * NORM_WARP_ROWS, 0, st>>>(p);
  return cudaGetLastError();
}

// A warp to a row where the row fits its registers beside what else it needs:
// without a residual up to 4,096 elements, with a bf16 residual up to 1,024
// (262,144 x 256: 81 against 100 us; at 1,024 81 either way, at 4,096 87 against
// 81).  Without one, bf16 / e4m3 us for 335 M elements in rows of
//            1,536      2,048      2,304      2,560      2,816      3,584      4,096
//   8        197 / 188  197 / 172
//   10       197 / 193  197 / 174  199 / 170  197 / 166
//   16       246 / 274  215 / 233  209 / 223  203 / 213  199 / 207  199 / 193  201 / 186
//   groups   221 / 238  219 / 236  231 / 254  223 / 240  250 / 266  229 / 246  221 / 240
// vectors to a lane (ten are as many as three CTAs to an SM leave registers for).
// Else groups of two vectors to a thread in CTAs of about 512 threads; past
// 8,192 elements four, so that a row fits a CTA.  Those rows, 134 M elements,
// bf16 / e4m3 us: with a bf16 residual 160 / 141 at 12,288, 160 / 139 at 16,384,
// 170 / 164 at 20,480, 164 / 152 at 32,768 (floors 160 / 140); without one 90 /
// 104, 98 / 92, 129 / 125 and 111 / 106 (80 / 60): one row to a CTA, whose loads
// wait for its reduction.
template <class R, bool kQ>
cudaError_t launch_norm_as(const NormParams& p, cudaStream_t st) {
  constexpr bool kRes = !std::is_same<R, NoResidual>::value;
  if constexpr (!std::is_same<R, float>::value) {
    if (p.H <= 256) return launch_norm_warps<kRes, kQ, 1, 6>(p, st);
    if (p.H <= 512) return launch_norm_warps<kRes, kQ, 2, 6>(p, st);
    if (p.H <= 1024) return launch_norm_warps<kRes, kQ, 4, 4>(p, st);
  }
  if constexpr (!kRes) {
    if (p.H <= 2048) return launch_norm_warps<false, kQ, 8, 3>(p, st);
    if (p.H <= 2560) return launch_norm_warps<false, kQ, 10, 3>(p, st);
    if (p.H <= 4096) return launch_norm_warps<false, kQ, 16, 2>(p, st);
  }
  // 32 registers and four CTAs to an SM pay without a residual to read, 40 and
  // three with one (16,384 x 4,096 fp32: 118 against 124 us)
  if (p.H <= 8192) return launch_norm_groups<R, kQ, 2, 512, kRes ? 2 : 4>(p, st);
  if (p.H <= 16384) return launch_norm_groups<R, kQ, 4, 512, 2>(p, st);
  return launch_norm_groups<R, kQ, 4, 1024, 1>(p, st);
}

template <bool kQ>
cudaError_t launch_norm(const NormParams& p, bool res, bool res_f32, cudaStream_t st) {
  if (!res) return launch_norm_as<NoResidual, kQ>(p, st);
  return res_f32 ? launch_norm_as<float, kQ>(p, st) : launch_norm_as<uint16_t, kQ>(p, st);
}

// How the backward runs rows of H: vectors per thread, the group, the groups
// of a CTA and the CTAs.  The latency of a row (its loads, a reduction, its
// stores) sets the pace, so as many rows as fit are worked on at once, the
// next one's loads in flight.
//   bf16 stream, H <= 2,048: one vector to a thread, two CTAs of 512 threads
//   (65,536 x 1,024: 85 us against 90 for the next shape); up to 8,192 two
//   vectors, one CTA of up to 896 threads (131,072 x 2,560: 305 us against 359
//   with 512 threads and 359 with one vector; 16,384 x 4,096: 85 against 89 and
//   89).  Two rows deep in shared memory: three and four take as long.
//   fp32 stream: straight from global memory, whose second read hits L1
//   (16,384 x 4,096: 190 us against 238 through shared memory, where a
//   thread's 32 bytes of a row halve every access).
//   Past 8,192 elements one row to a CTA, 1.3 to 2.5 times the floor (134 M
//   elements with the stream's own gradient, bf16 / fp32 stream: 237 / 526 us at
//   12,288, 213 / 440 at 16,384, 395 / 524 at 20,480, 295 / 571 at 32,768; floors
//   160 / 321).
struct NormBwdShape {
  int vpt, T, groups, ctas;
};
NormBwdShape norm_bwd_shape(int64_t N, int64_t H, bool f32) {
  NormBwdShape b;
  const bool one = H <= (f32 ? 4096 : 2048);
  b.vpt = one ? 1 : H <= 8192 ? 2 : 4;
  b.T = norm_group(H, b.vpt);
  b.groups = norm_groups(b.T, b.vpt == 2 ? 896 : 512);
  const int64_t most = (one ? 2LL : 1LL) * device_sms();
  b.ctas = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(ceil_div(N, b.groups), most)));
  return b;
}

template <class S, int VPT, int DEPTH, int MAXT, int CTAS>
cudaError_t launch_norm_bwd_as(const NormBwdParams& p, const NormBwdShape& b, cudaStream_t st) {
  const int threads = b.groups * b.T;
  const size_t stage = static_cast<size_t>(threads) * VPT * 8 * (2 + (p.up ? 2 : 1) * sizeof(S));
  // the rows in flight, then the groups' dweight: at most 2 x 86,016 bytes, and 57,344
  const size_t smem = std::max(DEPTH * stage, p.part ? static_cast<size_t>(b.groups - 1) * p.H * 4 : 0);
  auto kern = rms_norm_bwd_kernel<S, VPT, DEPTH, MAXT, CTAS>;
  if (smem > 32768) {  // (the kernel has 8 KB of its own beside it)
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 204800);
    if (e != cudaSuccess) return e;
  }
  kern<<<b.ctas, threads, smem, st>>>(p);
  return cudaGetLastError();
}

template <class S>
cudaError_t launch_norm_bwd(const NormBwdParams& p, const NormBwdShape& b, cudaStream_t st) {
  constexpr bool f32 = std::is_same<S, float>::value;
  if (b.vpt == 1) return launch_norm_bwd_as<S, 1, f32 ? 0 : 2, 512, 2>(p, b, st);
  if (b.vpt == 2) return launch_norm_bwd_as<S, 2, f32 ? 0 : 2, 896, 1>(p, b, st);
  if (b.T <= 512) return launch_norm_bwd_as<S, 4, f32 ? 0 : 1, 512, 1>(p, b, st);
  return launch_norm_bwd_as<S, 4, 0, 1024, 1>(p, b, st);
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
  // of either stream type
  return align256(static_cast<size_t>(std::max(norm_bwd_shape(N, H, false).ctas, norm_bwd_shape(N, H, true).ctas)) * H * 4);
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
  const NormBwdShape b = norm_bwd_shape(N, H, s_type == FLCE_F32);
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
