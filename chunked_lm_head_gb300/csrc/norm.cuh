// libflce: the root-mean-square norm in front of the LM head, with the
// residual's addition, in bf16 or in e4m3 with one scale per row, and its
// backward.
//
// Per row, with s the residual stream as it is stored:
//   s    = round(x + r)            (r's type; s = x without a residual)
//   rstd = 1 / sqrt(sum_j s_j^2 / H + eps)
//   y_j  = s_j rstd gain_j,        gain_j = weight_j + offset
// bf16: y rounded once.  e4m3: scale = max_j |y_j| / 448, q_j = e4m3(y_j / scale)
// straight from the 32-bit y.  Backward, with g_j = dy_j gain_j:
//   ds_j = up_j + rstd (g_j - s_j rstd^2 (sum_k g_k s_k) / H)
//   dweight_j = sum_rows dy_j s_j rstd
// (up: the gradient that reaches the stream past the norm).  Every sum is in
// fp32.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <cstdint>
#include <type_traits>

#include "gemm.cuh"

namespace flce {

struct NoResidual {};  // kernel residual type of a call without one

// 8 consecutive elements, as fp32.
__device__ __forceinline__ void load8(const uint16_t* p, float (&v)[8]) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    v[2 * k] = __uint_as_float(w[k] << 16);
    v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
// 8 values rounded to the element type; v becomes what was stored.
__device__ __forceinline__ void store8(uint16_t* p, float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    w[k] = pack_bf16x2(v[2 * k], v[2 * k + 1]);
    v[2 * k] = __uint_as_float(w[k] << 16);
    v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float* p, float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// 8 gains from column c on: weight (fp32 or bf16) + offset.
__device__ __forceinline__ void gain8(const void* w, int f32, float offset, int c, float (&v)[8]) {
  if (f32)
    load8(static_cast<const float*>(w) + c, v);
  else
    load8(static_cast<const uint16_t*>(w) + c, v);
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] += offset;
}

// A CTA holds `groups` rows at a time, each on its own group of T threads (a
// multiple of 32): sum (and maximum) over the group, in a fixed order, joined
// through the group's 2 x 32 floats of shared memory behind a named barrier
// (id 1 + group, at most 15 of them).  A group of one warp needs neither.
template <bool kMax>
__device__ __forceinline__ void group_reduce(float& sum, float& top, int T, int group, int t, float* smem) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, off);
    if constexpr (kMax) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
  }
  if (T > 32) {
    const int warp = t >> 5, lane = t & 31, warps = T >> 5;
    if (lane == 0) {
      smem[warp] = sum;
      if constexpr (kMax) smem[32 + warp] = top;
    }
    asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(T) : "memory");
    sum = lane < warps ? smem[lane] : 0.f;
    if constexpr (kMax) top = lane < warps ? smem[32 + lane] : 0.f;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      sum += __shfl_xor_sync(0xffffffffu, sum, off);
      if constexpr (kMax) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    }
  }
}

struct NormParams {
  const uint16_t* x;
  const void* r;       // residual, R
  const void* weight;  // bf16, or fp32 with w_f32
  long long ldx, ldr;  // row strides of x and r, in elements
  int N, H, w_f32;
  int T;               // threads of a row's group
  float offset, eps;
  uint16_t* y;         // bf16 [N][H]
  uint8_t* q;          // e4m3 [N][H] and
  float* scale;        // its row scales [N]
  void* s;             // the stream [N][H], R
  float* rstd;         // [N], or null
};

// One row on a group of T threads, VPT vectors of 8 elements to a thread in
// registers (H <= 8 T VPT): the row is read once.
constexpr int kNormGroups = 8;  // groups of a CTA at most

template <class R, bool kQ, int VPT>
__global__ void __launch_bounds__(1024) rms_norm_kernel(const __grid_constant__ NormParams p) {
  constexpr bool kRes = !std::is_same<R, NoResidual>::value;
  __shared__ float red[kNormGroups][64];
  const int T = p.T;
  const int group = threadIdx.x / T, t = threadIdx.x - group * T;
  const int row = blockIdx.x * (blockDim.x / T) + group;
  if (row >= p.N) return;  // whole groups
  const uint16_t* x = p.x + row * p.ldx;
  const long long o = static_cast<long long>(row) * p.H;
  const int nv = p.H / 8;

  // 8 elements of the stream from column c on, stored when there is a residual
  auto stream8 = [&](int c, float (&v)[8]) {
    load8(x + c, v);
    if constexpr (kRes) {
      float r8[8];
      load8(static_cast<const R*>(p.r) + row * p.ldr + c, r8);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] += r8[k];
      store8(static_cast<R*>(p.s) + o + c, v);
    }
  };
  float sum = 0.f, top = 0.f;
  float s[VPT][8];
  // one vector's share of the sum of squares; with kQ v becomes s gain and
  // its largest magnitude counts (max_j |y_j| = rstd max_j |s_j gain_j|)
  auto take8 = [&](int c, float (&v)[8]) {
    float g8[8];
    if constexpr (kQ) gain8(p.weight, p.w_f32, p.offset, c, g8);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      sum = fmaf(v[k], v[k], sum);
      if constexpr (kQ) {
        v[k] *= g8[k];
        top = fmaxf(top, fabsf(v[k]));
      }
    }
  };
#pragma unroll
  for (int i = 0; i < VPT; ++i)
    if (t + i * T < nv) stream8((t + i * T) * 8, s[i]);
#pragma unroll
  for (int i = 0; i < VPT; ++i)
    if (t + i * T < nv) take8((t + i * T) * 8, s[i]);
  group_reduce<kQ>(sum, top, T, group, t, red[group]);
  const float rstd = 1.f / sqrtf(sum / static_cast<float>(p.H) + p.eps);
  float f = rstd;
  if constexpr (kQ) {
    const float amax = rstd * top;
    // an all-zero row, and one that holds a NaN or an infinity, has scale 1
    const float sc = amax > 0.f ? amax / 448.f : 1.f;
    if (t == 0) p.scale[row] = sc;
    f = rstd / sc;
  }
  if (t == 0 && p.rstd != nullptr) p.rstd[row] = rstd;
  auto put8 = [&](int c, float (&v)[8]) {
    if constexpr (kQ) {
      uint32_t b[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * k] * f, v[4 * k + 1] * f),
                                                     __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * k + 2] * f, v[4 * k + 3] * f),
                                                     __NV_SATFINITE, __NV_E4M3);
        b[k] = lo | (hi << 16);
      }
      *reinterpret_cast<uint2*>(p.q + o + c) = make_uint2(b[0], b[1]);
    } else {
      float g8[8];
      gain8(p.weight, p.w_f32, p.offset, c, g8);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = v[k] * f * g8[k];
      store8(p.y + o + c, v);
    }
  };
#pragma unroll
  for (int i = 0; i < VPT; ++i)
    if (t + i * T < nv) put8((t + i * T) * 8, s[i]);
}

struct NormBwdParams {
  const uint16_t* dy;  // [N][H] bf16
  const void* s;       // the stream, S, row stride lds
  const void* up;      // [N][H] S: gradient of the stream, or null
  const void* weight;  // bf16, or fp32 with w_f32
  const float* rstd;
  long long lds;
  int N, H, w_f32;
  int T;               // threads of a row's group
  float offset;
  uint16_t* dx;        // bf16 [N][H], or null
  float* dr;           // fp32 [N][H], or null
  float* part;         // dweight partials [gridDim.x][H], or null
};

// 8 elements as they lie in memory.
template <class S>
struct Raw8 {
  uint4 q[sizeof(S) / 2];
  __device__ __forceinline__ void load(const S* p) {
#pragma unroll
    for (int k = 0; k < static_cast<int>(sizeof(S) / 2); ++k) q[k] = reinterpret_cast<const uint4*>(p)[k];
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int k = 0; k < static_cast<int>(sizeof(S) / 2); ++k) q[k] = make_uint4(0u, 0u, 0u, 0u);
  }
  __device__ __forceinline__ float at(int k) const {
    if constexpr (sizeof(S) == 4) {
      const uint4& u = q[k / 4];
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
      return __uint_as_float(w[k % 4]);
    } else {
      const uint32_t w[4] = {q[0].x, q[0].y, q[0].z, q[0].w};
      return __uint_as_float((k & 1) ? (w[k / 2] & 0xffff0000u) : (w[k / 2] << 16));
    }
  }
};

// Backward rows, dealt to the grid's groups in turn.  A group's loads of its
// next row are in flight while it reduces and writes the present one (kAhead);
// each thread keeps its columns' dweight in registers over all its rows, the
// groups of a CTA are joined in shared memory at the end, in group order.
template <class S, int VPT, int MAXT, bool kAhead>
__global__ void __launch_bounds__(MAXT, 1) rms_norm_bwd_kernel(const __grid_constant__ NormBwdParams p) {
  __shared__ float red[2][kNormGroups][64];
  extern __shared__ float dw_groups[];  // [groups - 1][H]
  const int T = p.T;
  const int group = threadIdx.x / T, t = threadIdx.x - group * T;
  const int groups = blockDim.x / T;
  const int nv = p.H / 8;
  const int step = gridDim.x * groups;
  struct Vec {
    Raw8<S> s, up;
    Raw8<uint16_t> dy;
  };
  auto load_row = [&](int row, Vec (&v)[VPT], float& rstd) {
    rstd = p.rstd[row];
    const S* s = static_cast<const S*>(p.s) + row * p.lds;
    const long long o = static_cast<long long>(row) * p.H;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (t + i * T) * 8;
      if (t + i * T < nv) {
        v[i].s.load(s + c);
        v[i].dy.load(p.dy + o + c);
        if (p.up != nullptr) v[i].up.load(static_cast<const S*>(p.up) + o + c);
      }
    }
  };
  float dw[VPT][8];
  Vec cur[VPT], ahead[kAhead ? VPT : 1];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    cur[i].up.zero();
#pragma unroll
    for (int k = 0; k < 8; ++k) dw[i][k] = 0.f;
  }
  if constexpr (kAhead) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) ahead[i].up.zero();
  }
  float rstd = 0.f, rstd_ahead = 0.f;
  int row = blockIdx.x * groups + group, phase = 0;
  if (row < p.N) load_row(row, cur, rstd);
  for (; row < p.N; row += step, phase ^= 1) {
    if constexpr (kAhead) {
      if (row + step < p.N) load_row(row + step, ahead, rstd_ahead);
    }
    float dot = 0.f, none = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      if (t + i * T < nv) {
        float w8[8];
        gain8(p.weight, p.w_f32, p.offset, (t + i * T) * 8, w8);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float sv = cur[i].s.at(k), dy = cur[i].dy.at(k);
          dw[i][k] = fmaf(dy, sv * rstd, dw[i][k]);
          dot = fmaf(dy * w8[k], sv, dot);
        }
      }
    }
    group_reduce<false>(dot, none, T, group, t, red[phase][group]);
    const float k2 = dot / static_cast<float>(p.H) * rstd * rstd;
    const long long o = static_cast<long long>(row) * p.H;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (t + i * T) * 8;
      if (t + i * T < nv) {
        float w8[8], d[8];
        gain8(p.weight, p.w_f32, p.offset, c, w8);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          d[k] = fmaf(rstd, cur[i].dy.at(k) * w8[k] - cur[i].s.at(k) * k2, cur[i].up.at(k));
        if (p.dr != nullptr) store8(p.dr + o + c, d);
        if (p.dx != nullptr) store8(p.dx + o + c, d);
      }
    }
    if constexpr (kAhead) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) cur[i] = ahead[i];
      rstd = rstd_ahead;
    } else {
      if (row + step < p.N) load_row(row + step, cur, rstd);
    }
  }
  if (p.part != nullptr) {
    if (groups > 1) {
      if (group > 0) {
#pragma unroll
        for (int i = 0; i < VPT; ++i)
          if (t + i * T < nv) store8(dw_groups + static_cast<size_t>(group - 1) * p.H + (t + i * T) * 8, dw[i]);
      }
      __syncthreads();
      if (group > 0) return;
      for (int g = 0; g < groups - 1; ++g)
#pragma unroll
        for (int i = 0; i < VPT; ++i)
          if (t + i * T < nv) {
            float v[8];
            load8(dw_groups + static_cast<size_t>(g) * p.H + (t + i * T) * 8, v);
#pragma unroll
            for (int k = 0; k < 8; ++k) dw[i][k] += v[k];
          }
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (t + i * T < nv) store8(p.part + static_cast<long long>(blockIdx.x) * p.H + (t + i * T) * 8, dw[i]);
  }
}

// dweight = the partials' sum over the CTAs, in their order (32 columns to a
// CTA, 32 runs of partials joined at the end).
template <class W>
__global__ void __launch_bounds__(1024) norm_dweight_kernel(const float* __restrict__ part, int slots, int H,
                                                           W* __restrict__ dw) {
  __shared__ float sh[32][33];
  const int lane = threadIdx.x & 31, run = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float a = 0.f;
  if (c < H)
    for (int i = run; i < slots; i += 32) a += part[static_cast<long long>(i) * H + c];
  sh[run][lane] = a;
  __syncthreads();
  if (run == 0 && c < H) {
#pragma unroll
    for (int k = 1; k < 32; ++k) a += sh[k][lane];
    if constexpr (std::is_same<W, float>::value)
      dw[c] = a;
    else
      dw[c] = static_cast<uint16_t>(pack_bf16x2(a, 0.f) & 0xffffu);
  }
}

}  // namespace flce
