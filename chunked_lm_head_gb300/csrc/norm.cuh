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

// 8 consecutive elements as they lie in memory; pair(k) as fp32.
template <class S>
struct Raw8 {
  static constexpr int kQuads = static_cast<int>(sizeof(S) / 2);
  uint4 q[kQuads];
  __device__ __forceinline__ void load(const S* p) {
#pragma unroll
    for (int k = 0; k < kQuads; ++k) q[k] = reinterpret_cast<const uint4*>(p)[k];
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int k = 0; k < kQuads; ++k) q[k] = make_uint4(0u, 0u, 0u, 0u);
  }
  __device__ __forceinline__ float2 pair(int k) const {
    if constexpr (sizeof(S) == 4) {
      const uint32_t w[4] = {q[k / 2].x, q[k / 2].y, q[k / 2].z, q[k / 2].w};
      return make_float2(__uint_as_float(w[2 * (k % 2)]), __uint_as_float(w[2 * (k % 2) + 1]));
    } else {
      const uint32_t w[4] = {q[0].x, q[0].y, q[0].z, q[0].w};
      return make_float2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xffff0000u));
    }
  }
};
// 8 values rounded to the element type; v becomes what was stored.
__device__ __forceinline__ void store8(uint16_t* p, float2 (&v)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    w[k] = pack_bf16x2(v[k].x, v[k].y);
    v[k] = make_float2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xffff0000u));
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float* p, const float2 (&v)[4]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
}
__device__ __forceinline__ void store8_e4m3(uint8_t* p, const float2 (&v)[4]) {
  uint32_t b[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(v[2 * k], __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(v[2 * k + 1], __NV_SATFINITE, __NV_E4M3);
    b[k] = lo | (hi << 16);
  }
  *reinterpret_cast<uint2*>(p) = make_uint2(b[0], b[1]);
}

// 8 gains from column c on: weight (fp32 or bf16) + offset.
__device__ __forceinline__ void gain8(const void* w, int f32, float offset, int c, float2 (&v)[4]) {
  if (f32) {
    Raw8<float> r;
    r.load(static_cast<const float*>(w) + c);
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = r.pair(k);
  } else {
    Raw8<uint16_t> r;
    r.load(static_cast<const uint16_t*>(w) + c);
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = r.pair(k);
  }
  if (offset != 0.f) {
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = add2(v[k], both(offset));
  }
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

// The e4m3 scale of a row from rstd and top = max_j |s_j gain_j|, and the
// factors with q_j = e4m3((s_j gain_j up) f): y / scale without a division per
// element.  448 / top passes fp32's range below 2^-119; such a row is taken
// times 2^64 first, which rounds nothing (tiny_row).
struct RowScale {
  float scale, f, up;
};
__device__ __forceinline__ RowScale row_scale(float rstd, float top) {
  const float s = rstd * top / 448.f;
  // an all-zero row (or one whose scale rounds to zero), and one that holds a
  // NaN or an infinity, has scale 1
  RowScale e{s > 0.f ? s : 1.f, 0.f, 1.f};
  if (s > 0.f && top < 0x1p-119f) e.up = 0x1p64f;
  e.f = rstd / (e.scale * e.up);
  return e;
}

// The e4m3 row whose factor `up` is not 1, from the stream s as it is in memory
// (each thread reads what it stored): a path of its own, so that no other row's
// registers pay for it.
template <class S>
__device__ __forceinline__ void tiny_row(const S* s, const NormParams& p, long long o, int t, int T, const RowScale& e) {
#pragma unroll 1
  for (int i = t; i < p.H / 8; i += T) {
    Raw8<S> v;
    v.load(s + i * 8);
    float2 g[4], y[4];
    gain8(p.weight, p.w_f32, p.offset, i * 8, g);
#pragma unroll
    for (int k = 0; k < 4; ++k) y[k] = mul2(mul2(mul2(v.pair(k), g[k]), both(e.up)), both(e.f));
    store8_e4m3(p.q + o + i * 8, y);
  }
}

// One row on a group of T threads, VPT vectors of 8 elements to a thread in
// registers (H <= 8 T VPT): the row is read once.  Bound by memory: with a bf16
// residual 32,768 x 4,096 takes 157 us in bf16 and 142 in e4m3 (6.8 and 6.6
// TB/s).
constexpr int kNormGroups = 15;  // groups of a CTA at most (named barriers 1 to 15)

template <class R, bool kQ, int VPT, int MAXT, int CTAS>
__global__ void __launch_bounds__(MAXT, CTAS) rms_norm_kernel(const __grid_constant__ NormParams p) {
  constexpr bool kRes = !std::is_same<R, NoResidual>::value;
  __shared__ float red[kNormGroups][64];
  const int T = p.T;
  const int group = threadIdx.x / T, t = threadIdx.x - group * T;
  const int row = blockIdx.x * (blockDim.x / T) + group;
  if (row >= p.N) return;  // whole groups
  const int nv = p.H / 8;
  const uint16_t* x = p.x + row * p.ldx;
  const long long o = static_cast<long long>(row) * p.H;
  float2 v[VPT][4];
  float2 sum2 = both(0.f);
  float top = 0.f;
  {
    Raw8<uint16_t> xr[VPT];
    Raw8<typename std::conditional<kRes, R, uint16_t>::type> rr[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (t + i * T) * 8;
      if (t + i * T < nv) {
        xr[i].load(x + c);
        if constexpr (kRes) rr[i].load(static_cast<const R*>(p.r) + row * p.ldr + c);
      }
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (t + i * T) * 8;
      if (t + i * T < nv) {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[i][k] = xr[i].pair(k);
        if constexpr (kRes) {
#pragma unroll
          for (int k = 0; k < 4; ++k) v[i][k] = add2(v[i][k], rr[i].pair(k));
          store8(static_cast<R*>(p.s) + o + c, v[i]);
        }
        // with kQ v becomes s gain, whose largest magnitude counts
        // (max_j |y_j| = rstd max_j |s_j gain_j|)
        float2 g[4];
        if constexpr (kQ) gain8(p.weight, p.w_f32, p.offset, c, g);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          sum2 = fma2(v[i][k], v[i][k], sum2);
          if constexpr (kQ) {
            v[i][k] = mul2(v[i][k], g[k]);
            top = fmaxf(top, fmaxf(fabsf(v[i][k].x), fabsf(v[i][k].y)));
          }
        }
      }
    }
  }
  float sum = sum2.x + sum2.y;
  group_reduce<kQ>(sum, top, T, group, t, red[group]);
  const float rstd = 1.f / sqrtf(sum / static_cast<float>(p.H) + p.eps);
  float f = rstd;
  if constexpr (kQ) {
    const RowScale e = row_scale(rstd, top);
    if (t == 0) p.scale[row] = e.scale;
    f = e.f;
    if (e.up != 1.f) {
      if (t == 0 && p.rstd != nullptr) p.rstd[row] = rstd;
      if constexpr (kRes)
        tiny_row(static_cast<const R*>(p.s) + o, p, o, t, T, e);
      else
        tiny_row(x, p, o, t, T, e);
      return;  // the whole group
    }
  }
  if (t == 0 && p.rstd != nullptr) p.rstd[row] = rstd;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (t + i * T) * 8;
    if (t + i * T < nv) {
#pragma unroll
      for (int k = 0; k < 4; ++k) v[i][k] = mul2(v[i][k], both(f));
      if constexpr (kQ) {
        store8_e4m3(p.q + o + c, v[i]);
      } else {
        float2 g[4];
        gain8(p.weight, p.w_f32, p.offset, c, g);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[i][k] = mul2(v[i][k], g[k]);
        store8(p.y + o + c, v[i]);
      }
    }
  }
}

// Rows on a warp each, VPL vectors of 8 elements to a lane (H <= 256 VPL), the
// bf16 stream kept as it is stored: no barrier, and the row's sums cost one
// butterfly instead of one per warp of a group.  131,072 x 2,560 without a
// residual: 197 us in bf16, 167 in e4m3 (6.8 and 6.0 TB/s).
constexpr int NORM_WARP_ROWS = 8;  // rows of a CTA
template <bool kRes, bool kQ, int VPL, int CTAS>
__global__ void __launch_bounds__(32 * NORM_WARP_ROWS, CTAS) rms_norm_warp_kernel(const __grid_constant__ NormParams p) {
  const int lane = threadIdx.x & 31;
  const int nv = p.H / 8;
  const int row = blockIdx.x * NORM_WARP_ROWS + (threadIdx.x >> 5);
  if (row >= p.N) return;
  const uint16_t* x = p.x + row * p.ldx + lane * 8;
  const long long o = static_cast<long long>(row) * p.H + lane * 8;
  Raw8<uint16_t> s[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i)
    if (lane + i * 32 < nv) s[i].load(x + i * 256);
  if constexpr (kRes) {
    const uint16_t* r = static_cast<const uint16_t*>(p.r) + row * p.ldr + lane * 8;
    constexpr int STEP = VPL < 8 ? VPL : 8;
#pragma unroll
    for (int i0 = 0; i0 < VPL; i0 += STEP) {
      Raw8<uint16_t> rr[STEP];
#pragma unroll
      for (int i = 0; i < STEP; ++i)
        if (lane + (i0 + i) * 32 < nv && i0 + i < VPL) rr[i].load(r + (i0 + i) * 256);
#pragma unroll
      for (int i = 0; i < STEP; ++i)
        if (lane + (i0 + i) * 32 < nv && i0 + i < VPL) {
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 v = add2(s[i0 + i].pair(k), rr[i].pair(k));
            w[k] = pack_bf16x2(v.x, v.y);
          }
          s[i0 + i].q[0] = make_uint4(w[0], w[1], w[2], w[3]);
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.s) + o + (i0 + i) * 256) = s[i0 + i].q[0];
        }
    }
  }
  float2 sum2 = both(0.f);
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < VPL; ++i)
    if (lane + i * 32 < nv) {
      float2 g[4];
      if constexpr (kQ) gain8(p.weight, p.w_f32, p.offset, lane * 8 + i * 256, g);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 v = s[i].pair(k);
        sum2 = fma2(v, v, sum2);
        if constexpr (kQ) {
          const float2 m = mul2(v, g[k]);
          top = fmaxf(top, fmaxf(fabsf(m.x), fabsf(m.y)));
        }
      }
    }
  float sum = sum2.x + sum2.y;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, off);
    if constexpr (kQ) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
  }
  const float rstd = 1.f / sqrtf(sum / static_cast<float>(p.H) + p.eps);
  float f = rstd;
  if constexpr (kQ) {
    const RowScale e = row_scale(rstd, top);
    if (lane == 0) p.scale[row] = e.scale;
    f = e.f;
    if (e.up != 1.f) {
      if (lane == 0 && p.rstd != nullptr) p.rstd[row] = rstd;
      const long long row_o = static_cast<long long>(row) * p.H;
      tiny_row(kRes ? static_cast<const uint16_t*>(p.s) + row_o : p.x + row * p.ldx, p, row_o, lane, 32, e);
      return;
    }
  }
  if (lane == 0 && p.rstd != nullptr) p.rstd[row] = rstd;
#pragma unroll
  for (int i = 0; i < VPL; ++i)
    if (lane + i * 32 < nv) {
      float2 g[4], v[4];
      gain8(p.weight, p.w_f32, p.offset, lane * 8 + i * 256, g);
      if constexpr (kQ) {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = mul2(mul2(s[i].pair(k), g[k]), both(f));
        store8_e4m3(p.q + o + i * 256, v);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = mul2(mul2(s[i].pair(k), both(f)), g[k]);
        store8(p.y + o + i * 256, v);
      }
    }
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

// 16 bytes of global memory into shared memory, in this thread's own time.
__device__ __forceinline__ void copy16_async(uint4* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// Backward rows, dealt to the grid's groups in turn.  Each thread copies its
// own columns of the next DEPTH - 1 rows into its own slots of shared memory
// (nothing is shared but the row's sum, so the copies need no barrier) and
// reads them from there in both passes over a row (DEPTH 0: from global
// memory); it keeps its columns' dweight (and, up to two vectors, their gains)
// in registers over all its rows.  The groups of a CTA are joined in shared
// memory at the end, in group order.
// 10 bytes an element with the stream's own gradient, 6 without: 16,384 x 4,096
// 85 us (6.3 TB/s), 131,072 x 2,560 305 us (6.6 TB/s).
template <class S, int VPT, int DEPTH, int MAXT, int CTAS>
__global__ void __launch_bounds__(MAXT, CTAS) rms_norm_bwd_kernel(const __grid_constant__ NormBwdParams p) {
  constexpr bool kGainRegs = VPT <= 2;
  constexpr int SQ = static_cast<int>(sizeof(S) / 2);  // 16-byte pieces of 8 elements of the stream
  __shared__ float red[2][kNormGroups][64];
  extern __shared__ uint4 slots[];  // [DEPTH][VPT][pieces][threads]; then [groups - 1][H] fp32
  const int T = p.T;
  const int group = threadIdx.x / T, t = threadIdx.x - group * T;
  const int groups = blockDim.x / T;
  const int nv = p.H / 8;
  const int step = gridDim.x * groups;
  const int pieces = p.up != nullptr ? 2 * SQ + 1 : SQ + 1;  // dy, the stream, up
  auto slot = [&](int stage, int i, int q) {
    return slots + static_cast<size_t>((stage * VPT + i) * pieces + q) * blockDim.x + threadIdx.x;
  };
  auto fetch = [&](int row, int stage) {
    if constexpr (DEPTH == 0) return;
    if (row < p.N) {
      const S* s = static_cast<const S*>(p.s) + row * p.lds;
      const long long o = static_cast<long long>(row) * p.H;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = (t + i * T) * 8;
        if (t + i * T < nv) {
          copy16_async(slot(stage, i, 0), p.dy + o + c);
#pragma unroll
          for (int q = 0; q < SQ; ++q) copy16_async(slot(stage, i, 1 + q), reinterpret_cast<const uint4*>(s + c) + q);
          if (p.up != nullptr) {
#pragma unroll
            for (int q = 0; q < SQ; ++q)
              copy16_async(slot(stage, i, 1 + SQ + q),
                           reinterpret_cast<const uint4*>(static_cast<const S*>(p.up) + o + c) + q);
          }
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  float2 dw[VPT][4], gain[kGainRegs ? VPT : 1][4];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
#pragma unroll
    for (int k = 0; k < 4; ++k) dw[i][k] = both(0.f);
    if constexpr (kGainRegs) {
      if (t + i * T < nv) gain8(p.weight, p.w_f32, p.offset, (t + i * T) * 8, gain[i]);
    }
  }
  int row = blockIdx.x * groups + group, phase = 0, stage = 0;
#pragma unroll
  for (int d = 0; d < DEPTH - 1; ++d) fetch(row + d * step, d);
  float rstd_next = row < p.N ? p.rstd[row] : 0.f;
  for (; row < p.N; row += step, phase ^= 1) {
    const long long o = static_cast<long long>(row) * p.H;
    const float rstd = rstd_next;
    rstd_next = row + step < p.N ? p.rstd[row + step] : 0.f;
    if constexpr (DEPTH > 0) {
      fetch(row + (DEPTH - 1) * step, stage == 0 ? DEPTH - 1 : stage - 1);
      asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH > 0 ? DEPTH - 1 : 0) : "memory");  // this row's copies are done
    }
    auto read = [&](int i, Raw8<uint16_t>& dy, Raw8<S>& s) {
      if constexpr (DEPTH > 0) {
        dy.q[0] = *slot(stage, i, 0);
#pragma unroll
        for (int q = 0; q < SQ; ++q) s.q[q] = *slot(stage, i, 1 + q);
      } else {
        dy.load(p.dy + o + (t + i * T) * 8);
        s.load(static_cast<const S*>(p.s) + row * p.lds + (t + i * T) * 8);
      }
    };
    float2 dot2 = both(0.f);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      if (t + i * T < nv) {
        Raw8<uint16_t> dy;
        Raw8<S> s;
        read(i, dy, s);
        if constexpr (!kGainRegs) gain8(p.weight, p.w_f32, p.offset, (t + i * T) * 8, gain[0]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 d = dy.pair(k), sv = s.pair(k);
          dw[i][k] = fma2(d, mul2(sv, both(rstd)), dw[i][k]);
          dot2 = fma2(mul2(d, gain[kGainRegs ? i : 0][k]), sv, dot2);
        }
      }
    }
    float dot = dot2.x + dot2.y, none = 0.f;
    group_reduce<false>(dot, none, T, group, t, red[phase][group]);
    const float k2 = dot / static_cast<float>(p.H) * rstd * rstd;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (t + i * T) * 8;
      if (t + i * T < nv) {
        Raw8<uint16_t> dy;
        Raw8<S> s, up;
        read(i, dy, s);
        up.zero();
        if (p.up != nullptr) {
          if constexpr (DEPTH > 0) {
#pragma unroll
            for (int q = 0; q < SQ; ++q) up.q[q] = *slot(stage, i, 1 + SQ + q);
          } else {
            up.load(static_cast<const S*>(p.up) + o + c);
          }
        }
        if constexpr (!kGainRegs) gain8(p.weight, p.w_f32, p.offset, c, gain[0]);
        float2 d[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          d[k] = fma2(both(rstd), fma2(s.pair(k), both(-k2), mul2(dy.pair(k), gain[kGainRegs ? i : 0][k])),
                      up.pair(k));
        if (p.dr != nullptr) store8(p.dr + o + c, d);
        if (p.dx != nullptr) store8(p.dx + o + c, d);
      }
    }
    stage = stage + 1 >= DEPTH ? 0 : stage + 1;
  }
  if (p.part != nullptr) {
    if (groups > 1) {
      float* join = reinterpret_cast<float*>(slots);
      __syncthreads();  // every group has read its last row
      if (group > 0) {
#pragma unroll
        for (int i = 0; i < VPT; ++i)
          if (t + i * T < nv) store8(join + static_cast<size_t>(group - 1) * p.H + (t + i * T) * 8, dw[i]);
      }
      __syncthreads();
      if (group > 0) return;
      for (int g = 0; g < groups - 1; ++g)
#pragma unroll
        for (int i = 0; i < VPT; ++i)
          if (t + i * T < nv) {
            Raw8<float> v;
            v.load(join + static_cast<size_t>(g) * p.H + (t + i * T) * 8);
#pragma unroll
            for (int k = 0; k < 4; ++k) dw[i][k] = add2(dw[i][k], v.pair(k));
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
