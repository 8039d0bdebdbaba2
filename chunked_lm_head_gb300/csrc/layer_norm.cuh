// libflce: the layer norm in front of the LM head, with the residual's addition,
// and its backward.
//
// Per row, with s the residual stream as it is stored:
//   s    = round(x + r)            (r's type; s = x without a residual)
//   mean = sum_j s_j / H,  rstd = 1 / sqrt(sum_j (s_j - mean)^2 / H + eps)
//   n_j  = (s_j - mean) rstd,  y_j = n_j gain_j + bias_j,  gain_j = weight_j + offset
// The row stays in registers, so the squares are summed about the mean that was
// found (not as a difference of two large sums).  Backward, g_j = dy_j gain_j:
//   ds_j      = up_j + rstd (g_j - (sum_k g_k) / H - n_j (sum_k g_k n_k) / H)
//   dweight_j = sum_rows dy_j n_j,  dbias_j = sum_rows dy_j
// (up: the gradient that reaches the stream past the norm).  Every sum is in
// fp32, in a fixed order.
#pragma once

#include "norm.cuh"
#include "topk.cuh"

namespace flce {

struct LayerParams {
  const uint16_t* x;
  const void* r;       // residual, R
  const void* weight;  // bf16, or fp32 with w_f32
  const void* bias;    // of weight's type, or null
  long long ldx, ldr;  // row strides of x and r, in elements
  int N, H, w_f32;
  int T;               // threads of a row's group
  float offset, eps;
  uint16_t* y;         // bf16 [N][H]
  void* s;             // the stream [N][H], R
  float* mean;         // [N], or null
  float* rstd;         // [N], or null
};

// n gain + bias for 8 elements from column c on.
__device__ __forceinline__ void layer_affine(const LayerParams& p, int c, float2 (&n)[4]) {
  float2 g[4];
  gain8(p.weight, p.w_f32, p.offset, c, g);
  if (p.bias != nullptr) {
    float2 b[4];
    gain8(p.bias, p.w_f32, 0.f, c, b);
#pragma unroll
    for (int k = 0; k < 4; ++k) n[k] = fma2(n[k], g[k], b[k]);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) n[k] = mul2(n[k], g[k]);
  }
}

// One row on a group of T threads, VPT vectors of 8 elements to a thread in
// registers as the stream is stored (H <= 8 T VPT): the row is read once.
template <class R, int VPT, int MAXT, int CTAS>
__global__ void __launch_bounds__(MAXT, CTAS) layer_norm_kernel(const __grid_constant__ LayerParams p) {
  constexpr bool kRes = !std::is_same<R, NoResidual>::value;
  constexpr bool kWide = std::is_same<R, float>::value;
  __shared__ float red[kNormGroups][64];
  const int T = p.T;
  const int group = threadIdx.x / T, t = threadIdx.x - group * T;
  const int row = blockIdx.x * (blockDim.x / T) + group;
  if (row >= p.N) return;  // whole groups
  const int nv = p.H / 8;
  const uint16_t* x = p.x + row * p.ldx;
  const long long o = static_cast<long long>(row) * p.H;
  Raw8<typename std::conditional<kWide, float, uint16_t>::type> s[VPT];
  float2 sum2 = both(0.f);
  {
    Raw8<uint16_t> xr[kRes ? VPT : 1];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (t + i * T) * 8;
      if (t + i * T < nv) {
        if constexpr (kRes) {
          xr[i].load(x + c);
          s[i].load(static_cast<const R*>(p.r) + row * p.ldr + c);
        } else {
          s[i].load(x + c);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (t + i * T) * 8;
      if (t + i * T < nv) {
        if constexpr (kRes) {
          s[i].add(xr[i]);
          s[i].store(static_cast<R*>(p.s) + o + c);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) sum2 = add2(sum2, s[i].pair(k));
      }
    }
  }
  float sum = sum2.x + sum2.y, none = 0.f;
  group_reduce<false>(sum, none, T, group, t, red[group]);
  const float mean = sum / static_cast<float>(p.H);
  sum2 = both(0.f);
#pragma unroll
  for (int i = 0; i < VPT; ++i)
    if (t + i * T < nv) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 d = add2(s[i].pair(k), both(-mean));
        sum2 = fma2(d, d, sum2);
      }
    }
  sum = sum2.x + sum2.y;
  group_reduce<false>(sum, none, T, group, t, red[group] + 32);
  const float rstd = 1.f / sqrtf(sum / static_cast<float>(p.H) + p.eps);
  if (t == 0) {
    if (p.mean != nullptr) p.mean[row] = mean;
    if (p.rstd != nullptr) p.rstd[row] = rstd;
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (t + i * T) * 8;
    if (t + i * T < nv) {
      float2 v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = mul2(add2(s[i].pair(k), both(-mean)), both(rstd));
      layer_affine(p, c, v);
      store8(p.y + o + c, v);
    }
  }
}

// Rows on a warp each, VPL vectors of 8 elements to a lane (H <= 256 VPL), the
// bf16 stream kept as it is stored: no barrier.
template <bool kRes, int VPL, int CTAS>
__global__ void __launch_bounds__(32 * NORM_WARP_ROWS, CTAS) layer_norm_warp_kernel(const __grid_constant__ LayerParams p) {
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
    Raw8<uint16_t> rr[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (lane + i * 32 < nv) rr[i].load(r + i * 256);
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (lane + i * 32 < nv) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 v = add2(s[i].pair(k), rr[i].pair(k));
          w[k] = pack_bf16x2(v.x, v.y);
        }
        s[i].q[0] = make_uint4(w[0], w[1], w[2], w[3]);
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.s) + o + i * 256) = s[i].q[0];
      }
  }
  float2 sum2 = both(0.f);
#pragma unroll
  for (int i = 0; i < VPL; ++i)
    if (lane + i * 32 < nv) {
#pragma unroll
      for (int k = 0; k < 4; ++k) sum2 = add2(sum2, s[i].pair(k));
    }
  const float mean = warp_sum(sum2.x + sum2.y) / static_cast<float>(p.H);
  sum2 = both(0.f);
#pragma unroll
  for (int i = 0; i < VPL; ++i)
    if (lane + i * 32 < nv) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 d = add2(s[i].pair(k), both(-mean));
        sum2 = fma2(d, d, sum2);
      }
    }
  const float rstd = 1.f / sqrtf(warp_sum(sum2.x + sum2.y) / static_cast<float>(p.H) + p.eps);
  if (lane == 0) {
    if (p.mean != nullptr) p.mean[row] = mean;
    if (p.rstd != nullptr) p.rstd[row] = rstd;
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i)
    if (lane + i * 32 < nv) {
      float2 v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = mul2(add2(s[i].pair(k), both(-mean)), both(rstd));
      layer_affine(p, lane * 8 + i * 256, v);
      store8(p.y + o + i * 256, v);
    }
}

struct LayerBwdParams {
  const uint16_t* dy;  // [N][H] bf16
  const void* s;       // the stream, S, row stride lds
  const void* up;      // [N][H] S: gradient of the stream, or null
  const void* weight;  // bf16, or fp32 with w_f32
  const float* mean;
  const float* rstd;
  long long lds;
  int N, H, w_f32;
  int T;               // threads of a row's group
  float offset;
  uint16_t* dx;        // bf16 [N][H], or null
  float* dr;           // fp32 [N][H], or null
  float* part_w;       // dweight partials [gridDim.x][H], or null
  float* part_b;       // dbias partials, or null
};

// Sums of two values over a group, in a fixed order (as group_reduce).
__device__ __forceinline__ void group_sum2(float2& a, int T, int group, int t, float2* smem) {
  const auto warp_both = [](float2& v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
      v = add2(v, make_float2(__shfl_xor_sync(0xffffffffu, v.x, off), __shfl_xor_sync(0xffffffffu, v.y, off)));
  };
  warp_both(a);
  if (T > 32) {
    const int warp = t >> 5, lane = t & 31, warps = T >> 5;
    if (lane == 0) smem[warp] = a;
    asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(T) : "memory");
    a = lane < warps ? smem[lane] : both(0.f);
    warp_both(a);
  }
}

// Backward rows, dealt to the grid's groups in turn; the rows' copies through
// shared memory and the sums over rows as rms_norm_bwd_kernel.  A thread keeps
// its columns' dweight and (kBias) dbias in registers over all its rows.
template <class S, bool kBias, int VPT, int DEPTH, int MAXT, int CTAS>
__global__ void __launch_bounds__(MAXT, CTAS) layer_norm_bwd_kernel(const __grid_constant__ LayerBwdParams p) {
  constexpr bool kGainRegs = VPT <= 2;
  constexpr int SQ = static_cast<int>(sizeof(S) / 2);  // 16-byte pieces of 8 elements of the stream
  __shared__ float2 red[2][kNormGroups][32];
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
  float2 dw[VPT][4], db[kBias ? VPT : 1][4], gain[kGainRegs ? VPT : 1][4];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      dw[i][k] = both(0.f);
      if constexpr (kBias) db[i][k] = both(0.f);
    }
    if constexpr (kGainRegs) {
      if (t + i * T < nv) gain8(p.weight, p.w_f32, p.offset, (t + i * T) * 8, gain[i]);
    }
  }
  const float inv = 1.f / static_cast<float>(p.H);
  int row = blockIdx.x * groups + group, phase = 0, stage = 0;
#pragma unroll
  for (int d = 0; d < DEPTH - 1; ++d) fetch(row + d * step, d);
  float rstd_next = row < p.N ? p.rstd[row] : 0.f, mean_next = row < p.N ? p.mean[row] : 0.f;
  for (; row < p.N; row += step, phase ^= 1) {
    const long long o = static_cast<long long>(row) * p.H;
    const float rstd = rstd_next, mean = mean_next;
    const bool more = row + step < p.N;
    rstd_next = more ? p.rstd[row + step] : 0.f;
    mean_next = more ? p.mean[row + step] : 0.f;
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
    // n = (s - mean) rstd: the difference first, so that a row far from 0 keeps its bits
    auto normed = [&](float2 s) { return mul2(add2(s, both(-mean)), both(rstd)); };
    float2 sum_g = both(0.f), sum_gn = both(0.f);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      if (t + i * T < nv) {
        Raw8<uint16_t> dy;
        Raw8<S> s;
        read(i, dy, s);
        if constexpr (!kGainRegs) gain8(p.weight, p.w_f32, p.offset, (t + i * T) * 8, gain[0]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 d = dy.pair(k), n = normed(s.pair(k));
          dw[i][k] = fma2(d, n, dw[i][k]);
          if constexpr (kBias) db[i][k] = add2(db[i][k], d);
          const float2 g = mul2(d, gain[kGainRegs ? i : 0][k]);
          sum_g = add2(sum_g, g);
          sum_gn = fma2(g, n, sum_gn);
        }
      }
    }
    float2 sums = make_float2(sum_g.x + sum_g.y, sum_gn.x + sum_gn.y);
    group_sum2(sums, T, group, t, red[phase][group]);
    const float c0 = -sums.x * inv, c1 = -sums.y * inv;
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
          d[k] = fma2(both(rstd),
                      fma2(normed(s.pair(k)), both(c1), fma2(dy.pair(k), gain[kGainRegs ? i : 0][k], both(c0))),
                      up.pair(k));
        if (p.dr != nullptr) store8(p.dr + o + c, d);
        if (p.dx != nullptr) store8(p.dx + o + c, d);
      }
    }
    stage = stage + 1 >= DEPTH ? 0 : stage + 1;
  }
  // the groups of a CTA are joined in shared memory, in group order
  auto join = [&](float2 (&a)[VPT][4], float* part) {
    if (part == nullptr) return;
    if (groups > 1) {
      float* other = reinterpret_cast<float*>(slots);
      __syncthreads();  // every group has read its last row (and the sums before these)
      if (group > 0) {
#pragma unroll
        for (int i = 0; i < VPT; ++i)
          if (t + i * T < nv) store8(other + static_cast<size_t>(group - 1) * p.H + (t + i * T) * 8, a[i]);
      }
      __syncthreads();
      if (group > 0) return;
      for (int g = 0; g < groups - 1; ++g)
#pragma unroll
        for (int i = 0; i < VPT; ++i)
          if (t + i * T < nv) {
            Raw8<float> v;
            v.load(other + static_cast<size_t>(g) * p.H + (t + i * T) * 8);
#pragma unroll
            for (int k = 0; k < 4; ++k) a[i][k] = add2(a[i][k], v.pair(k));
          }
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (t + i * T < nv) store8(part + static_cast<long long>(blockIdx.x) * p.H + (t + i * T) * 8, a[i]);
  };
  join(dw, p.part_w);
  if constexpr (kBias) join(db, p.part_b);
}

// dweight (blockIdx.y 0) and dbias (1) = their partials' sums over the CTAs, in
// their order (as norm_dweight_kernel).
template <class W>
__global__ void __launch_bounds__(1024) layer_dparam_kernel(const float* __restrict__ part_w,
                                                           const float* __restrict__ part_b, int slots, int H,
                                                           W* __restrict__ dw, W* __restrict__ db) {
  __shared__ float sh[32][33];
  const int lane = threadIdx.x & 31, run = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  const float* part = blockIdx.y == 0 ? part_w : part_b;
  W* out = blockIdx.y == 0 ? dw : db;
  if (out == nullptr) return;
  float a = 0.f;
  if (c < H)
    for (int i = run; i < slots; i += 32) a += part[static_cast<long long>(i) * H + c];
  sh[run][lane] = a;
  __syncthreads();
  if (run == 0 && c < H) {
#pragma unroll
    for (int k = 1; k < 32; ++k) a += sh[k][lane];
    if constexpr (std::is_same<W, float>::value)
      out[c] = a;
    else
      out[c] = static_cast<uint16_t>(pack_bf16x2(a, 0.f) & 0xffffu);
  }
}

}  // namespace flce
