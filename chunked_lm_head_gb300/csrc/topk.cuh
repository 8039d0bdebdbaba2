// libflce: the row kernels of the distillation from a teacher's top logits.
//
// Per row, with u the student's transformed logits, S the listed ids, p_k the
// teacher's mass of id k (equal ids added up), P their sum and T = max(0, 1 - P)
// with the tail (else 0), M = P + T:
//   lse_rest = log sum_{v not in S} e^u_v       (the forward GEMM's sum)
//   lse      = log(e^lse_rest + sum_{k in S} e^u_k),  R = e^(lse_rest - lse)
//   kl       = sum_k p_k (log p_k - (u_k - lse)) + T (log T - log R)
//   D_v      = M e^(u_v - lse) - p_v            v in S      (times w g f'(z))
//            = (M R - T) e^(u_v - lse_rest)     v not in S
// The listed columns never enter the GEMM's sum, so R keeps its precision
// when the listed ids hold nearly all of the student's mass, and no division
// by it is needed.  The few sums over K are taken in 64 bits.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <climits>
#include <cstdint>

#include "small_kernels.cuh"

namespace flce {

constexpr int TOPK_WARPS = 4;      // rows per CTA of the list kernel, one warp each
constexpr int TOPK_MAX_K = 1024;   // longest list (its shared memory: 8 bytes per entry and row)
constexpr int TOPK_ROWS = SMALL_THREADS / 32;  // rows per CTA of the row kernel

struct TopkTeacher {
  const void* ids;     // int32 or int64 [N][ld_ids]
  const void* logits;  // fp32, bf16 or fp16 [N][ld_logits]
  const float* lse;    // [N], or null: the row's list sums to one
  long long ld_ids, ld_logits;
  int ids_type, logits_type;  // flce_dtype
  int k, tail;
};

// What the row kernels hand on, per row i and list position j.
struct TopkRows {
  int* ids;          // [N][K] ascending, INT_MAX where there is no entry
  float* mass;       // [N][K] teacher mass of the id (of all its entries)
  float* val;        // [N][K] the student's u_k, then the gradient of its column
  double2* stat;     // [N] sum p log p (NaN: an id outside the vocabulary), P
  long long* mark;   // [N] V for a counted row, -1 for one without loss
  float* lse_rest;   // [N]
  float* coef;       // [N] w (M R - T)
};

__device__ __forceinline__ double warp_sum(double x) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  return x;
}
__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
  return x;
}

__device__ __forceinline__ float topk_logit(const TopkTeacher& t, long long row, int j) {
  const long long o = row * t.ld_logits + j;
  if (t.logits_type == 0) return __bfloat162float(static_cast<const __nv_bfloat16*>(t.logits)[o]);
  if (t.logits_type == 2) return __half2float(static_cast<const __half*>(t.logits)[o]);
  return static_cast<const float*>(t.logits)[o];
}

// The row's list in ascending order of id with the teacher's masses (one warp
// per row).  An entry's place is the number of entries before it (by id, then
// by position), counted in one walk over the list that also adds up the mass
// of equal ids: K^2 / 32 steps of a lane, no barrier.
__global__ void __launch_bounds__(32 * TOPK_WARPS)
    topk_list_kernel(const TopkTeacher t, const int64_t* __restrict__ targets, long long ignore, int N, int V,
                     const TopkRows out) {
  extern __shared__ int topk_smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int K = t.k;
  const long long i = static_cast<long long>(blockIdx.x) * TOPK_WARPS + warp;
  if (i >= N) return;
  int* sid = topk_smem + warp * 2 * K;
  float* sp = reinterpret_cast<float*>(sid + K);
  bool any = false, bad = false;
  float top = -INFINITY;
  for (int j = lane; j < K; j += 32) {
    const long long id = t.ids_type == 4 ? static_cast<const int64_t*>(t.ids)[i * t.ld_ids + j]
                                         : static_cast<const int32_t*>(t.ids)[i * t.ld_ids + j];
    const bool in = id >= 0 && id < V;
    bad |= id >= V;
    any |= in;
    const float u = in ? topk_logit(t, i, j) : -INFINITY;
    sid[j] = in ? static_cast<int>(id) : INT_MAX;
    sp[j] = u;
    top = fmaxf(top, u);
  }
  any = __any_sync(0xffffffffu, any);
  bad = __any_sync(0xffffffffu, bad);
  top = warp_max(top);
  double lse = 0.0;
  bool live = any || bad;
  if (t.lse != nullptr) {
    lse = t.lse[i];
  } else {
    live = live && (top > -INFINITY || bad);  // a list without mass sums to nothing
    double s = 0.0;
    for (int j = lane; j < K; j += 32) s += expf(sp[j] - top);
    lse = top + log(warp_sum(s));
  }
  live = live && (targets == nullptr || targets[i] != ignore);
  __syncwarp();
  // masses in place of the logits; log p = u - lse is needed once more below
  double own_h = 0.0, P = 0.0;
  for (int j = lane; j < K; j += 32) {
    const double lp = static_cast<double>(sp[j]) - lse;
    const float p = sid[j] == INT_MAX ? 0.f : expf(static_cast<float>(lp));
    P += p;
    if (p > 0.f) own_h += p * lp;
    sp[j] = p;
  }
  __syncwarp();
  int* ids_out = out.ids + i * K;
  float* mass_out = out.mass + i * K;
  double h_fix = 0.0;  // sum p log p of ids listed more than once, instead of their entries' own
  for (int j = lane; j < K; j += 32) {
    const int id = sid[j];
    int place = 0, same = 0;
    float m = 0.f;
    bool first = true;
    for (int q = 0; q < K; ++q) {
      const int o = sid[q];
      place += (o < id || (o == id && q < j)) ? 1 : 0;
      if (o == id) {
        m += sp[q];
        ++same;
        if (q < j) first = false;
      }
    }
    if (same > 1 && id != INT_MAX) {
      if (sp[j] > 0.f) h_fix -= static_cast<double>(sp[j]) * log(static_cast<double>(sp[j]));
      if (first && m > 0.f) h_fix += static_cast<double>(m) * log(static_cast<double>(m));
    }
    ids_out[place] = live ? id : INT_MAX;
    mass_out[place] = live && id != INT_MAX ? m : 0.f;
  }
  const double h = warp_sum(own_h + h_fix);
  P = warp_sum(P);
  if (lane == 0) {
    out.stat[i] = make_double2(bad ? static_cast<double>(__int_as_float(0x7fc00000)) : h, P);
    out.mark[i] = live ? V : -1;
  }
}

// Rows of a launch: row0 + j, or ri[j] where ri is given.
//   part [S][stride]: the forward's (max x log2 e, sum) over the columns that
//   are not listed.  Writes kl, lse, the coefficients of the backward
//   (out.lse_rest, out.coef, out.val) and the block's sums of -w kl and of
//   the counted rows.  skipped: the rows without loss were not computed.
template <bool kLong>
__global__ void __launch_bounds__(SMALL_THREADS)
    topk_row_kernel(const float2* __restrict__ part, int S, int stride, int row0, int rows, const int* __restrict__ ri,
                    int K, int tail, const float* __restrict__ weights, const TopkRows out, int tf_softcap,
                    float tf_a, float tf_b, float tf_d, int skipped, float* __restrict__ out_kl,
                    float* __restrict__ out_lse, double* __restrict__ blk_sum, long long* __restrict__ blk_cnt) {
  using idx_t = typename std::conditional<kLong, long long, int>::type;
  const int lane = threadIdx.x & 31;
  const int j0 = blockIdx.x * TOPK_ROWS + (threadIdx.x >> 5);
  double contrib = 0.0;
  long long cnt = 0;
  if (j0 < rows) {
    const long long i = ri ? ri[j0] : row0 + j0;
    const bool live = out.mark[i] >= 0;
    const int* ids = out.ids + i * K;
    const float* mass = out.mass + i * K;
    float* val = out.val + i * K;
    if (!live && skipped) {
      if (lane == 0) {
        if (out_kl) out_kl[i] = 0.f;
        if (out_lse) out_lse[i] = __int_as_float(0x7fc00000);
        out.lse_rest[i] = __int_as_float(0x7fc00000);
        out.coef[i] = 0.f;
      }
    } else {
      // the columns that are not listed
      float m2 = -INFINITY;
      for (int s = lane; s < S; s += 32) m2 = fmaxf(m2, part[static_cast<idx_t>(s) * stride + static_cast<idx_t>(i)].x);
      m2 = warp_max(m2);
      double rest = 0.0;
      if (m2 > -INFINITY)
        for (int s = lane; s < S; s += 32) {
          const float2 q = part[static_cast<idx_t>(s) * stride + static_cast<idx_t>(i)];
          rest += q.y * exp2f(q.x - m2);
        }
      rest = warp_sum(rest);
      const double rest_top = static_cast<double>(m2) * 0.6931471805599453;  // natural log units
      // the listed ones, each id once
      float mk = -INFINITY;
      for (int j = lane; j < K; j += 32)
        if (ids[j] != INT_MAX) mk = fmaxf(mk, val[j]);
      mk = warp_max(mk);
      const double A = fmax(rest_top, static_cast<double>(mk));
      double listed = 0.0;
      for (int j = lane; j < K; j += 32)
        if (ids[j] != INT_MAX && (j == 0 || ids[j - 1] != ids[j]))
          listed += expf(static_cast<float>(static_cast<double>(val[j]) - A));
      listed = warp_sum(listed);
      const double rest_A = m2 > -INFINITY ? rest * static_cast<double>(expf(static_cast<float>(rest_top - A))) : 0.0;
      const double lse = A + log(rest_A + listed);
      const double lse_rest = rest > 0.0 ? rest_top + log(rest) : static_cast<double>(-INFINITY);
      const double R = rest > 0.0 ? rest_A / (rest_A + listed) : 0.0;
      const double2 st = out.stat[i];
      const double T = tail && rest > 0.0 ? fmax(0.0, 1.0 - st.y) : 0.0;
      const double M = st.y + T;
      const float w = weights ? weights[i] : 1.f;
      double cross = 0.0;
      for (int j = lane; j < K; j += 32) {
        const int id = ids[j];
        if (id == INT_MAX) continue;
        const float u = val[j], p = mass[j];
        const double lq = static_cast<double>(u) - lse;
        if (p > 0.f && (j == 0 || ids[j - 1] != id)) cross += p * lq;
        const float fd = tf_softcap ? tf_d * (1.f - (u / tf_b) * (u / tf_b)) : tf_a;
        val[j] = w * static_cast<float>(M * expf(static_cast<float>(lq)) - p) * fd;
      }
      cross = warp_sum(cross);
      if (lane == 0) {
        double kl = st.x - cross;
        if (T > 0.0) kl += T * (log(T) - (lse_rest - lse));
        const float klf = live ? static_cast<float>(kl) : 0.f;
        if (out_kl) out_kl[i] = klf;
        if (out_lse) out_lse[i] = static_cast<float>(lse);
        out.lse_rest[i] = static_cast<float>(lse_rest);
        out.coef[i] = live ? w * static_cast<float>(M * R - T) : 0.f;
        if (live) {
          cnt = 1;
          contrib = -static_cast<double>(w) * kl;  // the final kernel negates the sum
        }
      }
    }
  }
  block_sum_store(contrib, cnt, blk_sum, blk_cnt);
}

// The listed columns of a dlogits block: D[r][id - v0] = val * scale, bf16,
// for the ids inside [v0, v0 + width).  Local row r is row row0 + r, or
// ri[first + r]; rows past the device-side count are left alone.
template <bool kLong>
__global__ void topk_scatter_kernel(uint16_t* __restrict__ D, int ldD, int v0, int width, int row0, int rows,
                                    const int* __restrict__ ri, const int* __restrict__ dyn_count, int first, int K,
                                    const int* __restrict__ ids, const float* __restrict__ val, float grad_scale,
                                    const long long* __restrict__ count, const int* __restrict__ count32,
                                    const float* __restrict__ scale_dev) {
  using idx_t = typename std::conditional<kLong, long long, int>::type;
  if (dyn_count != nullptr) rows = max(0, min(*dyn_count - first, rows));
  float g = grad_scale;
  if (count != nullptr) g *= 1.f / fmaxf(1.f, static_cast<float>(*count));
  if (count32 != nullptr) g /= fmaxf(1.f, static_cast<float>(*count32));
  if (scale_dev != nullptr) g *= *scale_dev;
  const long long total = static_cast<long long>(rows) * K;
  for (long long e = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; e < total;
       e += static_cast<long long>(gridDim.x) * blockDim.x) {
    const int r = static_cast<int>(e / K);
    const int j = static_cast<int>(e - static_cast<long long>(r) * K);
    const long long i = ri ? ri[first + r] : row0 + r;
    const int id = ids[i * K + j];
    if (id < v0 || id - v0 >= width) continue;
    D[static_cast<idx_t>(r) * ldD + (id - v0)] = static_cast<uint16_t>(pack_bf16x2(val[i * K + j] * g, 0.f) & 0xffffu);
  }
}

}  // namespace flce
