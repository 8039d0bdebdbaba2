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
// by it is needed.  All in fp32 (64-bit arithmetic took 10 us of latency per
// row): every term of kl is small where the two distributions are near, and
// logits are taken relative to the row's largest.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <climits>
#include <cstdint>

#include "norm.cuh"
#include "small_kernels.cuh"

namespace flce {

constexpr int TOPK_WARPS = 4;      // rows per CTA of the list kernel, one warp each
constexpr int TOPK_MAX_K = 1024;   // longest list (its shared memory: 8 bytes per entry and row)
constexpr int TOPK_ROWS = SMALL_THREADS / 32;  // rows per CTA of the row kernel

// ln 2 - kLn2
constexpr float kLn2Low = static_cast<float>(0.69314718055994530942 - static_cast<double>(kLn2));

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
  float2* stat;      // [N] P (NaN: an id outside the vocabulary), T = max(0, 1 - P)
  long long* mark;   // [N] V for a counted row, -1 for one without loss
  float* lse_rest;   // [N]
  float* coef;       // [N] w (M R - T)
};

// These kernels are launched with programmatic stream serialisation: their
// launch overlaps the kernel before, and the next one's overlaps theirs.
// Nothing is read before the wait, and what the kernel before writes is read
// through plain pointers (a read-only load may be moved above the wait).  The
// next kernel is let in only after the wait, so all but this one have ended
// when it starts.  One-call step: 256 x 2,048 x 248,320 682 -> 674 us, 1,501 x
// 1,096 x 32,003 312 -> 301, 600 x 2,048 x 50,000 341 -> 333 (with the row
// kernel letting the dlogits in early as well 679, 307 and 336).
__device__ __forceinline__ void dependent_start() {
  grid_dependency_wait();
  grid_launch_dependents();
}

__device__ __forceinline__ float warp_sum(float x) {
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

// x + y as a rounded sum and what the rounding left out.
__device__ __forceinline__ float2 two_sum(float x, float y) {
  const float s = x + y, b = s - x;
  return make_float2(s, (x - (s - b)) + (y - b));
}

// The row's list in ascending order of id with the teacher's masses and their
// logarithms (one warp per row).  An entry's place is the number of entries
// before it (by id, then by position), counted in one walk over the list that
// also adds up the mass of equal ids: K^2 / 32 comparisons of a lane, four of
// its entries against four of the list per shared-memory read, no barrier.
// t - lse carries what its rounding leaves out; with the tail the masses and
// their sum are taken in 64 bits, since T = 1 - P is small where they are not.
__global__ void __launch_bounds__(32 * TOPK_WARPS)
    topk_list_kernel(const TopkTeacher t, const int64_t* targets, long long ignore, int N, int V,
                     const TopkRows out) {
  dependent_start();
  extern __shared__ __align__(16) int topk_smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int K = t.k, Kp = (K + 3) & ~3;  // (the last few of Kp: no entries)
  const long long i = static_cast<long long>(blockIdx.x) * TOPK_WARPS + warp;
  if (i >= N) return;
  int* sid = topk_smem + warp * 2 * Kp;
  float* sp = reinterpret_cast<float*>(sid + Kp);
  if (lane < Kp - K) {
    sid[K + lane] = INT_MAX;
    sp[K + lane] = 0.f;
  }
  bool any = false, bad = false, nan = false;
  float top = -INFINITY;
  for (int j0 = lane; j0 < K; j0 += 128) {
    // four entries' ids and logits at once: one latency of memory, not eight
    long long id[4];
    float u[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int j = j0 + 32 * e;
      id[e] = -1;
      u[e] = -INFINITY;
      if (j < K) {
        id[e] = t.ids_type == 4 ? static_cast<const int64_t*>(t.ids)[i * t.ld_ids + j]
                                : static_cast<const int32_t*>(t.ids)[i * t.ld_ids + j];
        u[e] = topk_logit(t, i, j);
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int j = j0 + 32 * e;
      if (j >= K) break;
      const bool in = id[e] >= 0 && id[e] < V;
      bad |= id[e] >= V;
      any |= in;
      const float x = in ? u[e] : -INFINITY;
      nan |= x != x;  // (the maximum passes over it)
      sid[j] = in ? static_cast<int>(id[e]) : INT_MAX;
      sp[j] = x;
      top = fmaxf(top, x);
    }
  }
  any = __any_sync(0xffffffffu, any);
  bad = __any_sync(0xffffffffu, bad);
  nan = __any_sync(0xffffffffu, nan);
  top = warp_max(top);
  bool live = any || bad;
  // log p = (u - ref) - logsum: ref the teacher's log-sum-exp, or the list's
  // largest logit and the logarithm of its exponentials' sum beside it
  float ref = top, logsum = 0.f;
  if (t.lse != nullptr) {
    ref = t.lse[i];
  } else {
    // a list without mass sums to nothing; beside an id outside the vocabulary
    // its entries have mass 0
    const bool none = top == -INFINITY;
    live = live && (!none || bad || nan);
    ref = none ? 0.f : top;
    float s = 0.f;
    for (int j = lane; j < K; j += 32) s += expf(sp[j] - ref);
    logsum = none && !nan ? 0.f : logf(warp_sum(s));
  }
  live = live && (targets == nullptr || targets[i] != ignore);
  double P = 0.0;
  for (int j = lane; j < K; j += 32) {
    float p = 0.f;
    if (sid[j] != INT_MAX) {
      if (t.tail) {
        const double pd = exp(static_cast<double>(sp[j]) - static_cast<double>(ref));
        P += pd;
        p = static_cast<float>(pd);
      } else {
        const float2 d = two_sum(sp[j], -ref), e = two_sum(d.x, -logsum);
        // (infinities and NaN make no rest of their own)
        p = expf(e.x) * (1.f + (e.x - e.x == 0.f ? d.y + e.y : 0.f));
        P += p;
      }
    }
    sp[j] = p;
  }
  __syncwarp();
  int* ids_out = out.ids + i * K;
  float* mass_out = out.mass + i * K;
  for (int j0 = lane; j0 < K; j0 += 128) {
    int id[4], place[4] = {0, 0, 0, 0};
    float m[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int e = 0; e < 4; ++e) id[e] = j0 + 32 * e < K ? sid[j0 + 32 * e] : INT_MAX;
    for (int q = 0; q < K; q += 4) {
      const int4 o4 = *reinterpret_cast<const int4*>(sid + q);
      const float4 p4 = *reinterpret_cast<const float4*>(sp + q);
      const int o[4] = {o4.x, o4.y, o4.z, o4.w};
      const float p[4] = {p4.x, p4.y, p4.z, p4.w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int f = 0; f < 4; ++f) {
          place[e] += (o[f] < id[e] || (o[f] == id[e] && q + f < j0 + 32 * e)) ? 1 : 0;
          m[e] += o[f] == id[e] ? p[f] : 0.f;
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (j0 + 32 * e < K) {
        ids_out[place[e]] = live ? id[e] : INT_MAX;
        mass_out[place[e]] = live && id[e] != INT_MAX ? m[e] : 0.f;
      }
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) P += __shfl_xor_sync(0xffffffffu, P, off);
  if (lane == 0) {
    out.stat[i] = make_float2(bad ? __int_as_float(0x7fc00000) : static_cast<float>(P),
                              static_cast<float>(fmax(0.0, 1.0 - P)));
    out.mark[i] = live ? V : -1;
  }
}

// The forward of a few rows (at most TOPK_GEMV_ROWS): with so few, a 256-row
// tensor-core tile is nearly empty and the work is reading W once, so warps
// read it straight into fp32 multiply-adds.  A warp takes 4 vocabulary rows at
// a time (a row of h, in shared memory as fp32, is read once for the four) and
// 8 elements of each per lane and step; after the warp's sums, lane 4 r + c
// keeps row r's online maximum and sum over the c-th of the 4, and walks r's
// list, whose ids ascend with the warp's vocabulary rows.  One partial per CTA
// and row.
// Bound by the read of W: 151,936 x 4,096 takes 179, 185 and 217 us for 1, 2
// and 4 rows (7.0, 6.7 and 5.7 TB/s), where the tiled forward took 279, 260
// and 230 (few rows of h are few lines of L2, which every SM then asks for at
// once; 16 rows take it 194).  Two CTAs to an SM with 8 loads of 16 bytes in
// flight per lane; 4 loads and 2 CTAs 207 us, 4 loads and 4 CTAs 184.
constexpr int TOPK_GEMV_ROWS = 4;
constexpr int TOPK_GEMV_WARPS = 8;
constexpr int TOPK_GEMV_CTAS = 2;

__device__ __forceinline__ uint4 ld_stream(const uint16_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

template <int NR>
__global__ void __launch_bounds__(32 * TOPK_GEMV_WARPS, TOPK_GEMV_CTAS)
    topk_gemv_kernel(const uint16_t* __restrict__ h, const uint16_t* __restrict__ W, int N, int H, int V, int K,
                     const TopkRows rows, int tf_softcap, float tf_a, float tf_b, float2* __restrict__ part) {
  dependent_start();
  extern __shared__ float4 gemv_h[];  // [NR][H / 4]
  __shared__ float2 merged[TOPK_GEMV_WARPS][32];
  float* hs = reinterpret_cast<float*>(gemv_h);
  for (int e = threadIdx.x; e < NR * (H / 2); e += blockDim.x) {
    const int r = e / (H / 2), c = (e - r * (H / 2)) * 2;
    const uint32_t u = r < N ? *reinterpret_cast<const uint32_t*>(h + static_cast<long long>(r) * H + c) : 0u;
    hs[r * H + c] = __uint_as_float(u << 16);
    hs[r * H + c + 1] = __uint_as_float(u & 0xffff0000u);
  }
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int my_r = lane >> 2, my_c = lane & 3;  // this lane's row and place among the 4
  const bool mine = my_r < NR && my_r < N;
  const int* ids = rows.ids + static_cast<long long>(mine ? my_r : 0) * K;
  float* val = rows.val + static_cast<long long>(mine ? my_r : 0) * K;
  int at = 0;
  float m = -INFINITY, s = 0.f;
  const int warps = gridDim.x * TOPK_GEMV_WARPS;
  const int groups = (V + 3) / 4;
  for (int g = blockIdx.x * TOPK_GEMV_WARPS + warp; g < groups; g += warps) {
    const int v0 = 4 * g;
    float2 acc[NR][4];  // even and odd elements
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[r][c] = make_float2(0.f, 0.f);
    const uint16_t* w[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) w[c] = W + static_cast<long long>(min(v0 + c, V - 1)) * H + lane * 8;
#pragma unroll 2
    for (int k = lane * 8; k < H; k += 256) {
      uint4 q[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        q[c] = ld_stream(w[c]);
        w[c] += 256;
      }
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        Raw8<float> x;
        x.load(hs + r * H + k);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint32_t u[4] = {q[c].x, q[c].y, q[c].z, q[c].w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            acc[r][c] = fma2(make_float2(__uint_as_float(u[e] << 16), __uint_as_float(u[e] & 0xffff0000u)),
                             x.pair(e), acc[r][c]);
        }
      }
    }
    float z = 0.f;
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float a = acc[r][c].x + acc[r][c].y;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) a += __shfl_xor_sync(0xffffffffu, a, off);
        if (lane == 4 * r + c) z = a;
      }
    const int v = v0 + my_c;
    if (mine && v < V) {
      const float u = tf_softcap ? tf_b * tanhf(tf_a * z) : tf_a * z;
      while (at < K && ids[at] < v) ++at;
      if (at < K && ids[at] == v) {
        for (; at < K && ids[at] == v; ++at) val[at] = u;
      } else {
        const float u2 = u * kLog2e, nm = fmaxf(m, u2);
        if (u2 != -INFINITY) {  // (a NaN, which the maximum passes over, stays in the sum)
          s = s * exp2f(m - nm) + exp2f(u2 - nm);
          m = nm;
        }
      }
    }
  }
  merged[warp][lane] = make_float2(m, s);
  __syncthreads();
  if (warp == 0 && my_c == 0 && mine) {
    float M = -INFINITY, S = 0.f;
    for (int i = 0; i < TOPK_GEMV_WARPS; ++i)
      for (int c = 0; c < 4; ++c) M = fmaxf(M, merged[i][lane + c].x);
    const float base = M > -INFINITY ? M : 0.f;  // (sums without a maximum are 0 or NaN)
    for (int i = 0; i < TOPK_GEMV_WARPS; ++i)
      for (int c = 0; c < 4; ++c) S += merged[i][lane + c].y * exp2f(merged[i][lane + c].x - base);
    part[static_cast<long long>(blockIdx.x) * N + my_r] = make_float2(M, S);
  }
}

// Rows of a launch: row0 + j, or ri[j] where ri is given.
//   part [S][stride]: the forward's (max x log2 e, sum) over the columns that
//   are not listed.  Writes kl, lse, the coefficients of the backward
//   (out.lse_rest, out.coef, out.val) and the block's sums of -w kl and of
//   the counted rows.  skipped: the rows without loss were not computed.
template <bool kLong>
__global__ void __launch_bounds__(SMALL_THREADS)
    topk_row_kernel(const float2* part, int S, int stride, int row0, int rows, const int* ri, int K, int tail,
                    const float* weights, const TopkRows out, int tf_softcap, float tf_a, float tf_b, float tf_d,
                    int skipped, float* out_kl, float* out_lse, double* blk_sum, long long* blk_cnt) {
  grid_dependency_wait();  // (not dependent_start: dlogits CTAs that wait on the SMs cost more than they save)
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
    // four partials and four entries of each lane in registers, all read at
    // once: a row's time is the latency of its loads, one after another
    float2 pr[4];
    int idr[4];
    bool newr[4];
    float ur[4], pm[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int s = lane + 32 * e, j = lane + 32 * e;
      pr[e] = s < S ? part[static_cast<idx_t>(s) * stride + static_cast<idx_t>(i)] : make_float2(-INFINITY, 0.f);
      idr[e] = j < K ? ids[j] : INT_MAX;
      newr[e] = j < K && (j == 0 || ids[j - 1] != idr[e]);
      ur[e] = j < K ? val[j] : 0.f;
      pm[e] = j < K ? mass[j] : 0.f;
    }
    // f(position, id's first entry, u, mass) for this lane's entries
    auto entries = [&](auto&& f) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (idr[e] != INT_MAX) f(lane + 32 * e, newr[e], ur[e], pm[e]);
      for (int j = lane + 128; j < K; j += 32)
        if (ids[j] != INT_MAX) f(j, ids[j - 1] != ids[j], val[j], mass[j]);
    };
    if (!live && skipped) {
      if (lane == 0) {
        if (out_kl) out_kl[i] = 0.f;
        if (out_lse) out_lse[i] = __int_as_float(0x7fc00000);
        out.lse_rest[i] = __int_as_float(0x7fc00000);
        out.coef[i] = 0.f;
      }
    } else {
      // the columns that are not listed: log2 maximum m2 and sum of 2^(. - m2)
      float m2 = -INFINITY;
#pragma unroll
      for (int e = 0; e < 4; ++e) m2 = fmaxf(m2, pr[e].x);
      for (int s = lane + 128; s < S; s += 32)
        m2 = fmaxf(m2, part[static_cast<idx_t>(s) * stride + static_cast<idx_t>(i)].x);
      m2 = warp_max(m2);
      // (a partial without a maximum is 0 or, of logits that are no numbers, NaN)
      const float base2 = m2 > -INFINITY ? m2 : 0.f;
      float rest = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) rest += pr[e].y * exp2f(pr[e].x - base2);
      for (int s = lane + 128; s < S; s += 32) {
        const float2 q = part[static_cast<idx_t>(s) * stride + static_cast<idx_t>(i)];
        rest += q.y * exp2f(q.x - base2);
      }
      rest = warp_sum(rest);
      // the listed ones, each id once, relative to the larger of the two maxima
      float mk = -INFINITY;
      entries([&](int, bool, float u, float) { mk = fmaxf(mk, u); });
      mk = warp_max(mk);
      // m2 ln 2 as a rounded product and its rest (ln 2 in two parts)
      const float2 rt = m2 > -INFINITY ? make_float2(m2 * kLn2, fmaf(m2, kLn2, -(m2 * kLn2)) + m2 * kLn2Low)
                                       : make_float2(-INFINITY, 0.f);
      const float A = fmaxf(rt.x, mk);
      float listed = 0.f;
      entries([&](int, bool first, float u, float) {
        if (first) listed += expf(u - A);
      });
      listed = warp_sum(listed);
      // (no rest: exactly 0; a NaN goes on into lse and kl)
      const float rest_A = rest != 0.f ? rest * expf((rt.x - A) + rt.y) : 0.f;
      const float total = rest_A + listed;
      const float logtot = logf(total);
      const float log_rest = ((rt.x - A) + rt.y) + logf(rest);  // relative to A; -inf where there is no rest
      const float R = rest != 0.f ? rest_A / total : 0.f;
      const float2 st = out.stat[i];  // P (NaN: an id outside the vocabulary), T
      const float T = tail && rest != 0.f ? st.y : 0.f;
      const float w = weights ? weights[i] : 1.f;
      // P for the gradients: a bad id takes no part in them
      float P = st.x;
      if (P != P) {
        P = 0.f;
        entries([&](int, bool first, float, float p) {
          if (first) P += p;
        });
        P = warp_sum(P);
      }
      const float M = P + T;
      float kl = 0.f;
      entries([&](int j, bool first, float u, float p) {
        const float lq = (u - A) - logtot;
        if (p > 0.f && first) kl = fmaf(p, logf(p) - lq, kl);
        const float fd = tf_softcap ? tf_d * (1.f - (u / tf_b) * (u / tf_b)) : tf_a;
        val[j] = w * fmaf(M, expf(lq), -p) * fd;
      });
      kl = warp_sum(kl);
      if (lane == 0) {
        if (T > 0.f) kl += T * (logf(T) - (log_rest - logtot));
        if (st.x != st.x) kl = st.x;
        if (out_kl) out_kl[i] = live ? kl : 0.f;
        if (out_lse) out_lse[i] = A + logtot;
        out.lse_rest[i] = A + log_rest;
        out.coef[i] = live ? w * fmaf(M, R, -T) : 0.f;
        if (live) {
          cnt = 1;
          contrib = -static_cast<double>(w) * static_cast<double>(kl);  // the final kernel negates the sum
        }
      }
    }
  }
  block_sum_store(contrib, cnt, blk_sum, blk_cnt);
}

// dlogits of one row block of the one-call step, in place: the forward's
// fp16 exponentials E = 2^(u log2 e - chunk max) kExpScale (0 in the listed columns and
// past the vocabulary) become the bf16
//   D = E / kExpScale 2^(chunk max - lse_rest) coef g f'(z),  g = grad_scale / max(n_valid, 1)
// (split: g's power of two),
// then the listed columns get theirs.  A CTA takes `steps` runs of
// TOPK_DL_COLS columns of a row (blockIdx.y), a lane 8 neighbouring columns at
// a time, so that a warp's 16-byte accesses are contiguous.  Rows as
// fused_dlogits_kernel.  kLo: D in two parts, what the first one's rounding
// leaves out lo rows further on; the rows from `count` to lo are zeroed.
constexpr int TOPK_DL_COLS = SMALL_THREADS * 32;

// What the bf16 pair w = (x, y) leaves out of x and y, as a bf16 pair
// (nothing of values that are not finite).
__device__ __forceinline__ uint32_t bf16x2_rest(float x, float y, uint32_t w) {
  const float rx = x - __uint_as_float(w << 16), ry = y - __uint_as_float(w & 0xffff0000u);
  return pack_bf16x2(rx - rx == 0.f ? rx : 0.f, ry - ry == 0.f ? ry : 0.f);
}

template <bool kLong, bool kLo>
__global__ void __launch_bounds__(SMALL_THREADS)
    topk_dlogits_kernel(uint16_t* __restrict__ E, const float* __restrict__ mx, int ldD, int ld_mx, int steps, int row0,
                        int count, int lo, const int* __restrict__ ri, const TopkRows rows, int K, const int* __restrict__ n_valid,
                        float grad_scale, int split, int tf_softcap, float tf_a, float tf_b, float tf_d) {
  dependent_start();
  using idx_t = typename std::conditional<kLong, long long, int>::type;
  const int r = blockIdx.y;
  const int n = *n_valid;
  if (ri != nullptr && r >= (n - row0 + 63) / 64 * 64) return;  // row0: the block's first position
  const bool inside = !kLo || r < count;
  const long long i = !inside ? 0 : ri ? ri[r] : row0 + r;
  const float g = split ? split_scale(grad_scale, n_valid).pow2 : grad_scale / fmaxf(1.f, static_cast<float>(n));
  const bool live = inside && rows.mark[i] >= 0;
  const float scale = live ? rows.coef[i] * g : 0.f;
  uint16_t* row = E + static_cast<idx_t>(r) * ldD;
  uint16_t* row2 = row + static_cast<idx_t>(lo) * ldD;
  const float* rmx = mx + static_cast<idx_t>(r) * ld_mx;
  const int c0 = blockIdx.x * steps * TOPK_DL_COLS;
  const int c1 = min(ldD, c0 + steps * TOPK_DL_COLS);
  const int first = c0 + (threadIdx.x >> 5) * 1024 + (threadIdx.x & 31) * 8;
  if (scale == 0.f) {  // a row without loss or weight, whose exponentials may never have been written
    for (int c = c0 + threadIdx.x * 8; c < c1; c += SMALL_THREADS * 8) {
      *reinterpret_cast<uint4*>(row + c) = make_uint4(0u, 0u, 0u, 0u);
      if constexpr (kLo) *reinterpret_cast<uint4*>(row2 + c) = make_uint4(0u, 0u, 0u, 0u);
    }
  } else {
    const float nlse2 = -rows.lse_rest[i] * kLog2e;
    for (int cs = first; cs < c1; cs += TOPK_DL_COLS) {
      uint4 q[4];
      float cm[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int c = cs + k * 256;
        if (c < c1) {
          q[k] = *reinterpret_cast<const uint4*>(row + c);
          cm[k] = rmx[c / 32];
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int c = cs + k * 256;
        if (c >= c1) continue;
        uint32_t w[4] = {q[k].x, q[k].y, q[k].z, q[k].w};
        uint32_t w2[4];
        const float kf = ex2_approx(cm[k] + nlse2) * scale * (1.f / kExpScale);
        if (!tf_softcap) {
          const float2 f = both(kf * tf_a);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 d = mul2(__half22float2(*reinterpret_cast<const __half2*>(&w[e])), f);
            w[e] = pack_bf16x2(d.x, d.y);
            if constexpr (kLo) w2[e] = bf16x2_rest(d.x, d.y, w[e]);
          }
        } else {  // u = ln(E) + chunk max, tanh(a z) = u / b
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 ev = __half22float2(*reinterpret_cast<const __half2*>(&w[e]));
            const float el = ev.x, eh = ev.y;
            const float ul = (__log2f(el * (1.f / kExpScale)) + cm[k]) * kLn2 / tf_b;
            const float uh = (__log2f(eh * (1.f / kExpScale)) + cm[k]) * kLn2 / tf_b;
            const float dl = el > 0.f ? el * kf * tf_d * (1.f - ul * ul) : 0.f;
            const float dh = eh > 0.f ? eh * kf * tf_d * (1.f - uh * uh) : 0.f;
            w[e] = pack_bf16x2(dl, dh);
            if constexpr (kLo) w2[e] = bf16x2_rest(dl, dh, w[e]);
          }
        }
        *reinterpret_cast<uint4*>(row + c) = make_uint4(w[0], w[1], w[2], w[3]);
        if constexpr (kLo) *reinterpret_cast<uint4*>(row2 + c) = make_uint4(w2[0], w2[1], w2[2], w2[3]);
      }
    }
  }
  if (!live) return;  // (the whole CTA)
  __syncthreads();  // the listed columns after the CTA's own stores
  for (int j = threadIdx.x; j < K; j += SMALL_THREADS) {
    const int id = rows.ids[i * K + j];
    if (id >= c0 && id < c1 && id != INT_MAX) {
      const float d = rows.val[i * K + j] * g;
      const uint32_t w = pack_bf16x2(d, 0.f);
      row[id] = static_cast<uint16_t>(w & 0xffffu);
      if constexpr (kLo) row2[id] = static_cast<uint16_t>(bf16x2_rest(d, 0.f, w) & 0xffffu);
    }
  }
}

// The counted rows of up to TOPK_INDEX_ROWS rows in one CTA: their number,
// and (idx given) a permutation with them first, each part in row order.
constexpr int TOPK_INDEX_ROWS = 32768;
__global__ void __launch_bounds__(1024)
    topk_index_kernel(const long long* mark, int N, int* __restrict__ idx, int* __restrict__ total) {
  dependent_start();
  __shared__ int wsum[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int live = 0;  // of all rows
  for (int i = threadIdx.x; i < N; i += 1024) live += mark[i] >= 0 ? 1 : 0;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) live += __shfl_xor_sync(0xffffffffu, live, off);
  if (lane == 0) wsum[warp] = live;
  __syncthreads();
  int all = 0;
  for (int w = 0; w < 32; ++w) all += wsum[w];
  if (threadIdx.x == 0) *total = all;
  if (idx == nullptr) return;
  int before = 0;  // counted rows of the tiles before this one
  for (int t0 = 0; t0 < N; t0 += 1024) {
    const int i = t0 + threadIdx.x;
    const bool keep = i < N && mark[i] >= 0;
    const unsigned ballot = __ballot_sync(0xffffffffu, keep);
    __syncthreads();  // the last tile's sums have been read
    if (lane == 0) wsum[warp] = __popc(ballot);
    __syncthreads();
    int pos = before + __popc(ballot & ((1u << lane) - 1u)), tile = 0;
    for (int w = 0; w < 32; ++w) {
      if (w < warp) pos += wsum[w];
      tile += wsum[w];
    }
    if (keep)
      idx[pos] = i;
    else if (i < N)
      idx[all + i - pos] = i;
    before += tile;
  }
}

}  // namespace flce
