// libflce: the row kernels of the scores -- log-probability and entropy of the
// head's distribution, and its K likeliest words.
//
// With u_v = f(z_v), z = h W^T, per row:
//   lse = log sum_v e^u_v,  logp = u_t - lse
//   entropy = lse - sum_v p_v u_v = log S + C / S,
//     S = sum_v e^(u_v - m),  C = sum_v e^(u_v - m) (m - u_v)   (any m)
//   the K words with the largest z (f increases), ties to the lowest index
// The forward GEMM leaves a partial (m, S, C) per row and vocabulary split and,
// for the words, the two largest z of every 32-column chunk (gemm.cuh,
// score_key).
//
// The words' order.  The tensor cores' fp32 sums are off by some 1e-6 of the
// logits' size, and among the best of 151,936 logits neighbours are often nearer
// than that.  So the GEMM's z only names the candidates -- every word that its z
// leaves in the running, given how far z can be off -- and their products are
// summed again to 2^-45 or so (exact bf16 products, two fp32 sums), which then
// orders them.  The K words are those of the exact logits, whatever order the
// tensor cores add in.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "small_kernels.cuh"
#include "topk.cuh"

namespace flce {

constexpr int SCORE_MAX_K = 128;

// A partial of a row over some of its columns: m, S, C in units of log2, and a
// magnitude of its logits (the forward: the largest of every eighth).
struct ScorePart {
  float m, s, c, top;
};

// b's columns joined to a's.
__device__ __forceinline__ ScorePart score_join(const ScorePart& a, const ScorePart& b) {
  ScorePart o;
  o.m = fmaxf(a.m, b.m);
  o.top = fmaxf(a.top, b.top);
  // (a part without a maximum is empty, or NaN)
  const float da = a.m != -INFINITY ? o.m - a.m : 0.f, db = b.m != -INFINITY ? o.m - b.m : 0.f;
  const float fa = ex2_approx(-da), fb = ex2_approx(-db);
  o.s = fmaf(a.s, fa, b.s * fb);
  o.c = fmaf(fmaf(da, a.s, a.c), fa, fmaf(db, b.s, b.c) * fb);
  return o;
}

// A row's S partials joined by a warp, in a fixed order; the same in all lanes.
__device__ __forceinline__ ScorePart score_join_row(const float4* part, int S, int lane) {
  ScorePart a{-INFINITY, 0.f, 0.f, 0.f};
  for (int s = lane; s < S; s += 32) {
    const float4 q = part[s];
    a = score_join(a, ScorePart{q.x, q.y, q.z, q.w});
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    const ScorePart b{__shfl_xor_sync(0xffffffffu, a.m, off), __shfl_xor_sync(0xffffffffu, a.s, off),
                      __shfl_xor_sync(0xffffffffu, a.c, off), __shfl_xor_sync(0xffffffffu, a.top, off)};
    // (the lower lane's first, in both)
    a = (lane & off) ? score_join(b, a) : score_join(a, b);
  }
  return a;
}

// (lse, entropy); NaN where the row has a logit that is NaN or +infinity (with a
// soft-cap, any infinity), or none above -infinity.
__device__ __forceinline__ float2 score_of(const ScorePart& a) {
  const float nan = __int_as_float(0x7fc00000);
  if (!(a.s > 0.f) || !(fabsf(a.m) < INFINITY)) return make_float2(nan, nan);
  const float l2 = log2f(a.s);
  // m ln 2 + log S with ln 2 in two parts
  const float lse = fmaf(a.m, kLn2, fmaf(a.m, kLn2Low, l2 * kLn2));
  return make_float2(lse, fmaxf(0.f, (l2 + a.c / a.s) * kLn2));
}

struct ScoreOut {
  float* logp;     // [N], each may be null
  float* lse;
  float* entropy;
  int64_t* ids;    // [N][k]
  float* words;    // [N][k]
  int k;
};

// The outputs of a row without a result: 0 (a row that is skipped) or NaN, and
// no words.
__device__ __forceinline__ void score_no_row(const ScoreOut& o, long long i, float value, int t, int threads) {
  if (t == 0) {
    if (o.logp) o.logp[i] = value;
    if (o.lse) o.lse[i] = value;
    if (o.entropy) o.entropy[i] = value;
  }
  for (int j = t; j < o.k; j += threads) {
    if (o.ids) o.ids[i * o.k + j] = -1;
    if (o.words) o.words[i * o.k + j] = value;
  }
}

// Rows of one launch: row j of the pass is row0 + j, or with ri (the counted
// rows, *count of them) ri[first + j].
struct ScoreRows {
  int row0, rows;
  const int* ri;
  const int* count;
  int first;
  __device__ __forceinline__ long long at(int j) const {
    if (ri == nullptr) return j < rows ? row0 + j : -1;
    return j < rows && first + j < *count ? ri[first + j] : -1;
  }
};

// The rows that a skipping forward leaves out.
__global__ void __launch_bounds__(SMALL_THREADS)
    score_skipped_kernel(const int64_t* __restrict__ targets, long long ignore, int N, const ScoreOut out) {
  const int warps = gridDim.x * (SMALL_THREADS / 32);
  for (int i = blockIdx.x * (SMALL_THREADS / 32) + (threadIdx.x >> 5); i < N; i += warps)
    if (targets[i] == ignore) score_no_row(out, i, 0.f, threadIdx.x & 31, 32);
}

// lse, entropy and logp of the pass's rows, a warp to each.
template <bool kLong>
__global__ void __launch_bounds__(SMALL_THREADS)
    score_row_kernel(const float4* part, int S, const ScoreRows rows, const float* zt, const int64_t* targets,
                     long long ignore, int V, const ScoreOut out) {
  dependent_start();
  using idx_t = typename std::conditional<kLong, long long, int>::type;
  const int j = blockIdx.x * (SMALL_THREADS / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const long long i = rows.at(j);
  if (i < 0) return;
  const long long t = targets != nullptr ? targets[i] : -1;
  if (targets != nullptr && t == ignore) {
    score_no_row(out, i, 0.f, lane, 32);
    return;
  }
  const float2 r = score_of(score_join_row(part + static_cast<idx_t>(j) * S, S, lane));
  if (lane == 0) {
    if (out.lse) out.lse[i] = r.x;
    if (out.entropy) out.entropy[i] = r.y;
    // (a target outside the vocabulary has no logit)
    if (out.logp) out.logp[i] = t >= 0 && t < V ? zt[i] - r.x : __int_as_float(0x7fc00000);
  }
}

// x + y (two-part sums): the rounded sums' errors go to the low part.
__device__ __forceinline__ float2 two_add(float2 x, float2 y) {
  const float2 s = two_sum(x.x, y.x);
  return make_float2(s.x, s.y + (x.y + y.y));
}

// sum_k h_k w_k of two bf16 rows by a warp, as a rounded value and what the
// rounding leaves out: products of bf16 are exact in fp32, each step of the sum
// hands its rounding error to a second sum.  The same in all lanes.
__device__ __forceinline__ float2 exact_dot(const uint16_t* __restrict__ h, const uint16_t* __restrict__ w, int H,
                                            int lane) {
  float2 hi = both(0.f), lo = both(0.f);
  const float2 minus = both(-1.f);
#pragma unroll 2
  for (int k = lane * 8; k < H; k += 256) {
    Raw8<uint16_t> a, b;
    a.q[0] = __ldg(reinterpret_cast<const uint4*>(h + k));
    b.q[0] = __ldg(reinterpret_cast<const uint4*>(w + k));
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 p = mul2(a.pair(e), b.pair(e));
      const float2 s = add2(hi, p);
      const float2 y = fma2(hi, minus, s);                         // s - hi
      const float2 x = fma2(y, minus, s);                          // s - y
      lo = add2(lo, add2(fma2(x, minus, hi), fma2(y, minus, p)));  // (hi - x) + (p - y)
      hi = s;
    }
  }
  float2 d = two_add(make_float2(hi.x, lo.x), make_float2(hi.y, lo.y));
#pragma unroll
  for (int off = 16; off > 0; off >>= 1)
    d = two_add(d, make_float2(__shfl_xor_sync(0xffffffffu, d.x, off), __shfl_xor_sync(0xffffffffu, d.y, off)));
  // (a sum that is not finite has no rest; one that is NaN comes last)
  if (!(fabsf(d.x) < INFINITY)) return make_float2(d.x == INFINITY ? d.x : -INFINITY, 0.f);
  return two_sum(d.x, d.y);
}

// Whether word (a, i) comes before word (b, j): the larger logit, then the lower index.
__device__ __forceinline__ bool word_before(float2 a, int i, float2 b, int j) {
  if (a.x != b.x) return a.x > b.x;
  if (a.y != b.y) return a.y > b.y;
  return i < j;
}

struct SelectParams {
  const uint16_t* h;   // [N][H]
  const uint16_t* W;   // [V][H]
  const float4* part;  // [rows][S]
  const float2* rec;   // [rows][ld] chunk records, or
  const float* z;      // [rows][ld] logits
  int S, ld, H, V;
  ScoreRows rows;
  const int64_t* targets;
  long long ignore;
  float slack;         // how far a record can be off the logit, relative to the row's largest
  int tf_softcap;
  float tf_a, tf_b;
  ScoreOut out;
};

// The K likeliest words of a row on a CTA of T threads.
//   1. Each thread takes the largest of its records (kDense: of its logits); the
//      K-th largest of the threads' is a lower bound of the K-th largest logit,
//      close to it (K words on T threads seldom share one).
//   2. Candidates: the words that reach the bound, less what both can be off by.
//      Of a chunk whose second largest reaches it too, all 32.
//   3. Their logits again, a warp to a word, and a rank for each by counting.
// More candidates than the list holds (logits that are nearly all equal) go
// through it in runs, in index order, with the K best so far kept and the bound
// raised to theirs.
constexpr int SELECT_CAP = 1024;  // words of the list: more than SCORE_MAX_K and a chunk

template <int T, bool kDense, bool kLong>
__global__ void __launch_bounds__(T) score_select_kernel(const __grid_constant__ SelectParams p) {
  dependent_start();
  using idx_t = typename std::conditional<kLong, long long, int>::type;
  __shared__ float2 val[SELECT_CAP];
  __shared__ int word[SELECT_CAP];
  __shared__ __align__(16) float tops[T];
  __shared__ int sums[T / 32];
  __shared__ int found;
  __shared__ float bound;
  __shared__ float2 target_z;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int K = p.out.k;
  const int j = blockIdx.x;
  const long long i = p.rows.at(j);
  if (i < 0) return;
  const long long tgt = p.targets != nullptr ? p.targets[i] : -1;
  if (p.targets != nullptr && tgt == p.ignore) {
    score_no_row(p.out, i, 0.f, t, T);
    return;
  }
  const ScorePart whole = score_join_row(p.part + static_cast<idx_t>(j) * p.S, p.S, lane);
  const float2 r = score_of(whole);
  if (r.x != r.x) {  // (the same in every warp)
    score_no_row(p.out, i, r.x, t, T);
    return;
  }
  // a unit: a chunk and its record, or (kDense) a word and its logit
  const int units = kDense ? p.V : (p.V + 31) / 32;
  const idx_t base = static_cast<idx_t>(j) * p.ld;
  auto unit = [&](int c) {
    if constexpr (kDense) {
      const float z = p.z[base + c];
      return make_float2(z, z);
    } else {
      return p.rec[base + c];
    }
  };
  const uint16_t* h = p.h + i * p.H;
  float top = -INFINITY;
#pragma unroll 4
  for (int c = t; c < units; c += T) top = fmaxf(top, unit(c).x);
  tops[t] = top;
  if (t == 0) found = 0;
  const bool want_target = tgt >= 0 && tgt < p.V && p.out.logp != nullptr;
  if (want_target && warp == T / 32 - 1) {
    const float2 z = exact_dot(h, p.W + tgt * p.H, p.H, lane);
    if (lane == 0) target_z = z;
  }
  __syncthreads();
  int rank = 0;
  float most = -INFINITY;
  for (int q = 0; q < T; q += 4) {
    const float4 o = *reinterpret_cast<const float4*>(tops + q);
    rank += (o.x > top || (o.x == top && q < t)) + (o.y > top || (o.y == top && q + 1 < t)) +
            (o.z > top || (o.z == top && q + 2 < t)) + (o.w > top || (o.w == top && q + 3 < t));
    most = fmaxf(fmaxf(most, fmaxf(o.x, o.y)), fmaxf(o.z, o.w));
  }
  if (rank == K - 1) bound = top;
  __syncthreads();
  // (K threads with a record: K chunks; else every word is a candidate)
  const float low = bound;
  const float size = fmaxf(whole.top < INFINITY ? whole.top : 0.f, fmaxf(fabsf(most), low > -INFINITY ? fabsf(low) : 0.f));
  const float off = p.slack * size + 1e-43f;
  float reach = low - 2.f * off;
  // words of a unit that are still in the running
  auto words_of = [&](int c, float2 q) {
    if (!(q.x >= reach)) return 0;
    return !kDense && q.y >= reach ? min(32, p.V - 32 * c) : 1;
  };
  auto put = [&](int at, int c, float2 q, int n) {
    if constexpr (kDense) {
      word[at] = c;
    } else if (q.y >= reach) {
      for (int e = 0; e < n; ++e) word[at + e] = 32 * c + e;
    } else {
      word[at] = 32 * c + 31 - static_cast<int>(__float_as_uint(q.x) & 31u);
    }
  };
  // the logits of the words [from, total), then the best K of all in order at the list's front
  auto settle = [&](int from, int total) {
    for (int e = from + warp; e < total; e += T / 32) {
      const float2 z = exact_dot(h, p.W + static_cast<long long>(word[e]) * p.H, p.H, lane);
      if (lane == 0) val[e] = z;
    }
    __syncthreads();
    constexpr int PER = (SELECT_CAP + T - 1) / T;
    float2 v[PER];
    int w[PER], place[PER];
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      const int e = t + q * T;
      place[q] = K;
      if (e < total) {
        v[q] = val[e];
        w[q] = word[e];
        int before = 0;
        for (int o = 0; o < total; ++o) before += word_before(val[o], word[o], v[q], w[q]) ? 1 : 0;
        place[q] = before;
      }
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < PER; ++q)
      if (place[q] < K) {
        val[place[q]] = v[q];
        word[place[q]] = w[q];
      }
    __syncthreads();
  };
#pragma unroll 4
  for (int c = t; c < units; c += T) {
    const float2 q = unit(c);
    const int n = words_of(c, q);
    if (n > 0) {
      const int at = atomicAdd(&found, n);  // (the order within the list does not matter)
      if (at <= SELECT_CAP - n) put(at, c, q, n);
    }
  }
  __syncthreads();
  if (found <= SELECT_CAP) {
    settle(0, found);
  } else {
    // kept: words at the list's front that are settled; total: those in the list
    int kept = 0, total = 0;
    for (int c0 = 0; c0 < units;) {
      // the next T units, as many of them from the first as there is room for
      const int c = c0 + t;
      const float2 q = c < units ? unit(c) : make_float2(-INFINITY, -INFINITY);
      const int n = c < units ? words_of(c, q) : 0;
      int upto = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += x;
      }
      __syncthreads();  // found and the last run's sums have been read
      if (lane == 31) sums[warp] = upto;
      __syncthreads();
      for (int x = 0; x < warp; ++x) upto += sums[x];
      const bool fits = upto <= SELECT_CAP - total;
      if (fits && n > 0) put(total + upto - n, c, q, n);
      const int took = __syncthreads_count(fits);
      if (took > 0 && t == took - 1) found = upto;
      __syncthreads();
      if (took > 0) total += found;
      c0 += took;
      if (took < T || c0 >= units) {  // no room for the next unit (there is, once the list is settled), or the end
        settle(kept, total);
        kept = total = min(total, K);
        if (kept == K) reach = fmaxf(reach, val[K - 1].x - off);
      }
    }
  }
  // (the list holds K words at least: K chunks reach the bound, or there is none and all V do)
  for (int e = t; e <= K; e += T) {
    if (e == K && !want_target) break;
    const float z = e < K ? val[e].x : target_z.x;
    const float u = p.tf_softcap ? p.tf_b * tanhf(p.tf_a * z) : p.tf_a * z;
    if (e == K) {
      p.out.logp[i] = u - r.x;
    } else {
      if (p.out.ids) p.out.ids[i * K + e] = word[e];
      if (p.out.words) p.out.words[i * K + e] = u - r.x;
    }
  }
  if (t == 0) {
    if (p.out.lse) p.out.lse[i] = r.x;
    if (p.out.entropy) p.out.entropy[i] = r.y;
    if (p.out.logp && !want_target) p.out.logp[i] = __int_as_float(0x7fc00000);
  }
}

// Chunk records of N rows of logits (the few-row forward's), a warp to a chunk.
__global__ void __launch_bounds__(SMALL_THREADS)
    score_record_kernel(const float* z, int N, int V, int ldz, float2* rec, int ld) {
  dependent_start();
  const int chunks = (V + 31) / 32, lane = threadIdx.x & 31;
  const long long u = static_cast<long long>(blockIdx.x) * (SMALL_THREADS / 32) + (threadIdx.x >> 5);
  if (u >= static_cast<long long>(N) * chunks) return;
  const int r = static_cast<int>(u / chunks), c = static_cast<int>(u - static_cast<long long>(r) * chunks);
  const int v = 32 * c + lane;
  float m1 = v < V ? score_key(z[static_cast<long long>(r) * ldz + v], lane) : -INFINITY, m2 = -INFINITY;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    const float a = __shfl_xor_sync(0xffffffffu, m1, off), b = __shfl_xor_sync(0xffffffffu, m2, off);
    m2 = fmaxf(fmaxf(m2, b), fminf(m1, a));
    m1 = fmaxf(m1, a);
  }
  if (lane == 0) rec[static_cast<long long>(r) * ld + c] = make_float2(m1, m2);
}

// The forward of at most TOPK_GEMV_ROWS rows, as topk_gemv_kernel (a warp takes 4
// vocabulary rows at a time and sums them in fp32; lane 4 r + c keeps row r's
// partial over the c-th of the 4).  Writes the logits [N][ldz] where z is given,
// the target's transformed logit where zt is, and one partial per row and CTA
// ([N][gridDim.x]).
template <int NR>
__global__ void __launch_bounds__(32 * TOPK_GEMV_WARPS, TOPK_GEMV_CTAS)
    score_gemv_kernel(const uint16_t* __restrict__ h, const uint16_t* __restrict__ W, int N, int H, int V, float* z,
                      int ldz, const int64_t* targets, float* zt, int tf_softcap, float tf_a, float tf_b,
                      float4* __restrict__ part) {
  dependent_start();
  extern __shared__ float4 gemv_h[];  // [NR][H / 4]
  __shared__ ScorePart merged[TOPK_GEMV_WARPS][32];
  float* hs = reinterpret_cast<float*>(gemv_h);
  for (int e = threadIdx.x; e < NR * (H / 2); e += blockDim.x) {
    const int r = e / (H / 2), c = (e - r * (H / 2)) * 2;
    const uint32_t u = r < N ? *reinterpret_cast<const uint32_t*>(h + static_cast<long long>(r) * H + c) : 0u;
    hs[r * H + c] = __uint_as_float(u << 16);
    hs[r * H + c + 1] = __uint_as_float(u & 0xffff0000u);
  }
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int my_r = lane >> 2, my_c = lane & 3;
  const bool mine = my_r < NR && my_r < N;
  const long long tgt = mine && targets != nullptr && zt != nullptr ? targets[my_r] : -1;
  ScorePart a{-INFINITY, 0.f, 0.f, 0.f};
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
    float s = 0.f;
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float x = acc[r][c].x + acc[r][c].y;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
        if (lane == 4 * r + c) s = x;
      }
    const int v = v0 + my_c;
    if (mine && v < V) {
      if (z != nullptr) z[static_cast<long long>(my_r) * ldz + v] = s;
      const float u = tf_softcap ? fmaf(s, 0.f, tf_b * tanhf(tf_a * s)) : tf_a * s;
      if (v == tgt) zt[my_r] = u;
      const float u2 = u * kLog2e;
      const float top = fmaxf(a.top, fabsf(s));
      if (u2 != -INFINITY) a = score_join(a, ScorePart{u2, u2 != u2 ? u2 : 1.f, 0.f, 0.f});
      a.top = top;
    }
  }
  merged[warp][lane] = a;
  __syncthreads();
  if (warp == 0 && my_c == 0 && mine) {
    ScorePart o{-INFINITY, 0.f, 0.f, 0.f};
    for (int x = 0; x < TOPK_GEMV_WARPS; ++x)
      for (int c = 0; c < 4; ++c) o = score_join(o, merged[x][lane + c]);
    part[static_cast<long long>(my_r) * gridDim.x + blockIdx.x] = make_float4(o.m, o.s, o.c, o.top);
  }
}

}  // namespace flce
