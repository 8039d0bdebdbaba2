// libflce: the row kernels of the scores -- log-probability and entropy of the
// head's distribution, and its K likeliest words.
//
// With u_v = f(z_v), z = h W^T, per row:
//   lse = log sum_v e^u_v,  logp = u_t - lse
//   entropy = lse - sum_v p_v u_v = log S + C / S,
//     S = sum_v e^(u_v - m),  C = sum_v e^(u_v - m) (m - u_v)   (any m)
//   the K words with the largest z (f increases), ties to the lowest index
// The forward GEMM leaves a partial (m, S, C) per row and vocabulary split and,
// for the words, the three largest z of every 32-column chunk (gemm.cuh,
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

// A warp's partials joined, in a fixed order; the same in all lanes.
__device__ __forceinline__ ScorePart score_join_warp(ScorePart a, int lane) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    const ScorePart b{__shfl_xor_sync(0xffffffffu, a.m, off), __shfl_xor_sync(0xffffffffu, a.s, off),
                      __shfl_xor_sync(0xffffffffu, a.c, off), __shfl_xor_sync(0xffffffffu, a.top, off)};
    // (the lower lane's first, in both)
    a = (lane & off) ? score_join(b, a) : score_join(a, b);
  }
  return a;
}

// A row's S partials joined by a warp, in a fixed order; the same in all lanes.
// (Eight of a lane's are read at once: the joins wait on one another.)
__device__ __forceinline__ ScorePart score_join_row(const float4* part, int S, int lane) {
  ScorePart a{-INFINITY, 0.f, 0.f, 0.f};
  for (int s0 = lane; s0 < S; s0 += 256) {
    float4 q[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
      q[e] = s0 + 32 * e < S ? part[s0 + 32 * e] : make_float4(-INFINITY, 0.f, 0.f, 0.f);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (s0 + 32 * e < S) a = score_join(a, ScorePart{q[e].x, q[e].y, q[e].z, q[e].w});
  }
  return score_join_warp(a, lane);
}

// (lse, entropy); NaN where the row has a logit that is NaN or +infinity (with a
// soft-cap, any infinity), or none above -infinity.
__device__ __forceinline__ float2 score_of(const ScorePart& a) {
  const float nan = __int_as_float(0x7fc00000);
  if (!(a.s > 0.f && a.s < INFINITY) || !(fabsf(a.m) < INFINITY)) return make_float2(nan, nan);
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

// sum_k h_k w_k of a bf16 row with NW others by a warp, each as a rounded value
// and what the rounding leaves out: products of bf16 are exact in fp32, each step
// of the sum hands its rounding error to a second sum.  The same in all lanes.
// 256 G elements of each are read at once: a word's row is somewhere else in
// memory each time.
template <int NW, int G>
__device__ __forceinline__ void exact_dots(const uint16_t* __restrict__ h, const uint16_t* const (&w)[NW], int H,
                                           int lane, float2 (&out)[NW]) {
  float2 hi[NW], lo[NW];
#pragma unroll
  for (int i = 0; i < NW; ++i) hi[i] = lo[i] = both(0.f);
  const float2 minus = both(-1.f);
  for (int k0 = lane * 8; k0 < H; k0 += 256 * G) {
    Raw8<uint16_t> a[G], b[NW][G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int k = k0 + 256 * g;
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        if (k < H)
          b[i][g].q[0] = __ldg(reinterpret_cast<const uint4*>(w[i] + k));
        else
          b[i][g].zero();
      }
      if (k < H)
        a[g].q[0] = __ldg(reinterpret_cast<const uint4*>(h + k));
      else
        a[g].zero();
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
      if (k0 - lane * 8 + 256 * g >= H) break;  // (the whole warp)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 x = a[g].pair(e);
#pragma unroll
        for (int i = 0; i < NW; ++i) {
          const float2 p = mul2(x, b[i][g].pair(e));
          const float2 s = add2(hi[i], p);
          const float2 y = fma2(hi[i], minus, s);                                // s - hi
          const float2 r = fma2(y, minus, s);                                    // s - y
          lo[i] = add2(lo[i], add2(fma2(r, minus, hi[i]), fma2(y, minus, p)));  // (hi - r) + (p - y)
          hi[i] = s;
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NW; ++i) {
    float2 d = two_add(make_float2(hi[i].x, lo[i].x), make_float2(hi[i].y, lo[i].y));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
      d = two_add(d, make_float2(__shfl_xor_sync(0xffffffffu, d.x, off), __shfl_xor_sync(0xffffffffu, d.y, off)));
    // (a sum that is not finite has no rest; one that is NaN comes last)
    out[i] = !(fabsf(d.x) < INFINITY) ? make_float2(d.x == INFINITY ? d.x : -INFINITY, 0.f) : two_sum(d.x, d.y);
  }
}

// Whether word (a, i) comes before word (b, j): the larger logit, then the lower index.
__device__ __forceinline__ bool word_before(float2 a, int i, float2 b, int j) {
  if (a.x != b.x) return a.x > b.x;
  if (a.y != b.y) return a.y > b.y;
  return i < j;
}

// A float's bits in an unsigned order, and back (both infinities included).
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x);
  return u ^ ((u & 0x80000000u) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t k) {
  return __uint_as_float(k ^ ((k & 0x80000000u) ? 0x80000000u : 0xffffffffu));
}

struct SelectParams {
  const uint16_t* h;   // [N][H]
  const uint16_t* W;   // [V][H]
  const float4* part;  // [rows][S]
  const float2* rec;   // [rows][ld] chunk records: the two largest,
  const float* rec3;   // [rows][ld] and the third; or
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
//   1. Each thread takes the largest of its records (kDense: of its logits).  The
//      K-th largest of the threads', to 8 bits, by bisection with one counting
//      barrier a bit, is a lower bound of the K-th largest logit.
//   2. Listed are the words that reach the bound, less what both can be off by; of
//      a chunk whose third largest does too, all 32.  The K-th largest of the
//      listed is a better bound, and drops those that it rules out.
//   3. The logits of what is left, K words and their near ties, two words to a
//      warp at a time, and a rank for each by counting.
// More candidates than the list holds (logits that are nearly all equal) go
// through it in runs, in index order, with the K best so far kept and the bound
// raised to theirs.
constexpr int SELECT_CAP = 1024;  // words of the list
static_assert(SELECT_CAP >= SCORE_MAX_K + 32, "the list holds K words and a chunk");

// Bound by the gather of the words' rows and its latency: 64 words of 4,096 rows,
// 2.2 GB of a 1.24 GB head, take 495 us (three CTAs to an SM; two 580, four with
// half the loads in flight 560); 20 words of one row 21 us, four of them its
// products, the rest the steps' latencies.
template <int T, bool kDense, bool kLong>
__global__ void __launch_bounds__(T, T == 256 ? 3 : 1) score_select_kernel(const __grid_constant__ SelectParams p) {
  static_assert(T >= SCORE_MAX_K, "K threads have a largest record each");
  dependent_start();
  using idx_t = typename std::conditional<kLong, long long, int>::type;
  __shared__ float2 val[SELECT_CAP];
  __shared__ __align__(16) float near[SELECT_CAP + 4];  // the records' logits
  __shared__ int word[SELECT_CAP];
  __shared__ int sums[T / 32];
  __shared__ int found, kept_words, whole_chunks;
  __shared__ float best_k;
  __shared__ float2 target_z;
  __shared__ ScorePart parts[T / 32], row_part;
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
  // a unit: a chunk and its record, or (kDense) a word and its logit
  const int units = kDense ? p.V : (p.V + 31) / 32;
  const idx_t base = static_cast<idx_t>(j) * p.ld;
  auto unit = [&](int c) {
    if constexpr (kDense) {
      return make_float2(p.z[base + c], -INFINITY);
    } else {
      return p.rec[base + c];
    }
  };
  const uint16_t* h = p.h + i * p.H;
  float top = -INFINITY;
  // the row's partials, joined by warps and then by the first
  {
    ScorePart w{-INFINITY, 0.f, 0.f, 0.f};
    const float4* part = p.part + static_cast<idx_t>(j) * p.S;
    for (int s = t; s < p.S; s += T) {
      const float4 q = part[s];
      w = score_join(w, ScorePart{q.x, q.y, q.z, q.w});
    }
    w = score_join_warp(w, lane);
    if (lane == 0) parts[warp] = w;
  }
#pragma unroll(T == 256 ? 4 : 8)
  for (int c = t; c < units; c += T) top = fmaxf(top, unit(c).x);
  if (t == 0) found = kept_words = whole_chunks = 0;
  const uint32_t mine = ordered(top);
  uint32_t prefix = 0;
#pragma unroll 1
  for (uint32_t bit = 0x80000000u; bit >= 0x8000u; bit >>= 1) {
    if (__syncthreads_count(mine >= (prefix | bit)) >= K) prefix |= bit;
    if (bit == 0x80000000u && warp == 0) {
      const ScorePart w =
          score_join_warp(lane < T / 32 ? parts[lane] : ScorePart{-INFINITY, 0.f, 0.f, 0.f}, lane);
      if (lane == 0) row_part = w;
    }
  }
  const ScorePart whole = row_part;
  const float2 r = score_of(whole);
  if (r.x != r.x) {
    score_no_row(p.out, i, r.x, t, T);
    return;
  }
  // (fewer than K threads with a record above -infinity: every word is a candidate)
  const float low = prefix > ordered(-INFINITY) ? unordered(prefix) : -INFINITY;
  // the magnitude that records near the bound are off in proportion to
  const float off =
      p.slack * fmaxf(whole.top < INFINITY ? whole.top : 0.f, low > -INFINITY ? fabsf(low) : 0.f) + 1e-43f;
  float reach = low - 2.f * off;
  const bool want_target = tgt >= 0 && tgt < p.V && p.out.logp != nullptr;
  // words of a unit that are still in the running
  auto words_of = [&](int c, float2 q) {
    if (!(q.x >= reach)) return 0;
    if (kDense) return 1;
    if (reach == -INFINITY) return min(32, p.V - 32 * c);  // (also words whose logit is -infinity, which records leave out)
    if (!(q.y >= reach)) return 1;
    return p.rec3[base + c] >= reach ? min(32, p.V - 32 * c) : 2;
  };
  auto put = [&](int at, int c, float2 q, int n) {
    if (kDense) {
      word[at] = c;
      near[at] = q.x;
    } else if (n > 2 || reach == -INFINITY) {
      for (int e = 0; e < n; ++e) word[at + e] = 32 * c + e;
    } else {
      word[at] = 32 * c + 31 - static_cast<int>(__float_as_uint(q.x) & 31u);
      near[at] = q.x;
      if (n == 2) {
        word[at + 1] = 32 * c + 31 - static_cast<int>(__float_as_uint(q.y) & 31u);
        near[at + 1] = q.y;
      }
    }
  };
  // the logits of the words [from, total) (and, the first time, of the target),
  // then the best K of all in order at the list's front
  constexpr int PER = (SELECT_CAP + T - 1) / T;
  auto settle = [&](int from, int total) {
    const int end = total + (from == 0 && want_target ? 1 : 0);
    for (int e = from + 2 * warp; e < end; e += 2 * (T / 32)) {
      const long long v0 = e < total ? word[e] : tgt;
      const long long v1 = e + 1 < total ? word[e + 1] : e + 1 < end ? tgt : v0;
      const uint16_t* const w[2] = {p.W + v0 * p.H, p.W + v1 * p.H};
      float2 z[2];
      exact_dots<2, T == 256 ? 4 : 6>(h, w, p.H, lane, z);
      if (lane < 2 && e + lane < end) (e + lane < total ? val[e + lane] : target_z) = lane == 0 ? z[0] : z[1];
    }
    __syncthreads();
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
#pragma unroll 4
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
  auto zero_row = [&] {
    bool any = false;
    for (int k = t * 8; k < p.H; k += T * 8) {
      const uint4 x = __ldg(reinterpret_cast<const uint4*>(h + k));
      any |= ((x.x | x.y | x.z | x.w) & 0x7fff7fffu) != 0u;
    }
    return __syncthreads_or(any) == 0;
  };
#pragma unroll 4
  for (int c = t; c < units; c += T) {
    const float2 q = unit(c);
    const int n = words_of(c, q);
    if (n > 0) {
      const int at = atomicAdd(&found, n);  // (the order within the list does not matter)
      if (at <= SELECT_CAP - n) put(at, c, q, n);
      if (n > 2 || (!kDense && reach == -INFINITY)) whole_chunks = 1;
    }
  }
  __syncthreads();
  int listed = found;
  if (listed <= SELECT_CAP) {
    // the better bound (words of whole chunks have no record of their own)
    if (listed > K && whole_chunks == 0) {
      if (t < 4) near[listed + t] = -INFINITY;
      __syncthreads();
      float m[PER];
      int w[PER];
#pragma unroll
      for (int q = 0; q < PER; ++q) {
        const int e = t + q * T;
        m[q] = -INFINITY;
        if (e < listed) {
          m[q] = near[e];
          w[q] = word[e];
          int above = 0, equal = 0;
          for (int o = 0; o < listed; o += 4) {
            const float4 x = *reinterpret_cast<const float4*>(near + o);
            above += (x.x > m[q]) + (x.y > m[q]) + (x.z > m[q]) + (x.w > m[q]);
            equal += (x.x == m[q]) + (x.y == m[q]) + (x.z == m[q]) + (x.w == m[q]);
          }
          if (above < K && above + equal >= K) best_k = m[q];  // (one value, whoever writes it)
        }
      }
      __syncthreads();
      const float again = best_k - 2.f * off;
#pragma unroll
      for (int q = 0; q < PER; ++q)
        if (t + q * T < listed && m[q] >= again) word[atomicAdd(&kept_words, 1)] = w[q];
      __syncthreads();
      listed = kept_words;
    }
    settle(0, listed);
  } else if (zero_row()) {
    // (a row of padding, of which a batch may hold many: nothing to sum)
    for (int e = t; e < K; e += T) {
      val[e] = make_float2(0.f, 0.f);
      word[e] = e;
    }
    if (t == 0) target_z = make_float2(0.f, 0.f);
    __syncthreads();
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
  // (the list holds K words at least: K records reach the bound, or there is none and all V words do)
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

// dlogits of the scores from the forward's kept logits: with x = log2 p_v = E_v +
// mx - lse log2 e (E: fp16, relative to its chunk's maximum mx),
//   D_v = -p_v (ga + ge (x ln 2 + entropy)) f'(z) + [v = t] ga f'(z)
// The target's column is formed from its own fp32 logit zt: 1 - p_t is small where
// the target is likely, and E's p_t would not do.  Rows and columns as
// topk_dlogits_kernel: row r of E is row ri[r] (r without ri); a CTA takes
// `steps` runs of TOPK_DL_COLS columns, a lane 8 neighbouring ones at a time.
// kLo: D in two bf16 parts, what the first one's rounding leaves out lo rows
// further on; the rows from `rows` to lo are zeroed.
// The last CTA of a row copies its h as the dW GEMM reads it, zeros for an ignored
// row (whatever its h holds) and up to the next 64 listed ones.
// Bound by memory: 256 x 248,320, 254 MB read and written, in 37 us.
struct ScoreDlogits {
  const uint16_t* h;  // [N][H]
  uint16_t* hc;       // [rows][H], or null
  int H;
  const uint16_t* E;  // [rows][ldD]
  const float* mx;    // [rows][ld_mx]
  uint16_t* D;        // [rows][ldD]
  int ldD, ld_mx, steps, rows, lo, V;
  const int* ri;
  const int* count;
  const int64_t* targets;
  long long ignore;
  const float* zt;
  const float* lse;
  const float* entropy;
  const float* g_logp;
  const float* g_entropy;
  int tf_softcap;
  float tf_a, tf_b, tf_d;
};

template <bool kLong, bool kLo>
__global__ void __launch_bounds__(SMALL_THREADS) score_dlogits_kernel(const __grid_constant__ ScoreDlogits p) {
  dependent_start();
  using idx_t = typename std::conditional<kLong, long long, int>::type;
  const int r = blockIdx.y;
  const int n = p.ri != nullptr ? *p.count : p.rows;
  if (p.ri != nullptr && r >= (n + 63) / 64 * 64) return;
  const bool inside = r < n;
  const long long i = !inside ? 0 : p.ri ? p.ri[r] : r;
  const long long tgt = inside ? p.targets[i] : p.ignore;
  const float ga = inside && p.g_logp != nullptr ? p.g_logp[i] : 0.f;
  const float ge = inside && p.g_entropy != nullptr ? p.g_entropy[i] : 0.f;
  const bool live = inside && tgt != p.ignore && (ga != 0.f || ge != 0.f);
  if (blockIdx.x == gridDim.x - 1 && p.hc != nullptr && r < p.rows) {
    const uint16_t* from = p.h + i * p.H;
    uint16_t* to = p.hc + static_cast<long long>(r) * p.H;
    for (int k = threadIdx.x * 8; k < p.H; k += SMALL_THREADS * 8)
      *reinterpret_cast<uint4*>(to + k) =
          tgt != p.ignore ? *reinterpret_cast<const uint4*>(from + k) : make_uint4(0u, 0u, 0u, 0u);
  }
  uint16_t* row = p.D + static_cast<idx_t>(r) * p.ldD;
  uint16_t* row2 = row + static_cast<idx_t>(p.lo) * p.ldD;
  const int c0 = blockIdx.x * p.steps * TOPK_DL_COLS;
  const int c1 = min(p.ldD, c0 + p.steps * TOPK_DL_COLS);
  if (!live) {
    for (int c = c0 + threadIdx.x * 8; c < c1; c += SMALL_THREADS * 8) {
      *reinterpret_cast<uint4*>(row + c) = make_uint4(0u, 0u, 0u, 0u);
      if constexpr (kLo) *reinterpret_cast<uint4*>(row2 + c) = make_uint4(0u, 0u, 0u, 0u);
    }
    return;
  }
  const float lse = p.lse[i], ent = p.entropy[i];
  const float nlse2 = -lse * kLog2e, a = -ge * kLn2, b = -fmaf(ge, ent, ga);
  const uint16_t* src = p.E + static_cast<idx_t>(r) * p.ldD;
  const float* rmx = p.mx + static_cast<idx_t>(r) * p.ld_mx;
  const int first = c0 + (threadIdx.x >> 5) * 1024 + (threadIdx.x & 31) * 8;
  for (int cs = first; cs < c1; cs += TOPK_DL_COLS) {
    uint4 q[4];
    float cm[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = cs + k * 256;
      if (c < c1) {
        q[k] = *reinterpret_cast<const uint4*>(src + c);
        cm[k] = rmx[c / 32];
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = cs + k * 256;
      if (c >= c1) continue;
      uint32_t w[4] = {q[k].x, q[k].y, q[k].z, q[k].w};
      uint32_t w2[4];
      const float2 shift = both(cm[k] + nlse2);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 x = add2(__half22float2(*reinterpret_cast<const __half2*>(&w[e])), shift);
        const float2 pr = make_float2(ex2_approx(x.x), ex2_approx(x.y));
        // (p log p is 0 where p is)
        const float2 f = fma2(make_float2(fmaxf(x.x, -1000.f), fmaxf(x.y, -1000.f)), both(a), both(b));
        float2 dv = mul2(pr, f);
        if (p.tf_softcap) {  // f' = d (1 - tanh^2), tanh = u / b
          const float k2 = kLn2 / p.tf_b;
          const float2 th = make_float2(fmaf(x.x, k2, lse / p.tf_b), fmaf(x.y, k2, lse / p.tf_b));
          dv = mul2(dv, make_float2(p.tf_d * fmaxf(0.f, 1.f - th.x * th.x), p.tf_d * fmaxf(0.f, 1.f - th.y * th.y)));
        } else {
          dv = mul2(dv, both(p.tf_a));
        }
        w[e] = pack_bf16x2(dv.x, dv.y);
        if constexpr (kLo) w2[e] = bf16x2_rest(dv.x, dv.y, w[e]);
      }
      *reinterpret_cast<uint4*>(row + c) = make_uint4(w[0], w[1], w[2], w[3]);
      if constexpr (kLo) *reinterpret_cast<uint4*>(row2 + c) = make_uint4(w2[0], w2[1], w2[2], w2[3]);
    }
  }
  if (tgt < c0 || tgt >= c1 || tgt >= p.V) return;  // (the whole CTA; c0 >= 0)
  __syncthreads();  // the target's column after the CTA's own stores
  if (threadIdx.x == 0) {
    const float u = p.zt[i], lp = u - lse;
    const float slope = p.tf_softcap ? p.tf_d * fmaxf(0.f, 1.f - (u / p.tf_b) * (u / p.tf_b)) : p.tf_a;
    const float pt = expf(lp);
    // (1 - p_t straight from log p_t)
    const float dv = (-ga * expm1f(lp) - ge * pt * (fmaxf(lp, -1000.f) + ent)) * slope;
    const uint32_t w = pack_bf16x2(dv, 0.f);
    row[tgt] = static_cast<uint16_t>(w & 0xffffu);
    if constexpr (kLo) row2[tgt] = static_cast<uint16_t>(bf16x2_rest(dv, 0.f, w) & 0xffffu);
  }
}

// Chunk records of N rows of logits (the few-row forward's), a warp to a chunk
// (one row of 151,936 logits: 3.3 us).
__global__ void __launch_bounds__(SMALL_THREADS)
    score_record_kernel(const float* z, int N, int V, int ldz, float2* rec, float* rec3, int ld) {
  dependent_start();
  const int chunks = (V + 31) / 32, lane = threadIdx.x & 31;
  const long long u = static_cast<long long>(blockIdx.x) * (SMALL_THREADS / 32) + (threadIdx.x >> 5);
  if (u >= static_cast<long long>(N) * chunks) return;
  const int r = static_cast<int>(u / chunks), c = static_cast<int>(u - static_cast<long long>(r) * chunks);
  const int v = 32 * c + lane;
  float m1 = v < V ? score_key(z[static_cast<long long>(r) * ldz + v], lane) : -INFINITY;
  float m2 = -INFINITY, m3 = -INFINITY;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    const float a = __shfl_xor_sync(0xffffffffu, m1, off), b = __shfl_xor_sync(0xffffffffu, m2, off),
                d = __shfl_xor_sync(0xffffffffu, m3, off);
    // of two descending triples
    m3 = fmaxf(fmaxf(m3, d), fmaxf(fminf(m1, b), fminf(m2, a)));
    m2 = fmaxf(fmaxf(m2, b), fminf(m1, a));
    m1 = fmaxf(m1, a);
  }
  if (lane == 0) {
    rec[static_cast<long long>(r) * ld + c] = make_float2(m1, m2);
    rec3[static_cast<long long>(r) * ld + c] = m3;
  }
}

// The forward of at most TOPK_GEMV_ROWS rows, as topk_gemv_kernel (a warp takes 4
// vocabulary rows at a time and sums them in fp32; lane 4 r + c keeps row r's
// partial over the c-th of the 4).  Writes the logits [N][ldz] where z is given,
// the target's transformed logit where zt is, and one partial per row and CTA
// ([N][gridDim.x]).  Bound by reading W: 1 x 4,096 x 151,936 in 177 us, 7.0 TB/s.
// The whole forward, and the tiled one (us): one row 197 / 289, two 201 / 289, three
// 221 / 242, four 223 / 242.
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
