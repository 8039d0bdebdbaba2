// libflce host side: the entry points of the scores -- log-probability and
// entropy with their gradients, and the likeliest words (row kernels in
// score.cuh, the forward and the tiled backward in gemm.cuh and flce.cu).
#pragma once

namespace {

// Words from the logits themselves, or from chunk records.  A chunk that three of
// the K words share costs 32 products, so the records serve while chunks are
// many: about K^3 / 6 / chunks^2 of them are shared.  Below 4 K chunks (K / 96
// shared ones) the logits are held, at 4 bytes instead of 3/8 byte a column.
// (512 x 1,024, logits / records: 64 / 72 us at 3.9 K chunks, K 64, and 111 / 142, K
// 128; 164 / 126 at 7.8 K chunks, K 128, and 152 / 97 at 10 K.)
bool score_dense(int64_t V, int64_t k) { return ceil_div(V, 32) < 4 * k; }

constexpr size_t kScoreBlockBytes = size_t(256) << 20;  // of records or logits held at once

// Logits kept from the forward for the backward (flce_score's state): of one row
// block, and at most 32,768 rows (the dlogits pass puts one row per grid row).
// More than a tile of rows are compacted to the counted ones, as in
// flce_forward_backward; both calls decide it alike, by the row count alone.
constexpr int64_t kKeepMaxRows = 32768;
constexpr int64_t kKeepCompactRows = 2 * BM;

struct KeepLayout {
  size_t E = 0, mx = 0, zt = 0, idx = 0, count = 0, total = 0;
  long long ldD = 0, ld_mx = 0;
};
KeepLayout keep_layout(int64_t N, int64_t V) {
  KeepLayout L;
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += align256(bytes);
    return at;
  };
  L.ldD = round_up(V, 32);
  L.ld_mx = fused_ld_mx(V);
  L.E = take(static_cast<size_t>(N) * L.ldD * 2);
  L.mx = take(static_cast<size_t>(N) * L.ld_mx * 4);
  L.zt = take(static_cast<size_t>(N) * 4);
  if (N > kKeepCompactRows) {
    L.idx = take(static_cast<size_t>(N) * 4);
    L.count = take(256);
  }
  L.total = o;
  return L;
}

// At short rows of h the product costs no more than writing and reading what was
// kept.  Forward and backward with kept logits, and without (us):
//   rows x vocabulary      H  64        256        384        512        1,024
//     256 x 151,936        144 / 156  154 / 167  178 / 192  190 / 213  265 / 310
//     512 x 151,936        227 / 215  235 / 228
//   1,024 x 151,936        350 / 328  374 / 355  436 / 427
//   2,048 x 151,936                   648 / 630             830 / 870
//   4,096 x  32,000                   331 / 329             409 / 436  615 / 706
// So from 512 on, and up to one tile of rows, which are not compacted and whose
// backward is bound by its launches.  (At most 128 rows are kept in any case: only
// their dlogits from kept logits take two bf16 parts, fused_lo_rows, and one entry
// often holds most of so few rows' gradients.)
constexpr int64_t kKeepMinHidden = 512;

// Whether a call of these sizes keeps its logits: they fit the caller's dlogits
// budget (chunk_rows x V), and reading them costs less than their product again.
bool keep_pays(int64_t N, int64_t H, int64_t chunk_rows) {
  return N > 0 && N <= kKeepMaxRows && N <= round_up(std::max<int64_t>(1, chunk_rows), BM) &&
         (H >= kKeepMinHidden || N <= kKeepCompactRows);
}

// Whether a call lists the rows that count and leaves the others out.
bool score_skips(int64_t N, bool keep, bool gemv) {
  return keep ? N > kKeepCompactRows : !gemv && N >= skip_min_rows();
}

// The forward's splits where the device alone knows how many row tiles it has:
// planned for all of them, six row tiles in 12 splits of 11 column tiles keep 72 of
// 76 pairs busy, and five keep 60 as long.  So the splits are those that do best
// over every count from half the row tiles on (a unit costs a tenth of a tile beside
// its tiles: its partials, and its targets).  1,501 rows, a quarter masked, x 1,096 x
// 32,003: 86 us, 90 with the splits for all rows.
void plan_counted(FwdPlan& f, long long rows, int workers, size_t partials_cap) {
  if (opt(FLCE_OPT_FWD_SPLITS) > 0) return;
  const long long fit = std::max(1LL, static_cast<long long>(partials_cap) / (8 * std::max(1LL, rows)));
  const int smax = static_cast<int>(std::min<long long>(std::min(f.n_tiles, 256), fit));
  double best = 1e300;
  for (int s = 1; s <= smax; ++s) {
    const int tps = static_cast<int>(ceil_div(f.n_tiles, s)), se = static_cast<int>(ceil_div(f.n_tiles, tps));
    double cost = 0.;
    for (int m = (f.m_tiles + 1) / 2; m <= f.m_tiles; ++m)
      cost += static_cast<double>(ceil_div(static_cast<long long>(m) * se, workers)) * (tps + 0.1) / m;
    if (cost < best) {
      best = cost;
      f.S = se;
      f.tps = tps;
    }
  }
  f.units = f.m_tiles * f.S;
  f.grid = std::min(f.units, workers);
}

// CTA group of the score forwards.  Up to 128 rows each CTA takes a tile of its
// own: half of a pair's 256 rows would be empty, and its products cost as much as
// reading W (33 x 1,536 x 151,936: 98 us, pairs 111; 128 x 4,096: 205 and 211, with
// words 225 and 240).  So too where pairs' tiles hold so much more than the rows that
// their waves are more than 1.15 times as many; a tile takes 1.1 times a pair's (us,
// CTAs / pairs: 300 x 4,096 x 128,256 271 / 302, 384 rows 275 / 308; 256 x 2,048 x
// 151,936 135 / 125, 900 380 / 352; 600 x 4,096 x 32,000 134 / 117) -- but not where
// rows start inside a 128-byte line, whose loads are slower, and CTAs make half as
// many again for a product (384 x 1,096 x 151,936 136 / 133, with 1,088 100 / 109; 777
// x 1,096 x 32,003 70 / 60).  The backward keeps the pairs (33 x 1,536: 205 us, 232
// without).
int score_group(int64_t N, int64_t H, int64_t V) {
  if (N <= BM || cta_group() == 1) return 1;
  if (H % 64 != 0) return 2;
  const long long n = ceil_div(V, BN);
  return 1.15 * static_cast<double>(ceil_div(ceil_div(N, BM) * n, device_workers(1))) <
                 static_cast<double>(ceil_div(ceil_div(N, 2 * BM) * n, device_workers(2)))
             ? 1
             : 2;
}

struct ScorePlan {
  bool gemv = false, dense = false, keep = false;
  long long rows = 0;  // of a launch
  int S = 1;           // partials of a row
  long long ld = 0;    // row pitch of the records (float2) or logits (fp32)
  FwdPlan f;
};
ScorePlan score_plan(int64_t N, int64_t H, int64_t V, int64_t k, bool keep, int workers, int tm) {
  ScorePlan q;
  q.keep = keep;
  q.gemv = !keep && topk_gemv_for(N, H);
  q.dense = k > 0 && score_dense(V, k);
  // both cover whole tiles
  q.ld = k == 0 ? 0 : q.dense ? round_up(V, BN) : round_up(V, BN) / 32;
  q.rows = keep ? std::max<int64_t>(N, 1) : fwd_block_rows(N, tm);
  if (k > 0 && !q.gemv) {
    const long long fit = static_cast<long long>(kScoreBlockBytes / (static_cast<size_t>(q.ld) * (q.dense ? 4 : 12)));
    q.rows = std::min(q.rows, std::max<long long>(tm, fit / tm * tm));
  }
  // (a row has kScoreParts partials of 16 bytes to a split: four times the 8 that the cap counts)
  q.f = plan_forward(q.rows, H, V, workers, tm, kFwdPartialsCap / 4);
  if (score_skips(N, keep, q.gemv)) plan_counted(q.f, q.rows, workers, kFwdPartialsCap / 4);
  q.S = q.gemv ? topk_gemv_ctas(V) : kScoreParts * q.f.S;
  return q;
}

struct ScoreLayout {
  size_t zt = 0, part = 0, z = 0, rec = 0, rec3 = 0, bad = 0, idx = 0, blk = 0, count = 0, hc = 0, total = 0;
};
ScoreLayout score_layout(int64_t N, int64_t H, int64_t V, int64_t k, const ScorePlan& q) {
  ScoreLayout L;
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += align256(bytes);
    return at;
  };
  const size_t n = static_cast<size_t>(std::max<int64_t>(N, 1)), rows = static_cast<size_t>(std::max(1LL, q.rows));
  L.zt = take(k == 0 ? n * 4 : 0);
  L.part = take(rows * q.S * 16);
  L.z = take(k > 0 && (q.dense || q.gemv) ? rows * round_up(V, BN) * 4 : 0);
  L.rec = take(k > 0 && !q.dense ? rows * q.ld * 8 : 0);
  L.rec3 = take(k > 0 && !q.dense ? rows * q.ld * 4 : 0);
  L.bad = take(256);
  if (score_skips(N, q.keep, q.gemv)) {
    L.idx = take(n * 4);
    L.blk = take(static_cast<size_t>(ceil_div(N, COMPACT_ROWS_PER_BLOCK)) * 4);
    L.count = take(256);
    L.hc = take(rows * H * 2);
  }
  L.total = o;
  return L;
}

// How far a record or logit of the forward can be off the row's exact logits,
// relative to their largest magnitude.  Each of H / 16 steps cuts its running sum
// by less than one unit of its last place, 2^-23 of it (the few-row forward's
// rounded sums are off by less).  The running sum is at most |h| |w|, which is
// sqrt(H) / 4 times the row's largest logit where that is as large as the largest
// of some 30,000 products of random directions (4 |h| |w| / sqrt(H)), and 4 times
// is allowed for at least.  The column in a record's low bits changes it by 2^-18.
float score_slack(int64_t H) {
  const double steps = static_cast<double>(ceil_div(H, UMMA_K));
  return static_cast<float>(std::max(4.0, std::sqrt(static_cast<double>(H)) / 4.0) * steps / 8388608.0 + 1.0 / 131072.0);
}

flce_status score_rows(const ScorePlan& q, bool kLong, const ScoreRows& rows, const float4* part, const float2* rec,
                       const float* rec3, const float* z, const flce_bf16* h, const flce_bf16* W, const GemmParams& tf,
                       const int64_t* targets, long long ignore, const float* zt, const ScoreOut& out,
                       cudaStream_t st) {
  ProfScope ps(K_SCORE, st);
  if (out.k == 0) {
    const dim3 grid(static_cast<unsigned>(ceil_div(rows.rows, SMALL_THREADS / 32)));
    auto go = [&](auto kern) {
      return launch_dependent(kern, grid, SMALL_THREADS, 0, st, part, q.S, rows, zt, targets, ignore, tf.V, out);
    };
    FLCE_CUDA_TRY(kLong ? go(score_row_kernel<true>) : go(score_row_kernel<false>));
    return FLCE_OK;
  }
  SelectParams p{};
  p.h = h;
  p.W = W;
  p.part = part;
  p.rec = rec;
  p.rec3 = rec3;
  p.z = z;
  p.S = q.S;
  p.ld = static_cast<int>(q.ld);
  p.H = tf.H;
  p.V = tf.V;
  p.rows = rows;
  p.targets = targets;
  p.ignore = ignore;
  p.slack = score_slack(tf.H);
  p.tf_softcap = tf.tf_softcap;
  p.tf_a = tf.tf_a;
  p.tf_b = tf.tf_b;
  p.out = out;
  auto go = [&](auto kern, int threads) {
    return launch_dependent(kern, dim3(static_cast<unsigned>(rows.rows)), threads, 0, st, p);
  };
  // with a row to an SM, or fewer, a row's latency counts: more warps to its words
  // (152 rows x 2,048 x 151,936, K 64: 150 us, 170 with 256 threads; 777 x 1,096 x
  // 32,003, K 37: 138 with 512 threads, 107)
  const bool few = rows.rows <= device_sms();
  auto of = [&](auto dense) -> cudaError_t {
    constexpr bool D = decltype(dense)::value;
    if (kLong) return go(score_select_kernel<256, D, true>, 256);
    return few ? go(score_select_kernel<512, D, false>, 512) : go(score_select_kernel<256, D, false>, 256);
  };
  FLCE_CUDA_TRY(q.dense ? of(std::true_type{}) : of(std::false_type{}));
  return FLCE_OK;
}

flce_status score_gemv(const ScorePlan& q, const GemmParams& p, const flce_bf16* h, const flce_bf16* W, float* z,
                       float2* rec, float* rec3, const int64_t* targets, float* zt, float4* part, cudaStream_t st) {
  const int ldz = static_cast<int>(round_up(p.V, BN));
  {
    ProfScope ps(K_FWD, st);
    auto go = [&](auto kern, int nr) -> cudaError_t {
      const size_t smem = static_cast<size_t>(nr) * p.H * 4;
      cudaError_t e =
          cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kGemvMaxSmem));
      if (e != cudaSuccess) return e;
      return launch_dependent(kern, dim3(q.S), 32 * TOPK_GEMV_WARPS, smem, st, h, W, p.N, p.H, p.V, z, ldz, targets, zt,
                              p.tf_softcap, p.tf_a, p.tf_b, part);
    };
    FLCE_CUDA_TRY(p.N == 1   ? go(score_gemv_kernel<1>, 1)
                  : p.N == 2 ? go(score_gemv_kernel<2>, 2)
                             : go(score_gemv_kernel<4>, 4));
  }
  if (rec == nullptr) return FLCE_OK;
  ProfScope ps(K_SCORE, st);
  const long long units = static_cast<long long>(p.N) * ceil_div(p.V, 32);
  FLCE_CUDA_TRY(launch_dependent(score_record_kernel, dim3(static_cast<unsigned>(ceil_div(units, SMALL_THREADS / 32))),
                                 SMALL_THREADS, 0, st, static_cast<const float*>(z), p.N, p.V, ldz, rec,
                                 rec3, static_cast<int>(q.ld)));
  return FLCE_OK;
}

}  // namespace

extern "C" {

size_t flce_score_workspace_bytes(int64_t N, int64_t H, int64_t V, int64_t k) {
  if (!topk_sizes_ok(N, H, V) || k < 0 || k > SCORE_MAX_K || k > V) return 0;
  const int cg = score_group(N, H, V);
  const int workers = device_workers(cg);
  auto of = [&](bool keep) {
    return score_layout(N, H, V, k, score_plan(N, H, V, k, keep, workers, BM * cg)).total;
  };
  return k == 0 && N <= kKeepMaxRows ? std::max(of(false), of(true)) : of(false);
}

size_t flce_score_state_bytes(int64_t N, int64_t H, int64_t V, int64_t chunk_rows) {
  if (!topk_sizes_ok(N, H, V) || !keep_pays(N, H, chunk_rows)) return 0;
  return keep_layout(N, V).total;
}

flce_status flce_score(const flce_bf16* h, const flce_bf16* W, const int64_t* targets, int64_t N, int64_t H, int64_t V,
                       int64_t k, int64_t ignore_index, const flce_logit_transform* transform, float* out_logp,
                       float* out_lse, float* out_entropy, int64_t* out_ids, float* out_logprobs, void* state,
                       void* workspace, size_t workspace_bytes, void* stream) {
  if (!topk_sizes_ok(N, H, V) || k < 0 || k > V) return FLCE_ERR_INVALID_ARG;
  GemmParams tfp{};
  if (!transform_params(transform, tfp)) return FLCE_ERR_INVALID_ARG;
  // (an empty tensor has no address)
  if (N > 0 && !out_logp && !out_lse && !out_entropy && !out_ids && !out_logprobs) return FLCE_ERR_INVALID_ARG;
  if (N > 0 && ((out_logp && !targets) || ((out_ids || out_logprobs) != (k > 0)))) return FLCE_ERR_INVALID_ARG;
  if (N > 0 && (!h || !W)) return FLCE_ERR_INVALID_ARG;
  if (state && N > 0 && (k != 0 || !targets)) return FLCE_ERR_INVALID_ARG;
  if (k > SCORE_MAX_K || H % 8 != 0 || (state && N > kKeepMaxRows) || !aligned(state, 256)) return FLCE_ERR_UNSUPPORTED;
  if (!aligned(h, 16) || !aligned(W, 16) || !aligned(targets, 8) || !aligned(out_logp, 4) || !aligned(out_lse, 4) ||
      !aligned(out_entropy, 4) || !aligned(out_ids, 8) || !aligned(out_logprobs, 4))
    return FLCE_ERR_UNSUPPORTED;
  if (N == 0) return FLCE_OK;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int cg = score_group(N, H, V), tm = BM * cg;
  const int workers = device_workers(cg);
  const bool keep = state != nullptr;
  const ScorePlan q = score_plan(N, H, V, k, keep, workers, tm);
  const ScoreLayout L = score_layout(N, H, V, k, q);
  const KeepLayout K = keep_layout(N, V);
  uint8_t* kb = static_cast<uint8_t*>(state);
  Workspace ws;
  flce_status s = get_workspace(ws, workspace, workspace_bytes, L.total, st);
  if (s != FLCE_OK) return s;
  uint8_t* wb = static_cast<uint8_t*>(ws.ptr);
  float* zt = keep ? reinterpret_cast<float*>(kb + K.zt) : k == 0 ? reinterpret_cast<float*>(wb + L.zt) : nullptr;
  float4* part = reinterpret_cast<float4*>(wb + L.part);
  float* z = k > 0 && (q.dense || q.gemv) ? reinterpret_cast<float*>(wb + L.z) : nullptr;
  float2* rec = k > 0 && !q.dense ? reinterpret_cast<float2*>(wb + L.rec) : nullptr;
  float* rec3 = k > 0 && !q.dense ? reinterpret_cast<float*>(wb + L.rec3) : nullptr;
  const int Ni = static_cast<int>(N);
  if (targets != nullptr && validate_on()) {
    int* bad = reinterpret_cast<int*>(wb + L.bad);
    FLCE_CUDA_TRY(cudaMemsetAsync(bad, 0, sizeof(int), st));
    prep_kernel<<<static_cast<int>(ceil_div(N, SMALL_THREADS)), SMALL_THREADS, 0, st>>>(
        targets, Ni, static_cast<int>(V), ignore_index, nullptr, bad);
    FLCE_CUDA_TRY(cudaGetLastError());
    int nbad = 0;
    FLCE_CUDA_TRY(cudaMemcpyAsync(&nbad, bad, sizeof(int), cudaMemcpyDeviceToHost, st));
    FLCE_CUDA_TRY(cudaStreamSynchronize(st));
    if (nbad != 0) return FLCE_ERR_BAD_TARGET;
  }
  const ScoreOut out{out_logp, out_lse, out_entropy, out_ids, out_logprobs, static_cast<int>(k)};
  const bool kLong = q.rows * std::max<long long>({q.ld, q.S, keep ? K.ldD : 0}) >= INT_MAX;
  GemmParams p{};
  p.n_tiles = q.f.n_tiles;
  p.k_blocks = q.f.k_blocks;
  p.cols = q.f.S;
  p.n_per_unit = q.f.tps;
  p.kb_per_split = q.f.k_blocks;
  p.k_splits = 1;
  p.N = Ni;
  p.H = static_cast<int>(H);
  p.V = static_cast<int>(V);
  p.targets = targets;
  p.ignore_index = ignore_index;
  p.zt = zt;
  p.tf_softcap = tfp.tf_softcap;
  p.tf_a = tfp.tf_a;
  p.tf_b = tfp.tf_b;
  p.tf_d = tfp.tf_d;
  p.score_part = part;
  p.rec = rec;
  p.rec3 = rec3;
  p.z = q.dense ? z : nullptr;
  p.rec_ld = static_cast<int>(q.ld);
  if (q.gemv) {
    s = score_gemv(q, p, h, W, z, rec, rec3, targets, zt, part, st);
    if (s != FLCE_OK) return s;
    return score_rows(q, kLong, ScoreRows{0, Ni, nullptr, nullptr, 0}, part, rec, rec3, z, h, W, p, targets,
                      ignore_index, zt, out, st);
  }
  // the rows without a target to score are left out, as flce_forward_ex2 does
  const bool skip = targets != nullptr && (keep || compact_on()) && L.hc != 0;
  int* idx = reinterpret_cast<int*>(keep ? kb + K.idx : wb + L.idx);
  int* count = reinterpret_cast<int*>(keep ? kb + K.count : wb + L.count);
  uint16_t* hc = reinterpret_cast<uint16_t*>(wb + L.hc);
  if (skip) {
    s = list_valid_rows(targets, Ni, ignore_index, reinterpret_cast<int*>(wb + L.blk), idx, count, false, st);
    if (s != FLCE_OK) return s;
    ProfScope ps(K_SCORE, st);
    const long long grid = std::min<long long>(ceil_div(N, SMALL_THREADS / 32), 8LL * device_sms());
    score_skipped_kernel<<<static_cast<unsigned>(grid), SMALL_THREADS, 0, st>>>(targets, ignore_index, Ni, out);
    FLCE_CUDA_TRY(cudaGetLastError());
  }
  CUtensorMap tA, tB;
  if (!make_map(&tA, skip ? hc : h, H, skip ? q.rows : N, H, BK, BM) || !make_map(&tB, W, H, V, H, BK, BN / cg))
    return FLCE_ERR_CUDA;
  CUtensorMap tE;  // the kept logits
  if (keep) {
    if (!make_map(&tE, kb + K.E, K.ldD, N, K.ldD, 64, 32)) return FLCE_ERR_CUDA;
    p.mx = reinterpret_cast<float*>(kb + K.mx);
    p.ldD = static_cast<int>(K.ldD);
    p.ld_mx = static_cast<int>(K.ld_mx);
  }
  int* err = nullptr;
  FLCE_CUDA_TRY(cudaGetSymbolAddress(reinterpret_cast<void**>(&err), g_device_error));
  p.err = err;
  for (long long row0 = 0; row0 < N; row0 += q.rows) {
    GemmParams g = p;
    g.tf_a *= 1.f + mma_cut(H);
    g.row0 = static_cast<int>(row0);
    g.rows = static_cast<int>(std::min(q.rows, N - row0));
    g.rows_cap = g.rows;
    g.m_tiles = static_cast<int>(ceil_div(g.rows, tm));
    g.num_units = g.m_tiles * q.f.S;
    g.group_m = std::min(16, g.m_tiles);
    ScoreRows rows{g.row0, g.rows, nullptr, nullptr, 0};
    if (skip) {
      g.row0 = 0;
      g.row_idx = idx;
      g.dyn_count = count;
      g.chunk_first = static_cast<int>(row0);
      rows = ScoreRows{0, g.rows, idx, count, g.chunk_first};
      s = gather_rows(h, H, idx, count, Ni, row0, q.rows, hc, st);
      if (s != FLCE_OK) return s;
    }
    {
      ProfScope ps(K_FWD, st);
      const int w = std::min(g.num_units, workers);
      FLCE_CUDA_TRY(keep    ? (launch_scored<MODE_FUSED_FWD, SCORE_ENTROPY>(cg, kLong, tA, tB, tE, g, w, st))
                    : k > 0 ? (launch_scored<MODE_FWD, SCORE_TOP>(cg, kLong, tA, tB, tB, g, w, st))
                            : (launch_scored<MODE_FWD, SCORE_ENTROPY>(cg, kLong, tA, tB, tB, g, w, st)));
    }
    s = score_rows(q, kLong, rows, part, rec, rec3, z, h, W, p, targets, ignore_index, zt, out, st);
    if (s != FLCE_OK) return s;
  }
  return FLCE_OK;
}

}  // extern "C"

namespace {

// The backward from kept logits: the second half of flce_forward_backward's step
// over one row block.  D may take two bf16 parts (fused_lo_rows).
struct KeepBwdPlan {
  FusedPlan fp;
  size_t D = 0, dh_part = 0, hc = 0, total = 0;
};
KeepBwdPlan keep_bwd_plan(int64_t N, int64_t H, int64_t V, int workers, int tm) {
  KeepBwdPlan k;
  k.fp = plan_fused(N, H, V, std::max<long long>(2 * BM, round_up(N, BM)), workers, tm, OneCall::kListed);
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += align256(bytes);
    return at;
  };
  const size_t d_rows = static_cast<size_t>(k.fp.lo > 0 ? 2 * k.fp.lo : N);
  k.D = take(d_rows * k.fp.ldD * 2);
  k.dh_part = take(k.fp.b.dh_f32 ? static_cast<size_t>(k.fp.b.dh_splits) * k.fp.R * H * 4 : 0);
  k.hc = take(static_cast<size_t>(N) * H * 2);
  k.total = o;
  return k;
}

flce_status score_backward_kept(const flce_bf16* h, const flce_bf16* W, const int64_t* targets, const float* lse,
                                const ScoreGrads& sc, uint8_t* state, flce_bf16* dH, float* dW, int64_t N, int64_t H,
                                int64_t V, int64_t ignore_index, const GemmParams& tfp, uint8_t* wb, cudaStream_t st) {
  const int cg = cta_group(), tm = BM * cg, workers = device_workers(cg);
  const KeepLayout K = keep_layout(N, V);
  const KeepBwdPlan kp = keep_bwd_plan(N, H, V, workers, tm);
  const FusedPlan& fp = kp.fp;
  const int Ni = static_cast<int>(N);
  const bool compact = N > kKeepCompactRows;
  uint16_t* D = reinterpret_cast<uint16_t*>(wb + kp.D);
  uint16_t* hc = reinterpret_cast<uint16_t*>(wb + kp.hc);
  float* dh_part = fp.b.dh_f32 ? reinterpret_cast<float*>(wb + kp.dh_part) : nullptr;
  const int* idx = compact ? reinterpret_cast<const int*>(state + K.idx) : nullptr;
  const int* count = compact ? reinterpret_cast<const int*>(state + K.count) : nullptr;
  const bool kLong = std::max<long long>(N, 2 * fp.lo) * fp.ldD >= INT_MAX || N * H >= INT_MAX || V * H >= INT_MAX ||
                     static_cast<long long>(fp.b.dh_splits) * fp.R * H >= INT_MAX;
  if (compact && dH) FLCE_CUDA_TRY(cudaMemsetAsync(dH, 0, static_cast<size_t>(N) * H * 2, st));
  {
    ProfScope ps(K_DLOGITS, st);
    const long long runs = ceil_div(fp.ldD, TOPK_DL_COLS);
    const int steps = static_cast<int>(std::max<long long>(1, std::min<long long>(4, runs * N / (16LL * device_sms()))));
    ScoreDlogits d{};
    d.h = h;
    d.hc = dW != nullptr || sc.dW16 != nullptr ? hc : nullptr;
    d.H = static_cast<int>(H);
    d.E = reinterpret_cast<const uint16_t*>(state + K.E);
    d.mx = reinterpret_cast<const float*>(state + K.mx);
    d.D = D;
    d.ldD = static_cast<int>(fp.ldD);
    d.ld_mx = static_cast<int>(K.ld_mx);
    d.steps = steps;
    d.rows = Ni;
    d.lo = static_cast<int>(fp.lo);
    d.V = static_cast<int>(V);
    d.ri = idx;
    d.count = count;
    d.targets = targets;
    d.ignore = ignore_index;
    d.zt = reinterpret_cast<const float*>(state + K.zt);
    d.lse = lse;
    d.entropy = sc.entropy;
    d.g_logp = sc.g_logp;
    d.g_entropy = sc.g_entropy;
    d.tf_softcap = tfp.tf_softcap;
    d.tf_a = tfp.tf_a;
    d.tf_b = tfp.tf_b;
    d.tf_d = tfp.tf_d;
    const dim3 grid(static_cast<unsigned>(ceil_div(runs, steps)), static_cast<unsigned>(std::max<long long>(N, fp.lo)));
    auto go = [&](auto kern) { return launch_dependent(kern, grid, SMALL_THREADS, 0, st, d); };
    if (fp.lo > 0)
      FLCE_CUDA_TRY((kLong ? go(score_dlogits_kernel<true, true>) : go(score_dlogits_kernel<false, true>)));
    else
      FLCE_CUDA_TRY((kLong ? go(score_dlogits_kernel<true, false>) : go(score_dlogits_kernel<false, false>)));
  }
  int* err = nullptr;
  FLCE_CUDA_TRY(cudaGetSymbolAddress(reinterpret_cast<void**>(&err), g_device_error));
  const int d_rows = fp.lo > 0 ? static_cast<int>(2 * fp.lo) : Ni;
  CUtensorMap W_mn, B_dw, dW_map, dhp_map, D_k, D_mn;
  if (!make_map(&W_mn, W, H, V, H, 64, BK) || !make_map(&B_dw, hc, H, N, H, 64, BK) ||
      !make_map(&D_k, D, fp.ldD, d_rows, fp.ldD, BK, BM) || !make_map(&D_mn, D, fp.ldD, d_rows, fp.ldD, 64, BK))
    return FLCE_ERR_CUDA;
  if (dW && !make_map_t(&dW_map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, dW, H, V, H, 32, 32)) return FLCE_ERR_CUDA;
  if (sc.dW16 && !make_map(&dW_map, sc.dW16, H, V, H, 64, 32)) return FLCE_ERR_CUDA;
  if (dH && fp.b.dh_f32 &&
      !make_map_t(&dhp_map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, dh_part, H, fp.b.dh_splits * fp.R, H, 32, 32))
    return FLCE_ERR_CUDA;
  GemmParams p{};
  p.N = Ni;
  p.H = static_cast<int>(H);
  p.V = static_cast<int>(V);
  p.ldD = static_cast<int>(fp.ldD);
  p.D = D;
  p.dH = dH;
  p.dH_part = dh_part;
  p.dW = dW;
  p.err = err;
  p.rows = d_rows;
  p.rows_cap = static_cast<int>(fp.R);
  p.row_idx = idx;
  p.dyn_count = count;
  // (dlogits in two parts: both parts' rows, against the rows of h twice; the
  // parts of a dH row are sums of its reduction like the k-splits')
  p.dw_h_blocks = static_cast<int>(fp.lo / BK);
  BwdPlan reduce = fp.b;
  if (fp.lo > 0) {
    reduce.dh_splits *= 2;
    reduce.R = fp.lo;
  }
  const DhDwStage stage{cg, workers, tm, kLong, &fp.b, H, V, dh_part, dH, dW, &W_mn, &dW_map, &dhp_map,
                        sc.dW16 != nullptr};
  DhDwStage finish = stage;
  finish.plan = &reduce;
  const flce_status s = slab_dh_dw(stage, p, d_rows, 0, 0, 0, static_cast<int>(V), D_k, D_mn, B_dw, st);
  if (s != FLCE_OK) return s;
  return block_dh_finish(finish, 0, Ni, idx, count, 0, st);
}

}  // namespace

extern "C" {

size_t flce_score_backward_workspace_bytes(int64_t N, int64_t H, int64_t V, int64_t chunk_rows, int32_t dW_type) {
  const size_t again = flce_topk_kd_backward_workspace_bytes(N, H, V, chunk_rows, dW_type);
  if (again == 0 || !keep_pays(N, H, chunk_rows)) return again;
  const int cg = cta_group();
  return std::max(again, keep_bwd_plan(N, H, V, device_workers(cg), BM * cg).total);
}

flce_status flce_score_backward(const flce_bf16* h, const flce_bf16* W, const int64_t* targets, const float* lse,
                                const float* entropy, const float* g_logp, const float* g_entropy, const void* state,
                                flce_bf16* dH, void* dW, int32_t dW_type, int64_t N, int64_t H, int64_t V,
                                int64_t chunk_rows, int64_t ignore_index, const flce_logit_transform* transform,
                                void* workspace, size_t workspace_bytes, void* stream) {
  if (!topk_sizes_ok(N, H, V) || !topk_dw_ok(dW, dW_type)) return FLCE_ERR_INVALID_ARG;
  GemmParams tfp{};
  if (!transform_params(transform, tfp) || (N > 0 && !dH && !dW)) return FLCE_ERR_INVALID_ARG;
  if (N > 0 && (!h || !W || !targets || !lse || !entropy)) return FLCE_ERR_INVALID_ARG;
  if (H % 8 != 0 || !aligned(dW, 16) || !aligned(dH, 16) || !aligned(h, 16) || !aligned(W, 16) ||
      !aligned(targets, 8) || !aligned(lse, 4) || !aligned(entropy, 4) || !aligned(g_logp, 4) ||
      !aligned(g_entropy, 4) || !aligned(state, 256) || (state && N > kKeepMaxRows))
    return FLCE_ERR_UNSUPPORTED;
  if (N == 0 && !dW) return FLCE_OK;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool bf16 = dW != nullptr && dW_type == FLCE_BF16;
  ScoreGrads sc{entropy, g_logp, g_entropy, nullptr};
  Workspace ws;
  if (state && N > 0) {
    const int cg = cta_group();
    flce_status s = get_workspace(ws, workspace, workspace_bytes,
                                  keep_bwd_plan(N, H, V, device_workers(cg), BM * cg).total, st);
    if (s != FLCE_OK) return s;
    if (bf16) sc.dW16 = static_cast<flce_bf16*>(dW);
    // (the state is read alone)
    return score_backward_kept(h, W, targets, lse, sc, static_cast<uint8_t*>(const_cast<void*>(state)), dH,
                               bf16 ? nullptr : static_cast<float*>(dW), N, H, V, ignore_index, tfp,
                               static_cast<uint8_t*>(ws.ptr), st);
  }
  const TopkGrad tg = topk_grad(dW ? dW_type : FLCE_F32, N, H, V, bf16 ? topk_bwd_rows(N, H, V, chunk_rows) : 0);
  if (bf16 && !tg.scratch) sc.dW16 = static_cast<flce_bf16*>(dW);
  const size_t inner = align256(flce_workspace_bytes(N, H, V, chunk_rows));
  flce_status s = get_workspace(ws, workspace, workspace_bytes, inner + tg.bytes, st);
  if (s != FLCE_OK) return s;
  float* sum = tg.scratch ? reinterpret_cast<float*>(static_cast<uint8_t*>(ws.ptr) + inner)
                          : bf16 ? nullptr : static_cast<float*>(dW);
  s = backward_impl(h, W, targets, nullptr, lse, 1.f, dH, sum, N, H, V, chunk_rows, ignore_index, transform, ws.ptr,
                    inner, stream, nullptr, nullptr, nullptr, &sc);
  if (s != FLCE_OK || !tg.scratch) return s;
  return topk_round_dw(sum, V * H, dW, nullptr, 1.f, st);
}

}  // extern "C"
