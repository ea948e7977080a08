// Argument checks, workspace sizes and launches of the block-sparse path (rotary, block means and
// choice, the 8-bit store, attention over listed blocks).  Part of the library's one translation
// unit: mcs_api.cu includes it after its own helpers.
#pragma once

#include "block_attn.cuh"
#include "block_token.cuh"

namespace {

mcs_status check_block_shape(const mcs_block_shape& s) {
  if (s.B < 1 || s.H < 1 || s.Hkv < 1 || s.Nq < 1 || s.Nk < 1) return MCS_ERR_INVALID_ARG;
  if (s.d != 64 && s.d != 128) return MCS_ERR_SHAPE;
  if (s.H % s.Hkv || static_cast<long long>(s.B) * s.H > 65535) return MCS_ERR_SHAPE;
  // keys and query rows are 32-bit row numbers (TMA coordinates, row counters)
  if (s.Nq > (1 << 24) || s.Nk > (1 << 24) || static_cast<long long>(s.B) * s.H * s.Nq > 0x7FFFFFFFll ||
      static_cast<long long>(s.B) * s.Hkv * s.Nk > 0x7FFFFFFFll)
    return MCS_ERR_SHAPE;
  return MCS_OK;
}
// Launch as a dependent of the kernel before it on the stream: its CTAs may start while that one still
// runs, and wait for its results where they need them (wait_for_results).
template <typename... Params, typename... Args>
void launch_dependent(void (*kernel)(Params...), dim3 grid, unsigned threads, size_t smem, cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

// Does the first span of bytes share any with one of the others?  (The CTAs of a call write in any order.)
struct Span {
  const void* p;  // NULL: none
  size_t bytes;
};
bool shares(const Span& a, std::initializer_list<Span> others) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(a.p), hi = lo + a.bytes;
  for (const Span& o : others) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(o.p);
    if (a.p != nullptr && o.p != nullptr && lo < x + o.bytes && x < hi) return true;
  }
  return false;
}

bool block_rows_ok(int BK) { return BK == 32 || BK == 64 || BK == 128; }
bool query_rows_ok(int C) { return C == 1 || C == 16 || C == 64 || C == 128; }

// Opt-in shared memory, once per device and for the operator that is called.
template <int HD, bool KV8, bool PAIR>
bool block_attn_attrs() {
  // the kernel moves registers between its warpgroups and counts on 128 a thread at launch: a build
  // with another count would wait for registers that never come, so it is refused here
  cudaFuncAttributes fa{};
  return cudaFuncSetAttribute(block_attn_kernel<HD, KV8, PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              BlockSmem<HD, KV8>::BYTES) == cudaSuccess &&
         cudaFuncGetAttributes(&fa, block_attn_kernel<HD, KV8, PAIR>) == cudaSuccess &&
         static_cast<long long>(fa.numRegs) * kAttnThreads == 65536;
}
template <int HD, bool KV8>
bool block_token_attrs() {
  constexpr int bytes = TokenSmem<HD, KV8>::BYTES;
  return cudaFuncSetAttribute(block_token_kernel<HD, KV8, 8>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess &&
         cudaFuncSetAttribute(block_token_kernel<HD, KV8, 16>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess;
}
mcs_status topk_device(DeviceInfo** out) {
  mcs_status e = current_device(out);
  if (e != MCS_OK) return e;
  std::lock_guard<std::mutex> lock(g_mu);
  if (!(*out)->topk_attrs_set) {
    if (cudaFuncSetAttribute(block_pick_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kTopkMaxBlocks * 8) != cudaSuccess)
      return MCS_ERR_CUDA;
    (*out)->topk_attrs_set = true;
  }
  return MCS_OK;
}
mcs_status block_attn_device(DeviceInfo** out) {
  mcs_status e = current_device(out);
  if (e != MCS_OK) return e;
  std::lock_guard<std::mutex> lock(g_mu);
  if (!(*out)->block_attrs_set) {
    if (!block_token_attrs<64, false>() || !block_token_attrs<64, true>() || !block_token_attrs<128, false>() ||
        !block_token_attrs<128, true>() || !block_attn_attrs<64, false, false>() || !block_attn_attrs<64, false, true>() ||
        !block_attn_attrs<64, true, false>() || !block_attn_attrs<64, true, true>() ||
        !block_attn_attrs<128, false, false>() || !block_attn_attrs<128, false, true>() ||
        !block_attn_attrs<128, true, false>() || !block_attn_attrs<128, true, true>())
      return MCS_ERR_CUDA;
    (*out)->block_attrs_set = true;
  }
  return MCS_OK;
}

// How a call of mcs_block_attn runs; a function of its sizes alone, so that the workspace's size and the
// launch agree.  Without lists every query head of a key/value head attends to the same keys: their
// rows, which lie one behind the other, count as one head's.
struct BlockPlan {
  bool tensor;       // the tcgen05 kernel (else the one for few rows)
  bool pair;         // lists of 64 rows: two to a tile
  int H, Nq, C, GQ;  // as the kernel sees them
  int tiles, splits;
  size_t part, total;  // workspace: bytes of the parts' results, and all
};
constexpr int kPlanSms = 148;

BlockPlan plan_block_attn(const mcs_block_shape& s, int C, int BK, int kb, bool listed, bool kv8) {
  BlockPlan q{};
  q.H = listed ? s.H : s.Hkv;
  q.Nq = listed ? s.Nq : s.Nq * (s.H / s.Hkv);
  q.C = C;
  // Lists of 64 and 128 rows fill a tile; those of 1 and 16 do not.  Without lists the few-row kernel reads
  // the store once for every 16 rows and the tiles once for every 128, but the latter start and end
  // slower.  us, few rows | tiles, for B Hkv Nk key rows of 128 (64 for 30 k): bf16, 256 k keys, 8 rows 31 | 28,
  // 16 rows 42 | 29, 64 rows 107 | 30; 30 k keys, 16 rows 14 | 20, 64 rows 21 | 21, 128 rows 25 | 22; 2 k keys,
  // 128 rows 11 | 16.  8 bits: 960 k keys, 16 rows 77 | 103, 24 rows 123 | 104; 256 k keys, 16 rows 39 | 37,
  // 24 rows 51 | 37; 30 k keys, 64 rows 20 | 22, 128 rows 29 | 23.
  // (Lists of 16 rows have no other form: tiles of 128 rows would be an eighth full.  They read their keys once for
  // 16 rows: a clip of 24 heads, 37 of 252 blocks, 15.8 ms where lists of 128 rows take 2.0.)
  const long long reads = static_cast<long long>(s.B) * s.Hkv * s.Nk * ((q.Nq + 15) / 16);
  q.tensor = listed ? C >= 64 : q.Nq > (kv8 ? 16 : 8) && reads >= 131072;
  q.pair = q.tensor && listed && C == 64;
  if (!listed && !q.tensor) q.C = 16;
  q.GQ = (q.Nq + q.C - 1) / q.C;
  q.tiles = (q.Nq + kTile - 1) / kTile;
  q.splits = 1;
  const long long lists = static_cast<long long>(s.B) * q.H * (q.tensor ? q.tiles : q.GQ);
  if (q.tensor) {
    if (!q.pair) q.GQ = q.tiles;
    // Few tiles: the keys of a tile are split over several CTAs.  The cost of a choice, in stages of
    // 128 keys: waves times (the part's stages and about three of start and end), and six for the
    // join's launch.
    const int T = static_cast<int>((static_cast<long long>(kb) * BK + kTile - 1) / kTile);
    long long best = -1;
    for (int n = 1; n <= 32 && (n == 1 || T / n >= 4); ++n) {
      const long long cost = (lists * n + kPlanSms - 1) / kPlanSms * ((T + n - 1) / n + 3) + (n > 1 ? 6 : 0);
      if (best < 0 || cost < best) best = cost, q.splits = n;
    }
  } else {
    // Few lists: one wave of CTAs (32 lists of 8 k keys: 13 parts 21 us, 28 parts 25), else two or more, which
    // evens out lists of unlike lengths (192 lists of 10 k keys, a quarter of them past the end: 2 and 4
    // parts 97 us, 5 parts 89, 6 parts 94); each part has at least 256 keys.
    const long long keys = static_cast<long long>(kb) * BK;
    const long long wave = kPlanSms * (std::min(q.C, q.Nq) <= 8 ? 3 : 2);
    const long long n = lists * 4 <= wave ? wave / lists : (2 * wave + lists - 1) / lists;
    q.splits = static_cast<int>(std::max(1ll, std::min({n, keys / 256, 128ll})));
  }
  const size_t rows = static_cast<size_t>(s.B) * s.H * s.Nq;
  if (q.splits > 1) q.part = round_up(rows * q.splits * s.d * 4, 256);
  q.total = q.part + (q.splits > 1 ? round_up(rows * q.splits * 4, 256) : 256);
  return q;
}

// Parts of split lists, joined behind the kernel that wrote them.
template <int HD>
void join_parts(const BlockAttnParams& p, cudaStream_t st) {
  if (p.splits == 1) return;
  const long long rows = static_cast<long long>(p.B) * p.H * p.Nq;
  constexpr int per = 256 / (HD / 4) / kJoinGroups;
  launch_dependent(block_join_kernel<HD>, dim3(static_cast<unsigned>((rows + per - 1) / per)), 256, 0, st, p);
}

template <int HD>
mcs_status run_block_token(const BlockAttnParams& p, bool kv8, cudaStream_t st) {
  const unsigned grid = static_cast<unsigned>(static_cast<long long>(p.B) * p.H * p.GQ * p.splits);
  const bool few = std::min(p.C, p.Nq) <= 8;
  constexpr unsigned threads = kTokenWarps * 32;
  constexpr size_t b16 = TokenSmem<HD, false>::BYTES, b8 = TokenSmem<HD, true>::BYTES;
  if (kv8 && few) block_token_kernel<HD, true, 8><<<grid, threads, b8, st>>>(p);
  else if (kv8) block_token_kernel<HD, true, 16><<<grid, threads, b8, st>>>(p);
  else if (few) block_token_kernel<HD, false, 8><<<grid, threads, b16, st>>>(p);
  else block_token_kernel<HD, false, 16><<<grid, threads, b16, st>>>(p);
  join_parts<HD>(p, st);
  return launch_status();
}

template <int HD, bool KV8, bool PAIR>
mcs_status run_block_attn(const BlockAttnParams& p, cudaStream_t st, int sms) {
  alignas(64) CUtensorMap tmQ, tmK, tmV;
  if (!make_row_map(&tmQ, p.Q, static_cast<uint64_t>(p.B) * p.H * p.Nq, HD, kTile)) return MCS_ERR_CUDA;
  if (KV8) {
    tmK = tmV = tmQ;  // not used: 8-bit rows come by bulk copies
  } else {
    const uint64_t rows = static_cast<uint64_t>(p.B) * p.Hkv * p.Nk;
    if (!make_row_map(&tmK, p.K, rows, HD, p.BK) || !make_row_map(&tmV, p.V, rows, HD, p.BK)) return MCS_ERR_CUDA;
  }
  block_attn_kernel<HD, KV8, PAIR><<<std::min(p.num_units, sms), kAttnThreads, BlockSmem<HD, KV8>::BYTES, st>>>(tmQ, tmK, tmV, p);
  join_parts<HD>(p, st);
  return launch_status();
}
template <int HD>
mcs_status run_block_attn(const BlockAttnParams& p, bool kv8, bool pair, cudaStream_t st, int sms) {
  if (kv8) return pair ? run_block_attn<HD, true, true>(p, st, sms) : run_block_attn<HD, true, false>(p, st, sms);
  return pair ? run_block_attn<HD, false, true>(p, st, sms) : run_block_attn<HD, false, false>(p, st, sms);
}

void launch_means(int d, const __nv_bfloat16* X, const int32_t* len, float* means, int B, int H, int N, int BK,
                  cudaStream_t st) {
  MeansParams p{};
  p.X = X;
  p.len = len;
  p.means = means;
  p.H = H;
  p.N = N;
  p.BK = BK;
  p.nb = (N + BK - 1) / BK;
  p.blocks = static_cast<long long>(B) * H * p.nb;
  const unsigned grid = static_cast<unsigned>(p.blocks);
  if (d == 64) block_means_kernel<64><<<grid, kMeansThreads, 0, st>>>(p);
  else block_means_kernel<128><<<grid, kMeansThreads, 0, st>>>(p);
}

// Workspace of mcs_block_topk: the score keys of as many rows as kTopkKeyBytes hold (all of them in most
// calls; else the rows are worked off in parts, whole key heads or row ranges of one), then the mean
// query rows.
struct TopkPlan {
  int M, kv_step, m_step;  // rows of a key head; key heads and rows of each in one part
  size_t keys, total;
};
constexpr size_t kTopkKeyBytes = size_t{1} << 28;


TopkPlan plan_topk(const mcs_block_shape& s, int C, int BK) {
  TopkPlan q{};
  const int GQ = (s.Nq + C - 1) / C, kvs = s.B * s.Hkv;
  const size_t row = static_cast<size_t>((s.Nk + BK - 1) / BK) * 8;
  q.M = s.H / s.Hkv * GQ;
  const size_t fit = std::min<size_t>(std::max<size_t>(64, kTopkKeyBytes / row), size_t{1} << 21);  // rows (and grid)
  q.kv_step = static_cast<int>(std::min<size_t>(kvs, std::max<size_t>(1, fit / q.M)));
  q.m_step = static_cast<int>(std::min<size_t>(q.M, fit));
  q.keys = round_up(row * q.kv_step * q.m_step, 256);
  q.total = q.keys + (C > 1 ? round_up(static_cast<size_t>(s.B) * s.H * GQ * s.d * 4, 256) : 0);
  return q;
}

template <int HD>
void launch_topk(const TopkParams& p, int kvs, cudaStream_t st) {
  const unsigned few = static_cast<unsigned>((p.nb + kFewBlocks - 1) / kFewBlocks);
  const unsigned tiles = static_cast<unsigned>((p.nb + kScoreTile - 1) / kScoreTile);
  const unsigned mtiles = static_cast<unsigned>((p.mc + kScoreTile - 1) / kScoreTile);
  // few rows: the tile form would spend its 64 rows on them (3 rows, 64 key heads: 30 us against 8)
  const bool first = p.qbar == nullptr;  // nothing of this call runs before it
  if (p.mc <= kFewRows) {
    if (first) block_score_few_kernel<HD><<<dim3(few, 1, kvs), 128, 0, st>>>(p);
    else launch_dependent(block_score_few_kernel<HD>, dim3(few, 1, kvs), 128, 0, st, p);
  } else {
    if (first) block_score_kernel<HD><<<dim3(tiles, mtiles, kvs), kScoreThreads, 0, st>>>(p);
    else launch_dependent(block_score_kernel<HD>, dim3(tiles, mtiles, kvs), kScoreThreads, 0, st, p);
  }
  const long long rows = static_cast<long long>(kvs) * p.mc;
  const unsigned grid = static_cast<unsigned>((rows + 3) / 4);
  // a warp a row wherever its keys fit in registers (50 rows of 250: 12.5 us for the whole choice against 13.9
  // with a CTA a row, 2000 rows of 1000: 52 against 71)
  if (p.nb <= 8 * 32) launch_dependent(block_pick_warp_kernel<8>, grid, 128, 0, st, p, rows);
  else if (p.nb <= 16 * 32) launch_dependent(block_pick_warp_kernel<16>, grid, 128, 0, st, p, rows);
  else if (p.nb <= 32 * 32) launch_dependent(block_pick_warp_kernel<32>, grid, 128, 0, st, p, rows);
  else
    launch_dependent(block_pick_kernel, static_cast<unsigned>(std::min<long long>(rows, 4096)), kTopkThreads,
                     static_cast<size_t>(p.nb) * 8, st, p, rows);
}

template <int HD, int NORM>
void launch_rotary(const RotaryParams& p, bool halves, cudaStream_t st) {
  const unsigned grid = static_cast<unsigned>(p.B) * static_cast<unsigned>(p.tiles);
  if (halves) rotary_kernel<HD, NORM, true><<<grid, kRotThreads, 0, st>>>(p);
  else rotary_kernel<HD, NORM, false><<<grid, kRotThreads, 0, st>>>(p);
}
template <int HD>
void launch_rotary(const RotaryParams& p, int norm, bool halves, cudaStream_t st) {
  if (norm == kNormNone) launch_rotary<HD, kNormNone>(p, halves, st);
  else if (norm == kNormHead) launch_rotary<HD, kNormHead>(p, halves, st);
  else launch_rotary<HD, kNormToken>(p, halves, st);
}

}  // namespace

extern "C" {

mcs_status mcs_rotary(const mcs_rotary_args* a, const void* q, const void* k, const void* v, const void* pos,
                      const void* q_weight, const void* k_weight, void* Q, void* K, void* V, void* stream) {
  if (!a) return MCS_ERR_INVALID_ARG;
  if (a->B < 1 || a->N < 1 || a->H < 1 || a->Hkv < 1) return MCS_ERR_INVALID_ARG;
  if (a->d != 64 && a->d != 128) return MCS_ERR_SHAPE;
  if (a->N > (1 << 24) || static_cast<long long>(a->B) * a->N > 0x7FFFFFFFll || a->H > 65535 || a->Hkv > 65535)
    return MCS_ERR_SHAPE;
  if (a->axes < 1 || a->axes > kRotMaxAxes || a->norm < kNormNone || a->norm > kNormToken ||
      (a->pairs != 0 && a->pairs != 1) || !(a->theta > 0) || !(a->theta < 1e300) || !(a->eps >= 0.f) ||
      !(a->eps < 3e38f))
    return MCS_ERR_INVALID_ARG;
  int sum = 0;
  for (int i = 0; i < a->axes; ++i) {
    if (a->axis_dim[i] < 2 || a->axis_dim[i] % 2) return MCS_ERR_SHAPE;
    sum += a->axis_dim[i];
    if (sum > a->d) return MCS_ERR_SHAPE;
  }
  if (a->pairs == 1 && sum % 16) return MCS_ERR_SHAPE;  // the halves meet on an 8-element boundary
  if (!q || !Q || !pos || !k != !K || !v != !V) return MCS_ERR_INVALID_ARG;
  const void* src[3] = {q, k, v};
  void* dst[3] = {Q, K, V};
  for (int s = 0; s < 3; ++s) {
    if (!src[s]) continue;
    if (!aligned16(src[s]) || !aligned16(dst[s])) return MCS_ERR_DTYPE_ALIGN;
    for (int i = 0; i < 3; ++i) {
      if (a->stride[s][i] < 0) return MCS_ERR_INVALID_ARG;
      if (a->stride[s][i] % 8) return MCS_ERR_DTYPE_ALIGN;
    }
  }
  if ((q_weight && !aligned16(q_weight)) || (k_weight && !aligned16(k_weight)) || (reinterpret_cast<uintptr_t>(pos) & 3u))
    return MCS_ERR_DTYPE_ALIGN;
  DeviceInfo* di = nullptr;
  mcs_status e = current_device(&di);
  if (e != MCS_OK) return e;
  RotaryParams p{};
  for (int s = 0; s < 3; ++s) {
    p.x[s] = static_cast<const __nv_bfloat16*>(src[s]);
    p.y[s] = static_cast<__nv_bfloat16*>(dst[s]);
    p.sb[s] = a->stride[s][0];
    p.sn[s] = a->stride[s][1];
    p.sh[s] = a->stride[s][2];
    p.heads[s] = s == 0 ? a->H : a->Hkv;
  }
  p.w[0] = q_weight;
  p.w[1] = k_weight;
  p.pos = pos;
  // the frequencies of a model's layers are the same call after call: the last table of this thread is kept
  // (64 powers take longer than the rest of a small call's host work)
  struct Table {
    double theta = 0, turns[64];
    int axes = 0, dim[kRotMaxAxes], half = 0;
    unsigned char axis[64];
  };
  static thread_local Table tab;
  if (tab.axes != a->axes || tab.theta != a->theta || std::memcmp(tab.dim, a->axis_dim, sizeof(int) * a->axes) != 0) {
    constexpr double kTwoPi = 6.283185307179586476925;
    tab.half = 0;
    for (int i = 0; i < a->axes; ++i)
      for (int j = 0; j < a->axis_dim[i] / 2; ++j, ++tab.half) {
        tab.turns[tab.half] = std::pow(a->theta, -2.0 * j / a->axis_dim[i]) / kTwoPi;
        tab.axis[tab.half] = static_cast<unsigned char>(i);
      }
    tab.theta = a->theta;
    tab.axes = a->axes;
    std::memcpy(tab.dim, a->axis_dim, sizeof(int) * a->axes);
  }
  const int at = tab.half;
  std::memcpy(p.turns, tab.turns, sizeof(double) * at);
  std::memcpy(p.axis, tab.axis, at);
  p.B = a->B;
  p.N = a->N;
  p.A = a->axes;
  p.half = at;
  p.pos_float = a->pos_is_float != 0;
  p.pos_batch = a->pos_per_batch != 0;
  p.w_bf16 = a->weight_is_bf16 != 0;
  p.eps = a->eps;
  // a token for every group of lanes of a CTA, fewer tokens, and a token's heads shared among groups, where
  // that leaves SMs idle
  p.T = kRotThreads / (a->d / 8);
  while (p.T > 1 && static_cast<long long>(a->B) * ((a->N + p.T - 1) / p.T) < 2ll * di->sms) p.T /= 2;
  p.tiles = (a->N + p.T - 1) / p.T;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (a->d == 64) launch_rotary<64>(p, a->norm, a->pairs == 1, st);
  else launch_rotary<128>(p, a->norm, a->pairs == 1, st);
  return launch_status();
}

mcs_status mcs_block_means(mcs_shape s, const void* X, int BK, const int32_t* len, float* means, void* stream) {
  mcs_status e = check_shape(s);
  if (e != MCS_OK) return e;
  if (!block_rows_ok(BK)) return MCS_ERR_SHAPE;
  if (!X || !means) return MCS_ERR_INVALID_ARG;
  if (!aligned16(X) || !aligned16(means) || (reinterpret_cast<uintptr_t>(len) & 3u)) return MCS_ERR_DTYPE_ALIGN;
  DeviceInfo* di = nullptr;
  if ((e = current_device(&di)) != MCS_OK) return e;
  launch_means(s.d, static_cast<const __nv_bfloat16*>(X), len, means, s.B, s.H, s.N, BK, static_cast<cudaStream_t>(stream));
  return launch_status();
}

size_t mcs_block_topk_workspace_size(mcs_block_shape s, int C, int BK) {
  if (check_block_shape(s) != MCS_OK || !query_rows_ok(C) || !block_rows_ok(BK) || (s.Nk + BK - 1) / BK > kTopkMaxBlocks)
    return 0;
  return plan_topk(s, C, BK).total;
}

mcs_status mcs_block_topk(mcs_block_shape s, const void* Q, const float* means, int C, int BK, int kb,
                          const int32_t* kv_len, int32_t* blocks, void* ws, size_t ws_bytes, void* stream) {
  mcs_status e = check_block_shape(s);
  if (e != MCS_OK) return e;
  if (!query_rows_ok(C) || !block_rows_ok(BK) || (s.Nk + BK - 1) / BK > kTopkMaxBlocks) return MCS_ERR_SHAPE;
  const int nb = (s.Nk + BK - 1) / BK;
  if (kb < 1 || kb > nb || !Q || !means || !blocks) return MCS_ERR_INVALID_ARG;
  if (!aligned16(Q) || !aligned16(means) || (reinterpret_cast<uintptr_t>(blocks) & 3u) ||
      (reinterpret_cast<uintptr_t>(kv_len) & 3u))
    return MCS_ERR_DTYPE_ALIGN;
  if (!ws || ws_bytes < mcs_block_topk_workspace_size(s, C, BK)) return MCS_ERR_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(ws) & 255u) return MCS_ERR_DTYPE_ALIGN;
  DeviceInfo* di = nullptr;
  if ((e = topk_device(&di)) != MCS_OK) return e;
  const TopkPlan plan = plan_topk(s, C, BK);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  TopkParams p{};
  p.Q = static_cast<const __nv_bfloat16*>(Q);
  p.means = means;
  p.len = kv_len;
  p.keys = static_cast<unsigned long long*>(ws);
  p.blocks = blocks;
  p.Hkv = s.Hkv;
  p.Nk = s.Nk;
  p.M = plan.M;
  p.BK = BK;
  p.nb = nb;
  p.kb = kb;
  if (C > 1) {
    float* qbar = reinterpret_cast<float*>(static_cast<char*>(ws) + plan.keys);
    p.qbar = qbar;
    launch_means(s.d, p.Q, nullptr, qbar, s.B, s.H, s.Nq, C, st);
  }
  const int kvs = s.B * s.Hkv;
  for (int kv = 0; kv < kvs; kv += plan.kv_step)
    for (int m = 0; m < plan.M; m += plan.m_step) {
      p.kv0 = kv;
      p.m0 = m;
      p.mc = std::min(plan.m_step, plan.M - m);
      const int kn = std::min(plan.kv_step, kvs - kv);
      if (s.d == 64) launch_topk<64>(p, kn, st);
      else launch_topk<128>(p, kn, st);
    }
  return launch_status();
}

mcs_status mcs_cache_write(mcs_shape s, const void* K, const void* V, int BK, int start, int capacity,
                           const int32_t* len, void* K8, void* V8, float* k_scale, float* v_scale, float* means,
                           void* stream) {
  mcs_status e = check_shape(s);
  if (e != MCS_OK) return e;
  if (!block_rows_ok(BK) || capacity < 1 || capacity % BK || capacity > (1 << 24) ||
      static_cast<long long>(s.B) * s.H * capacity > 0x7FFFFFFFll)
    return MCS_ERR_SHAPE;
  if (start < 0 || start % BK || static_cast<long long>(start) + s.N > capacity) return MCS_ERR_INVALID_ARG;
  if (!K || !V || !K8 || !V8 || !k_scale || !v_scale) return MCS_ERR_INVALID_ARG;
  if (!aligned16(K) || !aligned16(V) || !aligned16(K8) || !aligned16(V8) || !aligned16(k_scale) || !aligned16(v_scale) ||
      (means && !aligned16(means)) || (reinterpret_cast<uintptr_t>(len) & 3u))
    return MCS_ERR_DTYPE_ALIGN;
  {
    const size_t heads = static_cast<size_t>(s.B) * s.H, blocks = heads * (capacity / BK);
    const Span k{K, heads * s.N * s.d * 2}, v{V, k.bytes}, l{len, static_cast<size_t>(s.B) * 4};
    const Span k8{K8, heads * capacity * s.d}, v8{V8, k8.bytes}, ks{k_scale, blocks * 4}, vs{v_scale, ks.bytes};
    const Span m{means, blocks * s.d * 4};
    if (shares(k8, {k, v, l, v8, ks, vs, m}) || shares(v8, {k, v, l, ks, vs, m}) || shares(ks, {k, v, l, vs, m}) ||
        shares(vs, {k, v, l, m}) || shares(m, {k, v, l}))
      return MCS_ERR_INVALID_ARG;
  }
  DeviceInfo* di = nullptr;
  if ((e = current_device(&di)) != MCS_OK) return e;
  CacheWriteParams p{};
  p.X[0] = static_cast<const __nv_bfloat16*>(K);
  p.X[1] = static_cast<const __nv_bfloat16*>(V);
  p.Y[0] = static_cast<uint8_t*>(K8);
  p.Y[1] = static_cast<uint8_t*>(V8);
  p.scale[0] = k_scale;
  p.scale[1] = v_scale;
  p.means = means;
  p.len = len;
  p.H = s.H;
  p.n = s.N;
  p.cap = capacity;
  p.start = start;
  p.BK = BK;
  p.nb = (s.N + BK - 1) / BK;
  const dim3 grid(p.nb, s.B * s.H, 2);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  constexpr int R64 = kCacheThreads / (64 / 16), R128 = kCacheThreads / (128 / 16);  // rows of a pass
  if (s.d == 64) {
    if (BK <= R64) cache_write_kernel<64, 1><<<grid, kCacheThreads, 0, st>>>(p);
    else cache_write_kernel<64, 128 / R64><<<grid, kCacheThreads, 0, st>>>(p);
  } else if (BK <= R128) {
    cache_write_kernel<128, 1><<<grid, kCacheThreads, 0, st>>>(p);
  } else if (BK <= 2 * R128) {
    cache_write_kernel<128, 2><<<grid, kCacheThreads, 0, st>>>(p);
  } else {
    cache_write_kernel<128, 128 / R128><<<grid, kCacheThreads, 0, st>>>(p);
  }
  return launch_status();
}

size_t mcs_block_attn_workspace_size(mcs_block_shape s, int C, int BK, int kb) {
  if (check_block_shape(s) != MCS_OK || !query_rows_ok(C) || !block_rows_ok(BK) || kb < 1 || kb > (s.Nk + BK - 1) / BK)
    return 0;
  const size_t n = plan_block_attn(s, C, BK, kb, true, false).total;
  if (kb < (s.Nk + BK - 1) / BK) return n;
  return std::max({n, plan_block_attn(s, C, BK, kb, false, false).total, plan_block_attn(s, C, BK, kb, false, true).total});
}

mcs_status mcs_block_attn(mcs_block_shape s, const void* Q, const void* K, const void* V, int kv_format,
                          const float* k_scale, const float* v_scale, const int32_t* blocks, int C, int BK, int kb,
                          const int32_t* kv_len, const void* R, void* out, float* lse, void* ws, size_t ws_bytes,
                          void* stream) {
  mcs_status e = check_block_shape(s);
  if (e != MCS_OK) return e;
  if (!query_rows_ok(C) || !block_rows_ok(BK)) return MCS_ERR_SHAPE;
  const int nb = (s.Nk + BK - 1) / BK;
  if (kb < 1 || kb > nb || (!blocks && kb != nb) || (kv_format != 0 && kv_format != 1)) return MCS_ERR_INVALID_ARG;
  if (kv_format == 1 && s.Nk % BK) return MCS_ERR_SHAPE;
  if (!Q || !K || !V || !out || (kv_format == 1) != (k_scale != nullptr) || (kv_format == 1) != (v_scale != nullptr))
    return MCS_ERR_INVALID_ARG;
  if (!aligned16(Q) || !aligned16(K) || !aligned16(V) || !aligned16(out) || (R && !aligned16(R)) ||
      (reinterpret_cast<uintptr_t>(lse) & 3u) || (reinterpret_cast<uintptr_t>(blocks) & 3u) ||
      (reinterpret_cast<uintptr_t>(kv_len) & 3u) || (reinterpret_cast<uintptr_t>(k_scale) & 3u) ||
      (reinterpret_cast<uintptr_t>(v_scale) & 3u))
    return MCS_ERR_DTYPE_ALIGN;
  if (!ws || ws_bytes < mcs_block_attn_workspace_size(s, C, BK, kb)) return MCS_ERR_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(ws) & 255u) return MCS_ERR_DTYPE_ALIGN;
  DeviceInfo* di = nullptr;
  if ((e = block_attn_device(&di)) != MCS_OK) return e;
  BlockAttnParams p{};
  p.Q = static_cast<const __nv_bfloat16*>(Q);
  p.K = K;
  p.V = V;
  p.ks = k_scale;
  p.vs = v_scale;
  p.blocks = blocks;
  p.len = kv_len;
  p.R = static_cast<const __nv_bfloat16*>(R);
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  const BlockPlan plan = plan_block_attn(s, C, BK, kb, blocks != nullptr, kv_format != 0);
  p.part = static_cast<float*>(ws);
  p.plse = reinterpret_cast<float*>(static_cast<char*>(ws) + plan.part);
  p.B = s.B;
  p.H = plan.H;
  p.Hkv = s.Hkv;
  p.Nq = plan.Nq;
  p.Nk = s.Nk;
  p.C = plan.C;
  p.BK = BK;
  p.nb = nb;
  p.GQ = plan.GQ;
  p.kb = kb;
  p.tiles = plan.tiles;
  p.splits = plan.splits;
  p.num_units = static_cast<int>(static_cast<long long>(s.B) * plan.H * plan.tiles * plan.splits);
  p.scale_log2 = (s.scale > 0.f ? s.scale : 1.0f / std::sqrt(static_cast<float>(s.d))) * kLog2e;
  p.wait_ns = g_attn_wait_ns.load();
  p.hold = g_attn_hold.load();
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (plan.tensor)
    return s.d == 64 ? run_block_attn<64>(p, kv_format != 0, plan.pair, st, di->sms)
                     : run_block_attn<128>(p, kv_format != 0, plan.pair, st, di->sms);
  return s.d == 64 ? run_block_token<64>(p, kv_format != 0, st) : run_block_token<128>(p, kv_format != 0, st);
}

}  // extern "C"
