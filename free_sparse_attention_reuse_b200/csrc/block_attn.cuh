// Attention over listed key blocks: for query row i of query block g,
//   o_i = sum_j softmax_j(scale q_i . k_j) v_j (+ R_i),   lse_i = log sum_j exp(scale q_i . k_j),
// j over the valid keys of the blocks that g lists.  A list ends at its first negative entry; without
// lists every block counts.  Keys and values are bf16, or e4m3 with one fp32 scale for each block of
// tokens and head (value = e4m3 * scale).  A row without a key gives 0 (+ R) and -inf.
#pragma once

#include "blocks.cuh"

namespace mcs {

struct BlockAttnParams {
  const __nv_bfloat16* Q;   // [B, H, Nq, d]
  const void* K;            // [B, Hkv, Nk, d], bf16 or e4m3
  const void* V;
  const float* ks;          // [B, Hkv, nb], e4m3 only
  const float* vs;
  const int32_t* blocks;    // [B, H, GQ, kb], nullable
  const int32_t* len;       // [B], nullable
  const __nv_bfloat16* R;   // [B, H, Nq, d], nullable
  __nv_bfloat16* out;       // [B, H, Nq, d]
  float* lse;               // [B, H, Nq], nullable
  float* part;              // [splits, B * H * Nq, d]: normalised partial results (splits > 1)
  float* plse;              // [splits, B * H * Nq]: their log-sum-exps in base 2
  int B, H, Hkv, Nq, Nk, C, BK, nb, GQ, kb;
  int tiles, splits, num_units;  // query tiles of a head; parts of a tile's keys; B * H * tiles * splits
  float scale_log2;              // scale * log2(e)
  unsigned long long wait_ns;    // bound on any single wait of this launch (nanoseconds)
  const uint32_t* hold;          // test hook (normally NULL): wait for *hold != 0 before any MMA
};

// ---------------------------------------------------------------------------------- tensor-core form
// A warp's walk over the usable entries of one list: block numbers within the store that hold a valid
// key, up to the first negative entry.  Lane l holds the l-th usable entry at hand, so that a stage's
// blocks are one shuffle away; 28 raw entries at a time are packed behind the (at most three) left
// over, with the next 28 fetched ahead.
struct ListWalk {
  static constexpr int WINDOW = 28;
  const int32_t* list;  // nullable: every block in turn
  int kb, nb, bk_log, len;
  int w0, raw;          // next window's first entry, and this lane's entry of it
  int cur, have, at;    // this lane's packed entry; how many there are; how many are taken
  bool end;             // no further window

  __device__ __forceinline__ int fetch() const {
    const int l = lane_id(), i = w0 + l;
    return l >= WINDOW || i >= kb ? -1 : list != nullptr ? list[i] : i;
  }
  // Usable lanes of the fetched window; moves on to the next.
  __device__ __forceinline__ uint32_t window(bool report) {
    constexpr uint32_t FULL = (1u << WINDOW) - 1u;
    const uint32_t neg = __ballot_sync(0xffffffffu, raw < 0) & FULL;
    const int upto = neg ? __ffs(neg) - 1 : WINDOW;
    const bool in = static_cast<int>(lane_id()) < upto;
    if (report && in && raw >= nb) raise_status(kStatusBadIndex);
    const uint32_t mask = __ballot_sync(0xffffffffu, in && raw < nb && (static_cast<long long>(raw) << bk_log) < len);
    end = neg != 0;
    w0 += WINDOW;
    return mask;
  }
  __device__ __forceinline__ void begin() {
    w0 = have = at = 0;
    end = false;
    raw = fetch();
  }
  // Usable entries of the whole list.
  __device__ __forceinline__ int count(bool report) {
    int n = 0;
    begin();
    while (!end) {
      n += __popc(window(report));
      if (!end) raw = fetch();
    }
    return n;
  }
  __device__ __forceinline__ void refill() {
    const int id = raw;
    uint32_t mask = window(false);
    if (!end) raw = fetch();
    const int left = have - at, n = __popc(mask);
    // the entry of rank l - left among the window's usable ones: its lane by halving
    int rank = static_cast<int>(lane_id()) - left, src = 0;
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) {
      const int c = __popc((mask >> src) & ((1u << s) - 1u));
      if (rank >= c) rank -= c, src += s;
    }
    const int old = __shfl_sync(0xffffffffu, cur, (at + static_cast<int>(lane_id())) & 31);
    const int fresh = __shfl_sync(0xffffffffu, id, src & 31);
    cur = static_cast<int>(lane_id()) < left ? old : fresh;
    have = left + n;
    at = 0;
  }
  // Start at usable entry `lo`.
  __device__ __forceinline__ void start(int lo) {
    cur = 0;
    begin();
    while (lo > 0) {
      const int n = min(lo, have - at);
      at += n;
      lo -= n;
      if (lo > 0) {
        if (end) return;
        refill();
      }
    }
  }
  // Have `n` <= 4 entries at hand if the list has them.
  __device__ __forceinline__ void ensure(int n) {
    while (have - at < n && !end) refill();
  }
};

// Valid keys, and scales, of a stage's four runs of 32 keys (each within one block).
struct StageInfo {
  int valid[4];
  float ks[4], vs[4];
};

template <int HD, bool KV8>
struct BlockSmem {
  static constexpr uint32_t TILE_BYTES = kTile * HD * 2;
  static constexpr int KST = KV8 ? (HD == 128 ? 2 : 4) : (HD == 128 ? 3 : 6);  // K ring
  static constexpr int VST = KST;                                            // V ring
  static constexpr uint32_t RAW_BYTES = kTile * HD;                            // an 8-bit tile before it is widened
  static constexpr int RAWS = KV8 ? (HD == 128 ? 4 : 8) : 0;                   // ring of those, K and V in turn
  static constexpr int INFOS = KV8 ? 8 : KST;
  static constexpr uint32_t Q_OFF = 0;
  static constexpr uint32_t K_OFF = Q_OFF + TILE_BYTES;
  static constexpr uint32_t V_OFF = K_OFF + KST * TILE_BYTES;
  static constexpr uint32_t RAW_OFF = V_OFF + VST * TILE_BYTES;
  static constexpr uint32_t XCH_OFF = RAW_OFF + RAWS * RAW_BYTES;  // 2 streams x 128 rows x (m, l)
  static constexpr uint32_t INFO_OFF = XCH_OFF + 2 * kTile * 8;    // StageInfo[INFOS]
  static constexpr uint32_t UNIT_OFF = INFO_OFF + INFOS * sizeof(StageInfo);  // stages of both streams, 4 units
  static constexpr uint32_t BAR_OFF = UNIT_OFF + 4 * 8;
  // q_full, q_empty, k_full[KST], k_empty[KST], v_full[VST], v_empty[VST]; per stream s_full, p_full,
  // pv_done, p_half, pvlo_done, s_hi; o_empty, drain, vfix[2], pair[4], u_full[4], raw_full[RAWS], raw_empty[RAWS]
  static constexpr int NBAR = 2 + 2 * KST + 2 * VST + 12 + 4 + 4 + 4 + 2 * RAWS;
  static constexpr uint32_t MISC_OFF = BAR_OFF + NBAR * 8;
  static constexpr uint32_t QEXP_OFF = MISC_OFF + 16;  // 8-bit form: exponents of Q's rows, two units
  static constexpr uint32_t BYTES = QEXP_OFF + (KV8 ? 2 * kTile : 0);
  static_assert(BAR_OFF % 8 == 0 && INFO_OFF % 16 == 0, "shared memory alignment");
  static_assert(BYTES <= 232448, "shared memory budget");
};

// Registers a thread: softmax (two warpgroups), producers, MMA (the 8-bit form's loader is one of its warps).
template <bool KV8>
struct BlockRegs {
  static constexpr uint32_t SOFTMAX = KV8 ? 184 : 192, PRODUCER = 80, MMA = KV8 ? 64 : 48;
  static_assert(2 * 128 * SOFTMAX + 128 * PRODUCER + 128 * MMA <= 512 * 128, "more registers than the launch has");
};

// 8 e4m3 values to bf16 (exact: 4 significant bits, exponents in range).
__device__ __forceinline__ void e4m3_to_bf16(uint32_t a, uint32_t b, uint32_t* w) {
  const uint32_t in[2] = {a, b};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t lo, hi;
    e4m3x4_to_f16(in[i], lo, hi);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    const float2 g = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    w[2 * i] = pack_bf16x2(f.x, f.y);
    w[2 * i + 1] = pack_bf16x2(g.x, g.y);
  }
}

// The pipeline of attn_kernel (two softmax streams per tile of 128 query rows, S and O in TMEM, P over
// S) with the keys of listed blocks in stages of 128: 128 / BK blocks a stage, a TMA box each, or, from an
// 8-bit store, loaded by bulk copies (warp 13) and widened in shared memory by the four producer warps,
// keys to fp16 (and Q with them), values to bf16.
//   PAIR = false  both streams work on the tile's 128 rows, alternate stages; merged at the end.
//   PAIR = true   lists of 64 rows: stream A takes rows 0-63 with their list, stream B rows 64-127
//                 with theirs.  The MMAs compute all 128 rows either way; no exponential is spent on
//                 a stream's other half, and the active warps lie on all four sub-partitions.
//                 d = 64: TMEM has room for four accumulators, so a stream's rows are worked on by
//                 two warps each, the first and the last 64 keys of every stage, with a running
//                 maximum, sum and O of their own, merged at the end like two streams (a stage's
//                 time is its longest chain of waits and exponentials: 1.17 us with one warp a row).
//                 d = 128: one warp a row.
// A unit with no usable entry has one stage of 128 masked keys, so that every unit takes the same path.
template <int HD, bool KV8, bool PAIR>
__global__ void __launch_bounds__(kAttnThreads, 1)
    block_attn_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const BlockAttnParams p) {
  using L = BlockSmem<HD, KV8>;
  using RG = BlockRegs<KV8>;
  constexpr int KST = L::KST, VST = L::VST;
  constexpr uint32_t HALF = kTile * 128;
  constexpr bool SUB = PAIR && HD == 64 && !KV8;       // a stream's keys in two halves, a warp pair each
  constexpr uint32_t ACTIVE = PAIR && !SUB ? 64 : 128;  // softmax threads of a stream
  constexpr int RUNS = SUB ? 2 : 4;                     // runs of 32 keys that a softmax thread takes
  constexpr int ISSUERS = SUB ? 4 : 1;                  // MMA-issuing warps
  static_assert(!SUB || (KST == VST && KST % 2 == 0), "SUB: each stream has half the slots");
  // (8-bit form: Q and K in fp16, whose two format fields are 0)
  constexpr uint32_t IDESC_QK = idesc_bf16(128, 32 * RUNS, false, false) & ~(KV8 ? (1u << 7 | 1u << 10) : 0u);
  constexpr uint32_t IDESC_PV = idesc_bf16(128, HD, false, true);
  constexpr uint32_t LAUNCH_REGS = 65536 / kAttnThreads;

  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t base = smem_u32(smem_raw);
  if (base & 1023u) {  // uniform across the CTA: nothing has started yet
    if (threadIdx.x == 0) raise_status(kStatusBadShape);
    return;
  }
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem_raw + L::BAR_OFF);
  uint64_t* q_full = bars + 0;
  uint64_t* q_empty = bars + 1;
  uint64_t* k_full = bars + 2;
  uint64_t* k_empty = k_full + KST;
  uint64_t* v_full = k_empty + KST;
  uint64_t* v_empty = v_full + VST;
  uint64_t* s_full = v_empty + VST;  // [2], per stream, as the next five
  uint64_t* p_full = s_full + 2;
  uint64_t* pv_done = p_full + 2;
  uint64_t* p_half = pv_done + 2;
  uint64_t* pvlo_done = p_half + 2;
  uint64_t* s_hi = pvlo_done + 2;  // SUB: S of a stage's second half (s_full: of its first)
  uint64_t* o_empty = s_hi + 2;
  uint64_t* drain = o_empty + 1;
  uint64_t* vfix = drain + 1;    // [2]: V stage whose last rows are cleared before it is handed on
  uint64_t* pair = vfix + 2;     // [4], one per row group (its two warps)
  uint64_t* u_full = pair + 4;   // [4], unit counts published
  uint64_t* q_ready = KV8 ? vfix : q_full;   // Q as the MMAs read it (8-bit form: once it is fp16)
  uint8_t* sQexp = smem_raw + L::QEXP_OFF;
  uint64_t* raw_full = u_full + 4;            // [RAWS] each: 8-bit tiles loaded, and widened
  uint64_t* raw_empty = raw_full + L::RAWS;
  StageInfo* sInfo = reinterpret_cast<StageInfo*>(smem_raw + L::INFO_OFF);
  int2* sUnit = reinterpret_cast<int2*>(smem_raw + L::UNIT_OFF);
  float2* sXch = reinterpret_cast<float2*>(smem_raw + L::XCH_OFF);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem_raw + L::MISC_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem_raw + L::MISC_OFF + 4);

  const uint32_t sQ = base + L::Q_OFF, sK = base + L::K_OFF, sV = base + L::V_OFF;
  const int warp = warp_id(), lane = lane_id();
  const uint64_t wl = p.wait_ns;

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, ISSUERS);
    for (int s = 0; s < KST; ++s) {
      mbar_init(k_full + s, KV8 ? 128 : 1);
      mbar_init(k_empty + s, ACTIVE);
    }
    for (int s = 0; s < VST; ++s) {
      mbar_init(v_full + s, KV8 ? 128 : 1);
      mbar_init(v_empty + s, SUB ? 2 : 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(s_full + x, 1);
      mbar_init(s_hi + x, 1);
      mbar_init(p_full + x, SUB ? 64 : ACTIVE);
      mbar_init(pv_done + x, 1);
      mbar_init(p_half + x, SUB ? 64 : ACTIVE);
      mbar_init(pvlo_done + x, 1);
    }
    mbar_init(o_empty, 2 * ACTIVE);
    mbar_init(drain, ISSUERS);
    mbar_init(vfix, KV8 ? 128 : 1);
    mbar_init(vfix + 1, 1);
    for (int g = 0; g < 4; ++g) mbar_init(pair + g, 64);
    for (int g = 0; g < 4; ++g) mbar_init(u_full + g, SUB ? 2 : 1);
    for (int s = 0; s < L::RAWS; ++s) {
      mbar_init(raw_full + s, 1);
      mbar_init(raw_empty + s, 128);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 12) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // The stages of a unit alternate between the streams while both have one; the longer stream's rest
  // follows.  tn = (stages of A, stages of B).
  auto stage_pos = [](int2 tn, int x, int i) {  // place of stream x's stage i in the unit
    const int m = min(tn.x, tn.y);
    return i < m ? 2 * i + x : m + i;
  };

  const int BPS = kTile / p.BK;  // blocks of a stage
  const int bk_log = 31 - __clz(p.BK);
  // What a producer warp learns of a unit: the walks over its lists, at their first entries, the
  // entries to take of each, and so the stages of both streams (`only` >= 0: of that list's alone).
  constexpr int LISTS = PAIR ? 2 : 1;
  struct Unit {
    int bh, ut, bkv, len;
    int left[LISTS], tn[2];
  };
  ListWalk wk[LISTS];
  auto open_unit = [&](int unit, int only, bool report) {
    Unit u;
    const int sp = unit % p.splits, tu = unit / p.splits;
    u.bh = tu / p.tiles;
    u.ut = tu - u.bh * p.tiles;
    const int b = u.bh / p.H;
    u.bkv = b * p.Hkv + (u.bh - b * p.H) / (p.H / p.Hkv);
    u.len = valid_rows(p.len, b, p.Nk);
    u.tn[0] = u.tn[1] = 0;
    auto open_list = [&](ListWalk& w, int x, int& left) {
      const int g = PAIR ? 2 * u.ut + x : u.ut;
      const bool some = g < p.GQ;  // not so: an odd last list, stream B has no rows here
      w.list = some && p.blocks != nullptr ? p.blocks + (static_cast<size_t>(u.bh) * p.GQ + g) * p.kb : nullptr;
      w.kb = some ? p.kb : 0;
      w.nb = p.nb;
      w.bk_log = bk_log;
      w.len = u.len;
      const int n = p.blocks != nullptr ? w.count(report) : min(p.nb, (u.len + p.BK - 1) >> bk_log);
      const int lo = static_cast<int>(static_cast<long long>(n) * sp / p.splits);
      left = static_cast<int>(static_cast<long long>(n) * (sp + 1) / p.splits) - lo;
      w.start(lo);
      return some ? max(1, (left + BPS - 1) / BPS) : 0;
    };
    if (only >= 0) {
      u.tn[only] = open_list(wk[0], only, u.left[0]);
    } else {
#pragma unroll
      for (int x = 0; x < LISTS; ++x) u.tn[x] = open_list(wk[x], x, u.left[x]);
      if (!PAIR) {
        u.tn[1] = u.tn[0] / 2;
        u.tn[0] -= u.tn[1];
      }
    }
    return u;
  };
  // The blocks of the next stage of walk x: their number; this lane's entries off and off2 among them
  // (meaningless from that number on).
  auto take = [&](Unit& u, int x, int off, int off2, int& blk, int& blk2) {
    auto from = [&](ListWalk& w, int& left) {
      w.ensure(BPS);
      const int n = min(min(BPS, left), w.have - w.at);
      blk = __shfl_sync(0xffffffffu, w.cur, (w.at + off) & 31);
      blk2 = __shfl_sync(0xffffffffu, w.cur, (w.at + off2) & 31);
      w.at += n;
      left -= n;
      return n;
    };
    return PAIR && x ? from(wk[LISTS - 1], u.left[LISTS - 1]) : from(wk[0], u.left[0]);
  };
  // The unit's counts for the other roles (`only` >= 0: that stream's), and its Q tile (after the last
  // QK^T of the one before).  The counts' slot was last the unit's four back: the MMAs of the unit
  // before this one are issued, so the epilogue of the one two before that has read its own.
  auto publish = [&](const Unit& u, uint32_t u_it, int only) -> bool {
    if (!mbar_wait_warp(q_empty, (u_it & 1) ^ 1, abort_flag, wl)) return false;
    if (lane == 0) {
      int2& slot = sUnit[u_it & 3];
      if (only <= 0) slot.x = u.tn[0];
      if (only != 0) slot.y = u.tn[1];
      mbar_arrive(u_full + (u_it & 3));
      if (only <= 0) {
        mbar_arrive_expect_tx(q_full, L::TILE_BYTES);
#pragma unroll
        for (int h = 0; h < HD / 64; ++h)
          tma_load_2d(sQ + h * HALF, &tmQ, h * 64, u.bh * p.Nq + u.ut * kTile, q_full);
      }
    }
    __syncwarp();
    return true;
  };

  if (warp >= 8 && warp < 12) {
    // ------------------------------------------------------------------ producer
    regs_to<RG::PRODUCER, LAUNCH_REGS>();
    const int pw = warp - 8;
    uint32_t u_it = 0;
    bool okp = true;
    if constexpr (!KV8) {
      // ---- bf16 rows by TMA, a box per block and 64 columns: warp 8 the keys, warp 9 the values; SUB:
      // of stream A's list, warps 10 and 11 those of stream B's
      if (SUB || pw < 2) {
        constexpr int HB = HD / 64;
        const bool keys = (pw & 1) == 0;
        const int only = SUB ? pw >> 1 : -1;
        const uint32_t ring = SUB ? KST / 2 : keys ? KST : VST;
        const int slot0 = SUB ? (pw >> 1) * (KST / 2) : 0;  // this warp's ring in the slots
        uint64_t* full = (keys ? k_full : v_full) + slot0;
        uint64_t* empty = (keys ? k_empty : v_empty) + slot0;
        uint64_t* fix = vfix + (SUB ? pw >> 1 : 0);
        const uint32_t tiles = (keys ? sK : sV) + slot0 * L::TILE_BYTES;
        const CUtensorMap* map = keys ? &tmK : &tmV;
        // lane l copies columns 64 (l % HB) .. of block l / HB of a stage, and sizes up run l % 4
        const int my_blk = lane / HB, my_col = lane % HB;
        const int run_blk = (lane & 3) * 32 >> bk_log, run_off = ((lane & 3) * 32) & (p.BK - 1);
        uint32_t n_fix = 0, issued = 0, q_issued = 0;
        for (int unit = blockIdx.x; unit < p.num_units && okp; unit += gridDim.x, ++u_it) {
          Unit u = open_unit(unit, only, keys);
          if (keys) {
            if (!publish(u, u_it, only)) { okp = false; break; }
            if (only <= 0) ++q_issued;
          }
          const int T = u.tn[0] + u.tn[1], both = 2 * min(u.tn[0], u.tn[1]), longer = u.tn[0] >= u.tn[1] ? 0 : 1;
          for (int t = 0; t < T; ++t) {
            int blk, rb;
            const int n = take(u, SUB ? 0 : t < both ? t & 1 : longer, my_blk, run_blk, blk, rb);  // blocks of this stage
            const int valid = run_blk < n ? min(32, max(0, u.len - rb * p.BK - run_off)) : 0;
            // a block reaches behind the last valid key
            const bool cut = __any_sync(0xffffffffu, run_blk < n && valid < 32);
            const uint32_t slot = issued % ring, ph = (issued / ring) & 1;
            if (!mbar_wait_warp(empty + slot, ph ^ 1, abort_flag, wl)) { okp = false; break; }
            const uint32_t dst = tiles + slot * L::TILE_BYTES;
            // masked keys weigh 0, but 0 times whatever lies in their V rows need not be 0: rows of no
            // block are cleared beside the copies, rows behind the last valid one after theirs
            auto clear = [&](int r) {
#pragma unroll
              for (int c = 0; c < HD / 8; ++c)
                asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(dst + sw128_offset(r, c, kTile)), "r"(0u)
                             : "memory");
            };
            if (keys) {
              if (lane < 4) sInfo[slot0 + slot].valid[lane] = valid;
            } else if (n < BPS) {
              for (int r = n * p.BK + lane; r < kTile; r += 32) clear(r);
              fence_proxy_async_smem();
            }
            const bool late = !keys && cut;
            uint64_t* land = late ? fix : full + slot;
            __syncwarp();
            if (lane == 0) mbar_arrive_expect_tx(land, static_cast<uint32_t>(n * p.BK) * HD * 2);
            __syncwarp();
            if (my_blk < n)
              tma_load_2d(dst + my_col * HALF + my_blk * p.BK * 128, map, my_col * 64, u.bkv * p.Nk + blk * p.BK, land);
            __syncwarp();
            if (late) {
              mbar_drain(fix, n_fix & 1);
              ++n_fix;
#pragma unroll
              for (int r = 0; r < 4; ++r)
                if (lane >= __shfl_sync(0xffffffffu, valid, r)) clear(r * 32 + lane);
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) mbar_arrive(full + slot);
              __syncwarp();
            }
            ++issued;
          }
        }
        // the copies issued land before the CTA releases its shared memory (consumed, and so at once, unless a
        // wait of some role ran out: this warp need not have noticed)
        if (q_issued > 0) mbar_drain(q_full, (q_issued - 1) & 1);
        for (uint32_t s = 0; s < ring && s < issued; ++s) {
          const uint32_t last = issued - 1 - ((issued - 1 + ring - s) % ring);
          mbar_drain(full + s, (last / ring) & 1);
        }
      }
    } else {
      // ---- 8-bit tiles, loaded by warp 13, widened (keys to fp16, values to bf16): every warp its run of 32 keys
      // of each
      constexpr int LPR = HD / 8, RPI = 32 / LPR, NIT = 32 / RPI;  // lanes to a row (8 values each), rows of a pass
      const int sub = lane / LPR, c = lane % LPR;
      constexpr uint32_t RAWS = L::RAWS;
      uint32_t it = 0, raw = 0;  // stages, 8-bit tiles so far
      // keys to fp16 (one instruction for two values), values to bf16 (P times their scale has its range; four);
      // rows from `rows` of this warp's run on become zero
      auto widen = [&](uint32_t src, uint32_t dst, int rows, bool keys) {
        const uint32_t from = src + (pw * 32 + sub) * HD + c * 8;
        // (a loop for each, rolled: with both in one, or eight loads unrolled, their code drove the softmax's out
        // of the instruction cache, 505 and 615 us against 484)
        if (keys) {
#pragma unroll 1
          for (int i0 = 0; i0 < NIT; i0 += 4) {  // four loads under way at a time
            uint32_t a[4], b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(a[i]), "=r"(b[i]) : "r"(from + (i0 + i) * RPI * HD));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int r = (i0 + i) * RPI + sub;
              uint32_t w[4];
              e4m3x4_to_f16(a[i], w[0], w[1]);
              e4m3x4_to_f16(b[i], w[2], w[3]);
              asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(dst + sw128_offset(pw * 32 + r, c, kTile)), "r"(w[0]),
                           "r"(w[1]), "r"(w[2]), "r"(w[3])
                           : "memory");
            }
          }
        } else {
#pragma unroll 1
          for (int i0 = 0; i0 < NIT; i0 += 4) {  // four loads under way at a time
            uint32_t a[4], b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(a[i]), "=r"(b[i]) : "r"(from + (i0 + i) * RPI * HD));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int r = (i0 + i) * RPI + sub;
              uint32_t w[4];
              if (r >= rows) a[i] = b[i] = 0u;
              e4m3_to_bf16(a[i], b[i], w);
              asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(dst + sw128_offset(pw * 32 + r, c, kTile)), "r"(w[0]),
                           "r"(w[1]), "r"(w[2]), "r"(w[3])
                           : "memory");
            }
          }
        }
        fence_proxy_async_smem();
      };
      for (int unit = blockIdx.x; unit < p.num_units && okp; unit += gridDim.x, ++u_it) {
        if (!mbar_wait_warp(u_full + (u_it & 3), (u_it >> 2) & 1, abort_flag, wl)) break;
        const int T = sUnit[u_it & 3].x + sUnit[u_it & 3].y;
        // Q to fp16 in place, a row a thread: times the power of two that brings its largest element into
        // [2^14, 2^15), whose exponent the softmax gets (exact down to 2^-28 of that element, off by at
        // most 2^-39 of it below; rows under 2^-107 are brought up by 2^121 alone)
        if (!mbar_wait_warp(q_full, u_it & 1, abort_flag, wl)) break;
        const int row = pw * 32 + lane;
        uint32_t top = 0;
#pragma unroll 4
        for (int k = 0; k < HD / 8; ++k) {
          const uint4 x = lds16(sQ + sw128_offset(row, k, kTile));
          top = __vmaxu2(__vmaxu2(top, x.x & 0x7fff7fffu), __vmaxu2(x.y & 0x7fff7fffu, __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu)));
        }
        const int e = min(max(static_cast<int>(max(top & 0xffffu, top >> 16) >> 7), 20), 254) - 127;
        const float up = __uint_as_float(static_cast<uint32_t>(14 - e + 127) << 23);
#pragma unroll 2
        for (int k = 0; k < HD / 8; ++k) {
          const uint32_t a = sQ + sw128_offset(row, k, kTile);
          float f[8];
          unpack8(lds16(a), f);
          asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(pack_f16x2(f[0] * up, f[1] * up)),
                       "r"(pack_f16x2(f[2] * up, f[3] * up)), "r"(pack_f16x2(f[4] * up, f[5] * up)),
                       "r"(pack_f16x2(f[6] * up, f[7] * up))
                       : "memory");
        }
        sQexp[(u_it & 1) * kTile + row] = static_cast<uint8_t>(e + 128);
        fence_proxy_async_smem();
        mbar_arrive(q_ready);
        for (int t = 0; t < T && okp; ++t, ++it) {
#pragma unroll 1
          for (int v = 0; v < 2; ++v, ++raw) {  // the stage's keys, then its values
            const uint32_t rs = raw % RAWS, slot = it % KST;
            if (!mbar_wait_warp(raw_full + rs, (raw / RAWS) & 1, abort_flag, wl) ||
                !mbar_wait_warp((v ? v_empty : k_empty) + slot, ((it / KST) & 1) ^ 1, abort_flag, wl)) {
              okp = false;
              break;
            }
            widen(base + L::RAW_OFF + rs * L::RAW_BYTES, (v ? sV : sK) + slot * L::TILE_BYTES,
                  v ? sInfo[it % L::INFOS].valid[pw] : 32, v == 0);
            mbar_arrive((v ? v_full : k_full) + slot);
            mbar_arrive(raw_empty + rs);
          }
        }
      }
    }
  } else if (warp >= 12) {
    // ------------------------------------------------------------------ MMA issuer
    regs_to<RG::MMA, LAUNCH_REGS>();
    if (warp < 12 + ISSUERS) {
      const uint64_t dQ = desc_sw128(sQ, 16, 1024);
      const uint64_t dK0 = desc_sw128(sK, 16, 1024);
      const uint64_t dV0 = desc_sw128(sV, HALF, 1024);
      constexpr uint64_t kSlotStep = L::TILE_BYTES >> 4;
      uint32_t u_it = 0;
      bool ok = true;
      if (p.hold != nullptr) {
        if (lane == 0) {
          const uint64_t t0 = globaltimer_ns();
          while (ld_acquire_gpu_u32(p.hold) == 0u) {
            if (globaltimer_ns() - t0 > wl) {
              raise_status(kStatusTimeout);
              *abort_flag = 1;
              ok = false;
              break;
            }
          }
        }
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      }
      auto wait_at = [&](uint64_t* full, uint32_t it, uint32_t ring) -> bool {  // stage `it` of a ring
        return mbar_wait_warp(full + it % ring, (it / ring) & 1, abort_flag, wl);
      };
      // S_x of the keys in a slot (SUB: of their half h)
      auto qk_mmas = [&](uint32_t slot, int x, int h) {
        const uint64_t dK = dK0 + slot * kSlotStep + h * (64 * 128 >> 4);
        const uint32_t dS = tmem + kTmS + x * kTile + h * 64;
#pragma unroll
        for (int kk = 0; kk < HD / 16; ++kk) {
          const uint64_t koff = ((kk >> 2) * HALF + (kk & 3) * 32) >> 4;
          mma_bf16_ss_warp(dS, dQ + koff, dK + koff, IDESC_QK, kk > 0 ? 1u : 0u);
        }
        mma_commit_warp((h ? s_hi : s_full) + x);
      };
      // k steps [from, to) of O += P V for the values in a slot (SUB: their half h)
      auto pv_mmas = [&](uint32_t slot, int x, int h, int from, int to, bool first) {
        const uint64_t dV = dV0 + slot * kSlotStep + h * (4 * 2048 >> 4);
        const uint32_t tO = tmem + kTmO + (SUB ? 2 * x + h : x) * HD, tP = tmem + kTmS + x * kTile + h * 64;
#pragma unroll
        for (int kk = from; kk < to; ++kk)
          mma_bf16_ts_warp(tO, tP + kk * 8, dV + kk * (2048 >> 4), IDESC_PV, (!first || kk > 0) ? 1u : 0u);
      };
      if constexpr (SUB) {
        // One warp for each stream and half of its keys, which waits for nothing of the others: the
        // streams have a ring each (a shared one's phases could pass a waiting warp by).
        constexpr uint32_t RING = KST / 2;
        const int x = (warp - 12) & 1, h = (warp - 12) >> 1;
        const uint32_t s0 = x * RING;
        uint32_t sc = 0;  // stages done (ring places and barrier phases)
        for (int unit = blockIdx.x; unit < p.num_units && ok; unit += gridDim.x, ++u_it) {
          ok = mbar_wait_warp(u_full + (u_it & 3), (u_it >> 2) & 1, abort_flag, wl);
          if (!ok) break;
          const int Tx = x ? sUnit[u_it & 3].y : sUnit[u_it & 3].x;
          ok = mbar_wait_warp(q_full, u_it & 1, abort_flag, wl) && (Tx == 0 || wait_at(k_full + s0, sc, RING));
          if (!ok) break;
          if (Tx > 0) qk_mmas(s0 + sc % RING, x, h);
          if (Tx <= 1) mma_commit_warp(q_empty);
          if (Tx == 0) ok = mbar_wait_warp(o_empty, (u_it & 1) ^ 1, abort_flag, wl);  // keep step with its phases
          for (int i = 0; i < Tx; ++i, ++sc) {
            const bool next = i + 1 < Tx;
            ok = (!next || wait_at(k_full + s0, sc + 1, RING)) && wait_at(v_full + s0, sc, RING) &&
                 (i != 0 || mbar_wait_warp(o_empty, (u_it & 1) ^ 1, abort_flag, wl)) &&
                 mbar_wait_warp((h ? p_full : p_half) + x, sc & 1, abort_flag, wl);
            if (!ok) break;
            tc_fence_after();  // P_x was written by tcgen05.st of the softmax
            pv_mmas(s0 + sc % RING, x, h, 0, 4, i == 0);
            mma_commit_warp((h ? pv_done : pvlo_done) + x);
            mma_commit_warp(v_empty + s0 + sc % RING);
            if (next) {
              qk_mmas(s0 + (sc + 1) % RING, x, h);
              if (i + 2 == Tx) mma_commit_warp(q_empty);
            }
          }
        }
      } else {
        uint32_t kv_base = 0, sc0 = 0, sc1 = 0;  // stages of earlier units; PVs issued per stream (barrier phases)
        for (int unit = blockIdx.x; unit < p.num_units && ok; unit += gridDim.x, ++u_it) {
          ok = mbar_wait_warp(u_full + (u_it & 3), (u_it >> 2) & 1, abort_flag, wl);
          if (!ok) break;
          const int2 tn = sUnit[u_it & 3];
          const int T = tn.x + tn.y, both = 2 * min(tn.x, tn.y), longer = tn.x >= tn.y ? 0 : 1;
          ok = mbar_wait_warp(q_ready, u_it & 1, abort_flag, wl) && wait_at(k_full, kv_base, KST) &&
               (both == 0 || wait_at(k_full, kv_base + 1, KST));
          if (!ok) break;
          qk_mmas(kv_base % KST, 0, 0);
          if (both > 0) qk_mmas((kv_base + 1) % KST, 1, 0);
          if (T == max(both, 1) && T <= 2) mma_commit_warp(q_empty);
          int n0 = 0, n1 = 0;  // stages of each stream done in this unit
          for (int t = 0; t < T && ok; ++t) {
            const int x = PAIR && t >= both ? longer : t & 1;
            const int mine = PAIR ? (x ? n1 : n0) : t >> 1;
            const bool next = PAIR ? mine + 1 < (x ? tn.y : tn.x) : t + 2 < T;
            const int tnext = PAIR ? stage_pos(tn, x, mine + 1) : t + 2;
            ok = mbar_wait_warp(p_half + x, (x ? sc1 : sc0) & 1, abort_flag, wl) && wait_at(v_full, kv_base + t, VST) &&
                 (t != 0 || mbar_wait_warp(o_empty, (u_it & 1) ^ 1, abort_flag, wl));
            if (!ok) break;
            tc_fence_after();  // P_x was written by tcgen05.st of the softmax
            pv_mmas((kv_base + t) % VST, x, 0, 0, 2 * kPSplit, mine == 0);
            mma_commit_warp(pvlo_done + x);
            ok = mbar_wait_warp(p_full + x, (x ? sc1 : sc0) & 1, abort_flag, wl) &&
                 (!next || wait_at(k_full, kv_base + tnext, KST));
            if (!ok) break;
            tc_fence_after();
            pv_mmas((kv_base + t) % VST, x, 0, 2 * kPSplit, kTile / 16, false);
            mma_commit_warp(pv_done + x);
            mma_commit_warp(v_empty + (kv_base + t) % VST);
            if (x) ++sc1, ++n1;
            else ++sc0, ++n0;
            if (next) {
              qk_mmas((kv_base + tnext) % KST, x, 0);
              if (tnext == T - 1) mma_commit_warp(q_empty);
            }
          }
          kv_base += T;
        }
      }
      // every MMA issued above has completed before TMEM is released
      mma_commit_warp(drain);
      mbar_drain(drain, 0);
    } else if (KV8 && warp == 13) {
      if constexpr (KV8) {
        constexpr uint32_t RAWS = L::RAWS;
        // ---- loader of the 8-bit tiles: K, then V, of every stage by bulk copies, a whole block each; its
        // blocks' scales and valid keys for the other roles.  An entry of sInfo is written eight stages after
        // its last use: the ring of widened tiles lets this warp no further ahead.
        uint32_t u_it = 0, it = 0, raw = 0;
        bool ok = true;
        const int run_blk = (lane & 3) * 32 >> bk_log, run_off = ((lane & 3) * 32) & (p.BK - 1);
        const uint32_t block_bytes = static_cast<uint32_t>(p.BK) * HD;
        for (int unit = blockIdx.x; unit < p.num_units && ok; unit += gridDim.x, ++u_it) {
          Unit u = open_unit(unit, -1, true);
          if (!publish(u, u_it, -1)) break;
          const int T = u.tn[0] + u.tn[1], both = 2 * min(u.tn[0], u.tn[1]), longer = u.tn[0] >= u.tn[1] ? 0 : 1;
          // a stage ahead, so that the scales are here when the stage is: its blocks, this lane's of them,
          // the valid keys and scales of run lane % 4
          int n = 0, blk = 0, valid = 0;
          float fks = 1.f, fvs = 1.f;
          auto look = [&](int t) {
            int rb;
            n = take(u, t < both ? t & 1 : longer, lane, run_blk, blk, rb);
            valid = run_blk < n ? min(32, max(0, u.len - rb * p.BK - run_off)) : 0;
            if (run_blk < n) {
              fks = p.ks[static_cast<size_t>(u.bkv) * p.nb + rb];
              fvs = p.vs[static_cast<size_t>(u.bkv) * p.nb + rb];
            }
          };
          look(0);
          for (int t = 0; t < T && ok; ++t, ++it) {
            const int cn = n, cblk = blk;
            const size_t at = (static_cast<size_t>(u.bkv) * p.Nk + static_cast<size_t>(lane < cn ? cblk : 0) * p.BK) * HD;
#pragma unroll
            for (int v = 0; v < 2; ++v, ++raw) {
              const uint32_t rs = raw % RAWS;
              ok = mbar_wait_warp(raw_empty + rs, ((raw / RAWS) & 1) ^ 1, abort_flag, wl);
              if (!ok) break;
              if (v == 0 && lane < 4) {
                StageInfo& info = sInfo[it % L::INFOS];
                info.valid[lane] = valid;
                info.ks[lane] = fks;
                info.vs[lane] = fvs;
              }
              __syncwarp();
              if (lane == 0) mbar_arrive_expect_tx(raw_full + rs, cn * block_bytes);
              __syncwarp();
              if (lane < cn)
                bulk_load(base + L::RAW_OFF + rs * L::RAW_BYTES + lane * block_bytes,
                          static_cast<const uint8_t*>(v ? p.V : p.K) + at, block_bytes, raw_full + rs);
              __syncwarp();
            }
            if (ok && t + 1 < T) look(t + 1);
          }
        }
        // the copies issued land before the CTA releases its shared memory, whatever the other roles did
        if (u_it > 0) mbar_drain(q_full, (u_it - 1) & 1);
        for (uint32_t s = 0; s < RAWS && s < raw; ++s) {
          const uint32_t last = raw - 1 - ((raw - 1 + RAWS - s) % RAWS);
          mbar_drain(raw_full + s, (last / RAWS) & 1);
        }
      }
    }  // the other warps only complete the warpgroup
  } else {
    // ------------------------------------------------------------------ softmax + epilogue
    regs_to<RG::SOFTMAX, LAUNCH_REGS>();
    const int rg = warp & 3, side = warp >> 2;  // row group, first or second of its two warps
    const int x = SUB ? rg >> 1 : side;         // stream
    if (!PAIR || SUB || (rg >> 1) == x) {
      const int row = rg * 32 + lane;  // tile row == TMEM lane
      const uint32_t lane_base = static_cast<uint32_t>(rg * 32) << 16;
      const int r0 = SUB ? 2 * side : 0;  // this thread's first run of a stage
      const uint32_t tS = tmem + lane_base + kTmS + x * kTile + r0 * 32;
      const uint32_t tOx = tmem + lane_base + kTmO + (SUB ? 2 * x + side : x) * HD;
      uint64_t* s_mine = SUB && side == 1 ? s_hi + x : s_full + x;
      uint64_t* pv_mine = SUB && side == 0 ? pvlo_done + x : pv_done + x;  // the last PV of this thread's P
      const float sl2 = p.scale_log2;
      uint32_t sc = 0, kv_base = 0, u_it = 0;
      bool ok = true;
      for (int unit = blockIdx.x; unit < p.num_units && ok; unit += gridDim.x, ++u_it) {
        const int sp = unit % p.splits, tu = unit / p.splits;
        const int bh = tu / p.tiles, ut = tu - bh * p.tiles;
        const int qrow = ut * kTile + row;
        const bool live = qrow < p.Nq;
        if (!mbar_wait_warp(u_full + (u_it & 3), (u_it >> 2) & 1, abort_flag, wl)) { ok = false; break; }
        const int2 tn = sUnit[u_it & 3];
        const int Tx = x ? tn.y : tn.x;
        float qscale = sl2;
        float m_used = -INFINITY, l_part = 0.f;  // -inf: no key of weight yet
        float m_pend = -INFINITY;  // a raise of the reference decided by the stream's previous stage
        for (int i = 0; i < Tx; ++i, ++sc) {
          if (!mbar_wait_warp(s_mine, sc & 1, abort_flag, wl)) { ok = false; break; }
          if (KV8 && i == 0)  // the power of two that Q's row was brought up by, taken back
            qscale = sl2 * __uint_as_float(static_cast<uint32_t>(sQexp[(u_it & 1) * kTile + row] - 128 - 14 + 127) << 23);
          const uint32_t slot = SUB ? x * (KST / 2) + sc % (KST / 2) : (kv_base + stage_pos(tn, x, i)) % KST;
          int vq[RUNS], all = 32;
          float kq[RUNS], vsq[RUNS];
#pragma unroll
          for (int q = 0; q < RUNS; ++q) {
            const StageInfo& info = sInfo[KV8 ? (kv_base + stage_pos(tn, x, i)) % L::INFOS : slot];
            vq[q] = info.valid[r0 + q];
            all &= vq[q];
            // (at least the smallest normal number: masked keys are -inf times this)
            kq[q] = KV8 ? fmaxf(qscale * info.ks[r0 + q], 1.17549435e-38f) : sl2;
            vsq[q] = KV8 ? info.vs[r0 + q] : 1.f;
          }
          // the QK^T that wrote S has read its K slot: hand the slot back to the producer
          mbar_arrive(k_empty + slot);
          tc_fence_after();
          auto rescale_o = [&](float alpha) {
#pragma unroll 1
            for (int c0 = 0; c0 < HD; c0 += 32) {
              uint32_t o[32];
              tmem_ld32(tOx + c0, o);
              tmem_ld_wait_regs(o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tmem_st32(tOx + c0, o);
            }
          };
          auto signal_half = [&]() {
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(p_half + x);
          };
          // P = exp2(S * scale - m) of one run of 32 keys, times its V scale, in bf16 pairs, and its
          // sums over the even and the odd keys
          auto chunk_exps = [&](const uint32_t* sr, float k, float vs, float m, uint32_t* pk, float2& cs) {
            cs = make_float2(0.f, 0.f);
            const float2 k2 = make_float2(k, k), nm2 = make_float2(-m, -m), v2 = make_float2(vs, vs);
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              const float2 xv =
                  __ffma2_rn(make_float2(__uint_as_float(sr[2 * c]), __uint_as_float(sr[2 * c + 1])), k2, nm2);
              float2 e = make_float2(fast_exp2(xv.x), fast_exp2(xv.y));
              cs = __fadd2_rn(cs, e);
              if (KV8) e = __fmul2_rn(e, v2);
              pk[c] = pack_bf16x2(e.x, e.y);
            }
          };
          uint32_t sr[32 * RUNS];
#pragma unroll
          for (int q = 0; q < RUNS; ++q) tmem_ld32(tS + 32 * q, sr + 32 * q);
          tmem_ld_wait_regs(sr);
#pragma unroll
          for (int q = 1; q < RUNS; ++q) reg_fence32(sr + 32 * q);
          if (__builtin_expect(all != 32, 0)) {  // masked keys: logits of -inf, whatever was computed
#pragma unroll
            for (int c = 0; c < 32 * RUNS; ++c) sr[c] = (c & 31) < vq[c >> 5] ? sr[c] : 0xff800000u;
          }
          // Rows without a reference yet (the first stage, or every key so far masked or at -inf; O_x
          // and l are 0 then) take the stage's exact maximum.
          if (__builtin_expect(__any_sync(0xffffffffu, m_used == -INFINITY), 0)) {
            float mx = -INFINITY;
#pragma unroll
            for (int q = 0; q < RUNS; ++q) {
              float a = -INFINITY, b = -INFINITY;
#pragma unroll
              for (int c = 0; c < 32; c += 2) {
                a = fmaxf(a, __uint_as_float(sr[32 * q + c]));
                b = fmaxf(b, __uint_as_float(sr[32 * q + c + 1]));
              }
              mx = fmaxf(mx, fmaxf(a, b) * kq[q]);
            }
            if (m_used == -INFINITY) m_used = mx;
          }
          // A stage whose P summed past 2^16 raised the reference for this one, applied once the
          // stream's previous PV has completed so that O_x and l follow.
          if (__builtin_expect(__any_sync(0xffffffffu, m_pend > m_used), 0)) {
            if (!mbar_wait_warp(pv_mine, (sc - 1) & 1, abort_flag, wl)) { ok = false; break; }
            tc_fence_after();
            const float alpha = m_pend > m_used ? fast_exp2(m_used - m_pend) : 1.f;
            rescale_o(alpha);
            l_part *= alpha;
            m_used = fmaxf(m_used, m_pend);
          }
          float2 rs = make_float2(0.f, 0.f);
          // known complete: the stream's previous PV (o_prev), also this stage's first part (o_lo)
          bool o_prev = false, o_lo = false;
#pragma unroll
          for (int q = 0; q < RUNS; ++q) {
            uint32_t pk[16];
            float2 cs;
            chunk_exps(sr + 32 * q, kq[q], vsq[q], m_used == -INFINITY ? 0.f : m_used, pk, cs);
            const bool big = !(cs.x + cs.y <= 4294967296.f);  // 2^32, or inf / NaN
            if (__builtin_expect(__any_sync(0xffffffffu, big), 0)) {
              // rare: raise this row's reference to the run's largest logit, by whole octaves where anything is
              // left of what is behind it (so that rescaling bf16 P is exact), rescale that, and redo the run with
              // its products rounded as the reference is: no key of it lies above its largest then, however
              // large they are
              const float mz = m_used == -INFINITY ? 0.f : m_used;
              float top = -INFINITY;
#pragma unroll
              for (int c = 0; c < 32; ++c) {
                const float s = __fmul_rn(__uint_as_float(sr[32 * q + c]), kq[q]);
                top = fmaxf(top, s);
                sr[32 * q + c] = __float_as_uint(s);
              }
              const bool raise = big && top > mz;
              const float xr = raise ? ceilf(top - mz) : 0.f;
              const int n = static_cast<int>(fminf(xr, 127.f));
              const float alpha = n >= 127 ? 0.f : __int_as_float((127 - n) << 23);  // 2^-n
              if (!SUB && q >= kPSplit && !o_lo) {
                if (!mbar_wait_warp(pvlo_done + x, sc & 1, abort_flag, wl)) { ok = false; break; }
                tc_fence_after();
                o_lo = o_prev = true;
              } else if (!o_prev) {
                if (!mbar_wait_warp(pv_mine, (sc - 1) & 1, abort_flag, wl)) { ok = false; break; }
                tc_fence_after();
                o_prev = true;
              }
              tmem_st_wait();
              rescale_o(alpha);
              l_part *= alpha;
              rs.x *= alpha;
              rs.y *= alpha;
#pragma unroll 1
              for (int q2 = !SUB && q >= kPSplit ? kPSplit : 0; q2 < q; ++q2) {
                uint32_t pv[16];
                tmem_ld16(tS + 16 * q2, pv);
                tmem_ld_wait_regs16(pv);
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                  const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&pv[e]));
                  pv[e] = pack_bf16x2(f.x * alpha, f.y * alpha);
                }
                tmem_st16(tS + 16 * q2, pv);
              }
              tmem_st_wait();
              if (raise) m_used = n >= 127 ? top : mz + xr;
              chunk_exps(sr + 32 * q, 1.f, vsq[q], m_used == -INFINITY ? 0.f : m_used, pk, cs);
            }
            rs = __fadd2_rn(rs, cs);
            tmem_st16(tS + 16 * q, pk);
            if (!SUB && q == kPSplit - 1) signal_half();
          }
          if (!ok) break;
          const float st = rs.x + rs.y;
          m_pend = st > 65536.f ? m_used + __log2f(st) : -INFINITY;
          l_part += st;
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(SUB && side == 0 ? p_half + x : p_full + x);
        }
        if (!ok) break;
        kv_base += tn.x + tn.y;
        const size_t orow = static_cast<size_t>(bh) * p.Nq + qrow;
        const size_t prow = static_cast<size_t>(sp) * p.B * p.H * p.Nq + orow;  // of a split's partial result
        if (Tx > 0) {
          // this stream's last PV of the unit
          if (!mbar_wait_warp(pv_mine, (sc - 1) & 1, abort_flag, wl)) { ok = false; break; }
          tc_fence_after();
        }
        // 8 output columns from column c on: R is added, or the partial result goes to the workspace
        auto store8 = [&](int c, float* v) {
          if (p.splits > 1) {
            float4* d = reinterpret_cast<float4*>(p.part + prow * HD + c);
            d[0] = make_float4(v[0], v[1], v[2], v[3]);
            d[1] = make_float4(v[4], v[5], v[6], v[7]);
            return;
          }
          *reinterpret_cast<uint4*>(p.out + orow * HD + c) = pack8(v);
        };
        const bool add = live && p.R != nullptr && p.splits == 1;
        float m_all = m_used, l_sum = l_part;
        if constexpr (PAIR && !SUB) {
          const float inv = l_sum == 0.f ? 0.f : 1.f / l_sum;
#pragma unroll 1
          for (int c0 = 0; c0 < HD; c0 += 64) {
            uint4 extra[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
              extra[e] = add ? *reinterpret_cast<const uint4*>(p.R + orow * HD + c0 + 8 * e) : make_uint4(0u, 0u, 0u, 0u);
            uint32_t o[64];
            tmem_ld64_wait(tOx + c0, o);
            if (live) {
#pragma unroll
              for (int c = 0; c < 64; c += 8) {
                float v[8], r[8];
                unpack8(extra[c / 8], r);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = fmaf(__uint_as_float(o[c + e]), inv, r[e]);
                store8(c0 + c, v);
              }
            }
          }
        } else {
          constexpr int NV = HD / 16;  // uint4 (8 bf16) per half row
          const int cx = side * (HD / 2);
          uint4 extra[NV];
#pragma unroll
          for (int e = 0; e < NV; ++e)
            extra[e] = add ? *reinterpret_cast<const uint4*>(p.R + orow * HD + cx + 8 * e) : make_uint4(0u, 0u, 0u, 0u);
          const bool has_b = SUB || tn.y > 0;
          sXch[side * kTile + row] = make_float2(m_used, l_part);
          tc_fence_before();
          mbar_arrive(pair + rg);
          if (!mbar_wait_warp(pair + rg, 0, abort_flag, wl)) { ok = false; break; }
          tc_fence_after();
          const float2 xa = sXch[row], xb = sXch[kTile + row];
          mbar_arrive(pair + rg);
          if (!mbar_wait_warp(pair + rg, 1, abort_flag, wl)) { ok = false; break; }
          m_all = fmaxf(xa.x, xb.x);
          const float mz = m_all == -INFINITY ? 0.f : m_all;
          const float wA = fast_exp2(xa.x - mz);
          const float wB = has_b ? fast_exp2(xb.x - mz) : 0.f;
          l_sum = xa.y * wA + xb.y * wB;
          const float inv = l_sum == 0.f ? 0.f : 1.f / l_sum;
          const float cA = wA * inv, cB = wB * inv;
          const uint32_t tOA = tmem + lane_base + kTmO + (SUB ? 2 * x * HD : 0) + cx, tOB = tOA + HD;
          uint32_t oab[HD];  // [0, HD/2): O_A; [HD/2, HD): O_B
          if constexpr (HD == 128) tmem_ld32x4_wait(tOA, tOA + 32, tOB, tOB + 32, oab);
          else tmem_ld32x2_wait(tOA, tOB, oab);
          if (live) {
#pragma unroll
            for (int c = 0; c < HD / 2; c += 8) {
              float v[8], r[8];
              unpack8(extra[c / 8], r);
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                // O_B holds no product of this unit when stream B had no stage: leave it out
                const float ob = has_b ? __uint_as_float(oab[HD / 2 + c + e]) * cB : 0.f;
                v[e] = fmaf(__uint_as_float(oab[c + e]), cA, ob) + r[e];
              }
              store8(cx + c, v);
            }
          }
        }
        if (live && ((PAIR && !SUB) || side == 0)) {
          const float l2 = l_sum == 0.f ? -INFINITY : m_all + __log2f(l_sum);
          if (p.splits > 1) p.plse[prow] = l2;
          else if (p.lse != nullptr) p.lse[orow] = l2 * 0.69314718055994531f;
        }
        tc_fence_before();
        mbar_arrive(o_empty);
      }
      // (after an abort) no load or store of this warp is still in flight when TMEM is released
      tmem_ld_wait();
      tmem_st_wait();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------------------------- splits joined
// out = sum_s 2^(l_s - l) o_s (+ R), l = log2 sum_s 2^l_s over the parts of a row's keys.  A CTA takes a few
// rows, HD / 4 lanes a row, and shares each row's parts out over its groups of lanes.
constexpr int kJoinGroups = 4;  // groups to a row

template <int HD>
__global__ void __launch_bounds__(256) block_join_kernel(const BlockAttnParams p) {
  constexpr int LPR = HD / 4, RPB = 256 / LPR / kJoinGroups;  // lanes to a row, rows of a CTA
  __shared__ float sm_m[kJoinGroups][RPB], sm_l[kJoinGroups][RPB];
  __shared__ __align__(16) float4 sm_o[kJoinGroups][RPB][LPR];
  const long long rows = static_cast<long long>(p.B) * p.H * p.Nq;
  const int lane = threadIdx.x % LPR, r = threadIdx.x / LPR % RPB, grp = threadIdx.x / LPR / RPB;
  const long long row = static_cast<long long>(blockIdx.x) * RPB + r;
  const bool live = row < rows;
  wait_for_results();
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  if (live) {
#pragma unroll 4
    for (int s = grp; s < p.splits; s += kJoinGroups) {
      const float x = p.plse[s * rows + row];
      const float4 v = *reinterpret_cast<const float4*>(p.part + (s * rows + row) * HD + lane * 4);
      const float mn = fmaxf(m, x), ref = mn == -INFINITY ? 0.f : mn;
      const float a = exp2f(m - ref), w = exp2f(x - ref);
      m = mn;
      l = fmaf(l, a, w);
      o = make_float4(fmaf(w, v.x, o.x * a), fmaf(w, v.y, o.y * a), fmaf(w, v.z, o.z * a), fmaf(w, v.w, o.w * a));
    }
  }
  if (lane == 0) sm_m[grp][r] = m, sm_l[grp][r] = l;
  sm_o[grp][r][lane] = o;
  __syncthreads();
  if (grp != 0 || !live) return;
#pragma unroll
  for (int i = 1; i < kJoinGroups; ++i) m = fmaxf(m, sm_m[i][r]);
  const float ref = m == -INFINITY ? 0.f : m;
  float f[4] = {0.f, 0.f, 0.f, 0.f};
  l = 0.f;
#pragma unroll
  for (int i = 0; i < kJoinGroups; ++i) {
    const float w = exp2f(sm_m[i][r] - ref);
    const float4 v = sm_o[i][r][lane];
    l = fmaf(w, sm_l[i][r], l);
    f[0] = fmaf(w, v.x, f[0]), f[1] = fmaf(w, v.y, f[1]), f[2] = fmaf(w, v.z, f[2]), f[3] = fmaf(w, v.w, f[3]);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  float add[4] = {0.f, 0.f, 0.f, 0.f};
  if (p.R != nullptr) {
    const uint2 u = *reinterpret_cast<const uint2*>(p.R + row * HD + lane * 4);
    const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.x));
    const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.y));
    add[0] = a.x, add[1] = a.y, add[2] = b.x, add[3] = b.y;
  }
  uint2 w;
  w.x = pack_bf16x2(fmaf(f[0], inv, add[0]), fmaf(f[1], inv, add[1]));
  w.y = pack_bf16x2(fmaf(f[2], inv, add[2]), fmaf(f[3], inv, add[3]));
  *reinterpret_cast<uint2*>(p.out + row * HD + lane * 4) = w;
  if (p.lse != nullptr && lane == 0) p.lse[row] = l == 0.f ? -INFINITY : (ref + log2f(l)) * 0.69314718055994531f;
}

}  // namespace mcs
