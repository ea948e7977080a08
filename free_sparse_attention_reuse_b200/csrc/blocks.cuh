// Key blocks: their means, their choice by a cheap score, and the 8-bit store that holds them.
#pragma once

#include <cuda_fp8.h>

#include <type_traits>

#include "rotary.cuh"

namespace mcs {

// ---------------------------------------------------------------------------------- lengths
// Valid rows of batch entry b: len[b] within [0, n]; a value outside is reported and clamped.
__device__ __forceinline__ int valid_rows(const int32_t* len, int b, int n) {
  if (len == nullptr) return n;
  const int v = len[b];
  if (v < 0 || v > n) {
    raise_status(kStatusBadIndex);
    return v < 0 ? 0 : n;
  }
  return v;
}

// Four e4m3 values to fp16, exact: the lower two and the upper two.
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t x, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(x));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 u;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "r"(a));
  return u;
}
// `bytes` consecutive bytes (a multiple of 16, as both addresses are) into shared memory; completes them on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// ---------------------------------------------------------------------------------- means
// means[bh, j, :] = mean of the valid rows of block j (zero where it has none).  The sum is taken in
// fp64, which holds a sum of up to 128 bf16 values exactly unless their exponents are more than 38
// octaves apart, and rounded once to fp32 after the division: the mean does not depend on the order
// of the rows, so scores of equal blocks tie exactly.
struct MeansParams {
  const __nv_bfloat16* X;  // [B, H, N, d]
  const int32_t* len;      // [B], nullable
  float* means;            // [B, H, nb, d]
  int H, N, nb, BK;
  long long blocks;        // B * H * nb
};

constexpr int kMeansThreads = 128;

// One CTA a block, its warps a share of the rows each.  Bound: device memory, with the widening to fp64 (XU)
// at two thirds of that time; a warp a block left a last wave of few CTAs (46 us against 36 for 198 MB).
template <int HD>
__global__ void __launch_bounds__(kMeansThreads) block_means_kernel(const MeansParams p) {
  constexpr int LPR = HD / 8, RPP = kMeansThreads / LPR;  // lanes of a row, rows of a pass
  constexpr int WARPS = kMeansThreads / 32;
  __shared__ double sums[WARPS][HD];
  let_dependents_start();
  const int t = threadIdx.x, lane = lane_id(), c = t % LPR;
  const long long blk = blockIdx.x, bh = blk / p.nb;
  const int j = static_cast<int>(blk - bh * p.nb);
  const int n = min(p.BK, valid_rows(p.len, static_cast<int>(bh / p.H), p.N) - j * p.BK);
  const __nv_bfloat16* row = p.X + (static_cast<size_t>(bh) * p.N + static_cast<size_t>(j) * p.BK) * HD + c * 8;
  double acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.0;
  auto add = [&](const uint4& u) {
    float f[8];
    unpack8(u, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] += static_cast<double>(f[i]);
  };
  int r = t / LPR;
  for (; r + 7 * RPP < n; r += 8 * RPP) {  // eight rows in flight
    uint4 u[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) u[k] = load16(row + static_cast<size_t>(r + k * RPP) * HD);
#pragma unroll
    for (int k = 0; k < 8; ++k) add(u[k]);
  }
  for (; r < n; r += RPP) add(load16(row + static_cast<size_t>(r) * HD));
#pragma unroll
  for (int o = LPR; o < 32; o <<= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
  if (lane < LPR)
#pragma unroll
    for (int i = 0; i < 8; ++i) sums[warp_id()][c * 8 + i] = acc[i];
  __syncthreads();
  for (int e = t; e < HD; e += kMeansThreads) {
    double s = 0.0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) s += sums[w][e];
    p.means[static_cast<size_t>(blk) * HD + e] = n > 0 ? static_cast<float>(s / static_cast<double>(n)) : 0.f;
  }
}

// ---------------------------------------------------------------------------------- choice
// score(g, j) = qbar_g . kbar_j of the fp32 means, in fp64 (their products are exact there), so that the
// choice is the definition's and not a summation order's; then the kb largest of a row, ties to the lower
// block.  Rows are query blocks; those of the H / Hkv heads that share a key head lie one behind the other
// and make one matrix of M rows against its nb means.
//
// Order of scores as unsigned integers: 0 is no candidate, then NaN below every number, both zeros alike.
__device__ __forceinline__ unsigned long long score_key(double s) {
  if (s != s) return 1ull;
  if (s == 0.0) s = 0.0;
  const unsigned long long u = static_cast<unsigned long long>(__double_as_longlong(s));
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

struct TopkParams {
  const __nv_bfloat16* Q;  // [B, H, Nq, d]: the rows themselves where C = 1
  const float* qbar;       // [B, H, GQ, d]: their means else
  const float* means;      // [B, Hkv, nb, d]
  const int32_t* len;      // [B], nullable
  unsigned long long* keys;  // [rows of this launch, nb]
  int32_t* blocks;           // [B, H, GQ, kb]
  int Hkv, Nk, M, BK, nb, kb;
  int kv0, m0, mc;  // rows of this launch: key heads from kv0 on (the grid's), rows [m0, m0 + mc) of each
};

__device__ __forceinline__ int candidate_blocks(const TopkParams& p, int kv) {
  return (valid_rows(p.len, kv / p.Hkv, p.Nk) + p.BK - 1) / p.BK;
}

// D += A B, 8 x 8 x 4, fp64: lane l holds A[l / 4][l % 4], B[l % 4][l / 4] and D[l / 4][2 (l % 4) + {0, 1}].
__device__ __forceinline__ void mma_f64(double& d0, double& d1, double a, double b) {
  asm("mma.sync.aligned.m8n8k4.row.col.f64.f64.f64.f64 {%0,%1}, {%2}, {%3}, {%0,%1};" : "+d"(d0), "+d"(d1) : "d"(a), "d"(b));
}

// 64 rows by 64 blocks a CTA on the fp64 tensor cores, 32 x 32 a warp, 32 columns of d at a time from shared
// memory (rows four doubles longer than that, so that a half warp's fragment reads hit all banks).  Bound:
// the fp64 pipe (195 M multiply-adds for 24 heads of 252 x 252 blocks of 128: 11 us at its full rate);
// multiply-adds from 4 x 4 and 8 x 4 values a thread were bound by the reads of shared memory (48, 31 us).
constexpr int kScoreTile = 64, kScoreDepth = 32, kScoreThreads = 128;

template <int HD>
__global__ void __launch_bounds__(kScoreThreads) block_score_kernel(const TopkParams p) {
  __shared__ __align__(16) double as[kScoreTile][kScoreDepth + 4], bs[kScoreTile][kScoreDepth + 4];
  const int t = threadIdx.x, lane = lane_id(), fr = lane >> 2, fk = lane & 3;
  const int wm = (warp_id() >> 1) * 32, wn = (warp_id() & 1) * 32;  // this warp's rows and blocks
  const int kv = p.kv0 + blockIdx.z, m0 = blockIdx.y * kScoreTile, j0 = blockIdx.x * kScoreTile;
  const int nv = candidate_blocks(p, kv);
  let_dependents_start();
  wait_for_results();  // the mean query rows (in every CTA: a grid that ends has seen the one before it end)
  if (j0 >= nv) return;
  const size_t row0 = static_cast<size_t>(kv) * p.M + p.m0 + m0;
  const int rows = p.mc - m0;
  double acc[4][4][2];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j][0] = acc[i][j][1] = 0.0;
  float4 a[4], b[4];
  auto load = [&](int k0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = (t >> 3) + 16 * i, k = (t & 7) * 4;
      a[i] = b[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < rows) {
        const size_t at = (row0 + r) * HD + k0 + k;
        if (p.qbar != nullptr) {
          a[i] = *reinterpret_cast<const float4*>(p.qbar + at);
        } else {
          const uint2 u = *reinterpret_cast<const uint2*>(p.Q + at);
          const float2 x = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.x));
          const float2 y = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.y));
          a[i] = make_float4(x.x, x.y, y.x, y.y);
        }
      }
      if (j0 + r < nv) b[i] = *reinterpret_cast<const float4*>(p.means + (static_cast<size_t>(kv) * p.nb + j0 + r) * HD + k0 + k);
    }
  };
  load(0);
  for (int k0 = 0; k0 < HD; k0 += kScoreDepth) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = (t >> 3) + 16 * i, k = (t & 7) * 4;
      *reinterpret_cast<double2*>(&as[r][k]) = make_double2(a[i].x, a[i].y);
      *reinterpret_cast<double2*>(&as[r][k + 2]) = make_double2(a[i].z, a[i].w);
      *reinterpret_cast<double2*>(&bs[r][k]) = make_double2(b[i].x, b[i].y);
      *reinterpret_cast<double2*>(&bs[r][k + 2]) = make_double2(b[i].z, b[i].w);
    }
    __syncthreads();
    if (k0 + kScoreDepth < HD) load(k0 + kScoreDepth);
#pragma unroll 4
    for (int k = 0; k < kScoreDepth; k += 4) {
      double x[4], y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = as[wm + i * 8 + fr][k + fk], y[i] = bs[wn + i * 8 + fr][k + fk];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) mma_f64(acc[i][j][0], acc[i][j][1], x[i], y[j]);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = wm + i * 8 + fr;
    if (r >= rows) continue;
    unsigned long long* out = p.keys + (static_cast<size_t>(blockIdx.z) * p.mc + m0 + r) * p.nb;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int c = j0 + wn + j * 8 + fk * 2 + e;
        if (c < nv) out[c] = score_key(acc[i][j][e]);
      }
  }
}

// At most kFewRows rows (one token): every mean is read once, eight lanes to a block and four blocks to a
// lane at a time, so that the rows' reads from shared memory serve four blocks (one block to a lane was
// bound by them: 25 us).  Bound: reading the means (33.5 MB for 64 key heads of 1024 blocks of 128: 5 us).
constexpr int kFewRows = 4, kFewBlocks = 128;

template <int HD>
__global__ void __launch_bounds__(128, 4) block_score_few_kernel(const TopkParams p) {
  constexpr int CH = HD / 32, J = 4;  // 4-column pieces of a lane; blocks of a lane
  __shared__ __align__(16) double q[kFewRows][HD];
  const int lane = lane_id(), c = lane & 7, sub = lane >> 3;
  const int kv = p.kv0 + blockIdx.z;
  const int nv = candidate_blocks(p, kv);
  const int first = blockIdx.x * kFewBlocks, last = min(nv, first + kFewBlocks);
  let_dependents_start();
  wait_for_results();  // the mean query rows
  if (first >= nv) return;
  const float* mk = p.means + static_cast<size_t>(kv) * p.nb * HD + c * 4;
  for (int i = threadIdx.x; i < kFewRows * HD; i += 128) {
    const int r = i / HD, e = i - r * HD;
    const size_t at = (static_cast<size_t>(kv) * p.M + p.m0 + r) * HD + e;
    double x = 0.0;
    if (r < p.mc) x = p.qbar != nullptr ? static_cast<double>(p.qbar[at]) : static_cast<double>(__bfloat162float(p.Q[at]));
    q[r][e] = x;
  }
  __syncthreads();
  for (int j0 = first + warp_id() * 4 + sub; j0 - sub < last; j0 += 16 * J) {
    float4 v[J][CH];
#pragma unroll
    for (int k = 0; k < J; ++k)
#pragma unroll
      for (int h = 0; h < CH; ++h)
        v[k][h] = *reinterpret_cast<const float4*>(mk + static_cast<size_t>(min(j0 + k * 16, last - 1)) * HD + h * 32);
    double s[J][kFewRows];
#pragma unroll
    for (int k = 0; k < J; ++k)
#pragma unroll
      for (int r = 0; r < kFewRows; ++r) s[k][r] = 0.0;
#pragma unroll
    for (int h = 0; h < CH; ++h) {
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        double2 y[kFewRows];
#pragma unroll
        for (int r = 0; r < kFewRows; ++r) y[r] = *reinterpret_cast<const double2*>(&q[r][h * 32 + c * 4 + e]);
#pragma unroll
        for (int k = 0; k < J; ++k) {
          const double x0 = e == 0 ? v[k][h].x : v[k][h].z, x1 = e == 0 ? v[k][h].y : v[k][h].w;
#pragma unroll
          for (int r = 0; r < kFewRows; ++r) s[k][r] = fma(x1, y[r].y, fma(x0, y[r].x, s[k][r]));
        }
      }
    }
#pragma unroll
    for (int r = 0; r < kFewRows; ++r) {
      if (r >= p.mc) break;
#pragma unroll
      for (int o = 4; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < J; ++k) s[k][r] += __shfl_xor_sync(0xffffffffu, s[k][r], o);
#pragma unroll
      for (int k = 0; k < J; ++k) {
        const int j = j0 + k * 16;
        if (c == 0 && j < last) p.keys[(static_cast<size_t>(blockIdx.z) * p.mc + r) * p.nb + j] = score_key(s[k][r]);
      }
    }
  }
}

// The kb largest keys of a row, one warp a row with its keys in registers (nb <= 32 KPL): the kk-th
// largest high word bit by bit, by counting; the low words only where the cut falls among equal high words.
template <int KPL>
__global__ void __launch_bounds__(128) block_pick_warp_kernel(const TopkParams p, long long rows) {
  const long long r = static_cast<long long>(blockIdx.x) * 4 + warp_id();
  if (r >= rows) return;
  const int lane = lane_id();
  const int kv = p.kv0 + static_cast<int>(r / p.mc);
  const int nv = candidate_blocks(p, kv), kk = min(p.kb, nv);
  wait_for_results();  // the keys
  const unsigned long long* keys = p.keys + static_cast<size_t>(r) * p.nb;
  int32_t* out = p.blocks + (static_cast<size_t>(kv) * p.M + p.m0 + static_cast<int>(r % p.mc)) * p.kb;
  uint32_t w[KPL];  // high words, then the low words of the keys at the cut
#pragma unroll
  for (int i = 0; i < KPL; ++i) {
    const int j = i * 32 + lane;
    w[i] = j < nv ? static_cast<uint32_t>(keys[j] >> 32) : 0u;
  }
  auto count = [&](uint32_t cand) {
    int n = 0;
#pragma unroll
    for (int i = 0; i < KPL; ++i) n += w[i] >= cand ? 1 : 0;
    return __reduce_add_sync(0xffffffffu, n);
  };
  // the largest cut that at least `want` words reach; `reach` = how many do (all for cut 0)
  auto search = [&](int want, int all, int& reach) {
    uint32_t cut = 0;
    reach = all;
    for (int bit = 31; bit >= 0 && reach != want; --bit) {
      const uint32_t cand = cut | (1u << bit);
      const int n = count(cand);
      if (n >= want) cut = cand, reach = n;
    }
    return cut;
  };
  uint32_t chosen = 0, at_cut = 0;  // bit i: key 32 i + lane
  int reach;
  uint32_t cut = search(kk, nv, reach);
  int ties = 0;  // keys to take of those at the cut
#pragma unroll
  for (int i = 0; i < KPL; ++i) {
    const bool in = i * 32 + lane < nv;
    if (in && (w[i] > cut || (reach == kk && w[i] == cut))) chosen |= 1u << i;
    if (in && reach != kk && w[i] == cut) at_cut |= 1u << i;
  }
  if (reach != kk) {
    const int eq = __reduce_add_sync(0xffffffffu, __popc(at_cut));
    ties = kk - (reach - eq);
    // low words + 1 would overflow: a key at the cut whose low word is 0 counts for cut 0 alone
#pragma unroll
    for (int i = 0; i < KPL; ++i) w[i] = at_cut >> i & 1u ? static_cast<uint32_t>(keys[i * 32 + lane]) : 0u;
    cut = search(ties, eq, reach);
    uint32_t rest = 0;
#pragma unroll
    for (int i = 0; i < KPL; ++i) {
      if (!(at_cut >> i & 1u)) continue;
      if (w[i] > cut || (reach == ties && w[i] == cut)) chosen |= 1u << i;
      else if (w[i] == cut) rest |= 1u << i;
    }
    ties = reach == ties ? 0 : ties - (reach - __reduce_add_sync(0xffffffffu, __popc(rest)));
    at_cut = rest;
  }
  int base = 0, tied = 0;
  const uint32_t lt = (1u << lane) - 1u;
#pragma unroll
  for (int i = 0; i < KPL; ++i) {
    bool take = chosen >> i & 1u;
    if (ties > 0) {
      const uint32_t eq = __ballot_sync(0xffffffffu, at_cut >> i & 1u);
      take |= (at_cut >> i & 1u) && tied + __popc(eq & lt) < ties;
      tied += __popc(eq);
    }
    const uint32_t got = __ballot_sync(0xffffffffu, take);
    if (take) out[base + __popc(got & lt)] = i * 32 + lane;
    base += __popc(got);
  }
  for (int i = kk + lane; i < p.kb; i += 32) out[i] = -1;
}

constexpr int kTopkThreads = 256;
constexpr int kTopkMaxBlocks = 24576;  // keys of a row in shared memory: 8 bytes each

// The same for longer rows, a CTA a row with its keys in shared memory.  Two bits a step: the counts of three
// candidates in one 64-bit sum.
__global__ void __launch_bounds__(kTopkThreads) block_pick_kernel(const TopkParams p, long long rows) {
  extern __shared__ __align__(16) unsigned long long tkeys[];  // nb
  constexpr int WARPS = kTopkThreads / 32;
  __shared__ unsigned long long red[2][WARPS];
  const int t = threadIdx.x, lane = lane_id(), warp = warp_id();
  wait_for_results();  // the keys
  for (long long r = blockIdx.x; r < rows; r += gridDim.x) {
    const int kv = p.kv0 + static_cast<int>(r / p.mc);
    const int nv = candidate_blocks(p, kv), kk = min(p.kb, nv);
    const unsigned long long* keys = p.keys + static_cast<size_t>(r) * p.nb;
    int32_t* out = p.blocks + (static_cast<size_t>(kv) * p.M + p.m0 + static_cast<int>(r % p.mc)) * p.kb;
    __syncthreads();  // the row before this one is done with the keys
    for (int j = t; j < nv; j += kTopkThreads) tkeys[j] = keys[j];
    __syncthreads();
    // keys that reach c1, c2 and c3 (c1 <= c2 <= c3): counts of at most 24576 in 16 bits each
    int turn = 0;
    auto count = [&](unsigned long long c1, unsigned long long c2, unsigned long long c3) {
      uint32_t lo = 0, hi = 0;
      for (int j = t; j < nv; j += kTopkThreads) {
        const unsigned long long k = tkeys[j];
        lo += (k >= c1 ? 1u : 0u) + (k >= c2 ? 1u << 16 : 0u);
        hi += k >= c3 ? 1u : 0u;
      }
      lo = __reduce_add_sync(0xffffffffu, lo);
      hi = __reduce_add_sync(0xffffffffu, hi);
      if (lane == 0) red[turn][warp] = static_cast<unsigned long long>(hi) << 32 | lo;
      __syncthreads();
      unsigned long long n = 0;
#pragma unroll
      for (int i = 0; i < WARPS; ++i) n += red[turn][i];
      turn ^= 1;  // the sums of the call before this one may still be read
      return n;
    };
    // the kk-th largest key, two bits a step; at_cut = keys that reach it
    unsigned long long cut = 0;
    int at_cut = nv;
    for (int bit = 62; bit >= 0 && at_cut != kk; bit -= 2) {
      const unsigned long long one = 1ull << bit;
      const unsigned long long n = count(cut | one, cut | (one << 1), cut | (one << 1) | one);
      const int n1 = static_cast<int>(n & 0xffff), n2 = static_cast<int>(n >> 16 & 0xffff), n3 = static_cast<int>(n >> 32);
      if (n3 >= kk) cut |= (one << 1) | one, at_cut = n3;
      else if (n2 >= kk) cut |= one << 1, at_cut = n2;
      else if (n1 >= kk) cut |= one, at_cut = n1;
    }
    // keys above the cut, and of those equal to it the first `ties`
    int ties = kk;
    if (at_cut != kk) ties = kk - (cut == ~0ull ? 0 : static_cast<int>(count(cut + 1, cut + 1, cut + 1) & 0xffff));
    int base = 0, eq_base = 0;
    for (int j0 = 0; j0 < nv; j0 += kTopkThreads) {
      const int j = j0 + t;
      const unsigned long long k = j < nv ? tkeys[j] : 0ull;
      const bool eq = j < nv && at_cut != kk && k == cut;
      const bool gt = j < nv && (at_cut != kk ? k > cut : k >= cut);
      // counts of both kinds in the warps before this one, packed in one word
      const unsigned beq = __ballot_sync(0xffffffffu, eq), bgt = __ballot_sync(0xffffffffu, gt);
      if (lane == 0) red[turn][warp] = __popc(bgt) | (__popc(beq) << 16);
      __syncthreads();
      int gt_before = 0, eq_before = 0, gt_all = 0, eq_all = 0;
#pragma unroll
      for (int i = 0; i < WARPS; ++i) {
        const int v = static_cast<int>(red[turn][i]);
        if (i < warp) gt_before += v & 0xffff, eq_before += v >> 16;
        gt_all += v & 0xffff, eq_all += v >> 16;
      }
      turn ^= 1;
      const unsigned lt = (1u << lane) - 1u;
      const int eq_rank = eq_base + eq_before + __popc(beq & lt);  // this key's place among the equal ones
      const int gt_rank = base + gt_before + __popc(bgt & lt);     // chosen keys above the cut before it
      if (gt || (eq && eq_rank < ties)) out[gt_rank + min(eq_rank, ties)] = j;
      base += gt_all;
      eq_base += eq_all;
    }
    for (int i = kk + t; i < p.kb; i += kTopkThreads) out[i] = -1;
  }
}

// ---------------------------------------------------------------------------------- 8-bit store
// One block of tokens of one head: scale = max(amax / 448, 2^-100) (1 for a block of zeros), values
// e4m3(x / scale), round to nearest even, saturating.  amax runs over the finite values; NaN is kept
// as NaN and an infinity becomes the largest value.  The quotient is the rounded fp32 one, so that a
// value half way between two e4m3 numbers goes to the even one.
struct CacheWriteParams {
  const __nv_bfloat16* X[2];  // K, V: [B, H, n, d]
  uint8_t* Y[2];              // [B, H, cap, d]
  float* scale[2];            // [B, H, cap / BK]
  float* means;               // [B, H, cap / BK, d] of K, nullable
  const int32_t* len;         // [B], nullable: valid rows of this write
  int H, n, cap, start, BK, nb;
};

constexpr int kCacheThreads = 256;

// Four e4m3 values of x / scale: the rounded fp32 quotient, to the nearest e4m3.  With the rounded reciprocal
// y of the scale at hand, q = RN(x y) and RN(q + RN(x - q scale) y) is the rounded quotient (P. Markstein,
// Computation of elementary functions on the IBM RISC System/6000, 1990, for a q within a step of it; for
// the quotients that occur here, 8-bit x by the fp32 rounding of an 8-bit number / 448, all mantissas are
// checked on the CPU): two multiply-adds where a division is some ten instructions and one of the XU's.
template <bool PLAIN>
__device__ __forceinline__ unsigned quantise4(const float* x, float scale, float inv) {
  float y[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float q = x[e] * inv;
    y[e] = PLAIN ? fmaf(fmaf(-q, scale, x[e]), inv, q) : x[e] / scale;
  }
  const unsigned lo = __nv_cvt_float2_to_fp8x2(make_float2(y[0], y[1]), __NV_SATFINITE, __NV_E4M3);
  const unsigned hi = __nv_cvt_float2_to_fp8x2(make_float2(y[2], y[3]), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// One CTA a block, its rows in registers between the maximum and the rounding, so that they are read once.
// NIT: passes of the CTA over a block (its rows / (256 / (HD / 16)), at least 1).  Bound: device memory (480p
// clip, 594 MB: 113 us, 80 % of the copy rate), which wants CTAs to overlap: five an SM; four 115 us, three
// 119, and with a division for every value 187.
template <int HD, int NIT>
__global__ void __launch_bounds__(kCacheThreads, 5) cache_write_kernel(const CacheWriteParams p) {
  constexpr int CG = HD / 16;                       // 16-element pieces of a row
  constexpr int RG = kCacheThreads / CG;            // rows of one pass
  constexpr int WARPS = kCacheThreads / 32;
  __shared__ unsigned wmax[WARPS];
  __shared__ double wsum[WARPS][HD];
  const int j = blockIdx.x, bh = blockIdx.y, which = blockIdx.z;
  const int rows = min(p.BK, valid_rows(p.len, bh / p.H, p.n) - j * p.BK);
  if (rows <= 0) return;
  const int t = threadIdx.x, lane = lane_id(), warp = warp_id();
  const int c = t % CG, r0 = t / CG;
  const __nv_bfloat16* src = p.X[which] + (static_cast<size_t>(bh) * p.n + static_cast<size_t>(j) * p.BK) * HD + c * 16;
  uint4 u[NIT][2];
  unsigned top = 0;  // largest finite |x| as bf16 bits
#pragma unroll
  for (int i = 0; i < NIT; ++i) {
    const int r = r0 + i * RG;
    if (r < rows) {
      const uint4* s = reinterpret_cast<const uint4*>(src + static_cast<size_t>(r) * HD);
      u[i][0] = s[0];
      u[i][1] = s[1];
    } else {
      u[i][0] = u[i][1] = make_uint4(0u, 0u, 0u, 0u);
    }
  }
  // |x| as 16-bit integers, two at a time; infinities and NaN, which lie above every number, are left
  // out in a second look where there are any
  unsigned pairs = 0;
#pragma unroll
  for (int i = 0; i < NIT; ++i) {
    const unsigned* w = reinterpret_cast<const unsigned*>(u[i]);
#pragma unroll
    for (int e = 0; e < 8; ++e) pairs = __vmaxu2(pairs, w[e] & 0x7fff7fffu);
  }
  top = max(pairs & 0xffffu, pairs >> 16);
  const bool special = top >= 0x7f80u;
  if (special) {
    top = 0;
#pragma unroll
    for (int i = 0; i < NIT; ++i) {
      const unsigned* w = reinterpret_cast<const unsigned*>(u[i]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const unsigned a = w[e] & 0x7fffu, b = (w[e] >> 16) & 0x7fffu;
        top = max(top, a < 0x7f80u ? a : 0u);
        top = max(top, b < 0x7f80u ? b : 0u);
      }
    }
  }
  top = __reduce_max_sync(0xffffffffu, top);
  if (lane == 0) wmax[warp] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < WARPS; ++i) top = max(top, wmax[i]);
  const float amax = __uint_as_float(top << 16);
  const float scale = top == 0u ? 1.f : fmaxf(amax / 448.f, 7.8886090522101181e-31f);  // 2^-100
  const float inv = 1.f / scale;
  const size_t blk = static_cast<size_t>(bh) * (p.cap / p.BK) + p.start / p.BK + j;
  if (t == 0) p.scale[which][blk] = scale;
  uint8_t* dst = p.Y[which] + (static_cast<size_t>(bh) * p.cap + p.start + static_cast<size_t>(j) * p.BK) * HD + c * 16;
  auto store = [&](auto plain) {
#pragma unroll
    for (int i = 0; i < NIT; ++i) {
      const int r = r0 + i * RG;
      if (r < rows) {
        unsigned w[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float f[8];
          unpack8(u[i][h], f);
          w[2 * h] = quantise4<decltype(plain)::value>(f, scale, inv);
          w[2 * h + 1] = quantise4<decltype(plain)::value>(f + 4, scale, inv);
        }
        *reinterpret_cast<uint4*>(dst + static_cast<size_t>(r) * HD) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  };
  // infinities and NaN, and scales so small that a remainder could underflow, are divided
  if (!special && scale >= 8.2718061255302767e-25f) store(std::true_type{});  // 2^-80
  else store(std::false_type{});
  if (which == 0 && p.means != nullptr) {
    // the block's mean key, of the values before rounding (fp64 sums as in block_means_kernel)
    // eight columns at a time: the sums of sixteen would not fit beside the tile
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      double acc[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = 0.0;
#pragma unroll
      for (int i = 0; i < NIT; ++i) {
        float f[8];
        unpack8(u[i][half], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] += static_cast<double>(f[e]);
      }
#pragma unroll
      for (int o = CG; o < 32; o <<= 1)
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] += __shfl_xor_sync(0xffffffffu, acc[e], o);
      if (lane < CG)
#pragma unroll
        for (int e = 0; e < 8; ++e) wsum[warp][c * 16 + half * 8 + e] = acc[e];
    }
    __syncthreads();
    if (t < HD) {
      double s = 0.0;
#pragma unroll
      for (int i = 0; i < WARPS; ++i) s += wsum[i][t];
      p.means[blk * HD + t] = static_cast<float>(s / static_cast<double>(rows));
    }
  }
}

}  // namespace mcs
