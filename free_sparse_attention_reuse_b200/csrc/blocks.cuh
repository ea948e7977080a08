// Key blocks: their means, their choice by a cheap score, and the 8-bit store that holds them.
#pragma once

#include <cuda_fp8.h>

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

constexpr int kMeansThreads = 256;

template <int HD>
__global__ void __launch_bounds__(kMeansThreads) block_means_kernel(const MeansParams p) {
  constexpr int LPR = HD / 8, RPW = 32 / LPR;
  const int lane = lane_id(), c = lane % LPR, sub = lane / LPR;
  const long long blk = static_cast<long long>(blockIdx.x) * (kMeansThreads / 32) + warp_id();
  if (blk >= p.blocks) return;
  const long long bh = blk / p.nb;
  const int j = static_cast<int>(blk - bh * p.nb);
  const int n = min(p.BK, valid_rows(p.len, static_cast<int>(bh / p.H), p.N) - j * p.BK);
  const __nv_bfloat16* row = p.X + (static_cast<size_t>(bh) * p.N + static_cast<size_t>(j) * p.BK) * HD + c * 8;
  double acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.0;
#pragma unroll 4
  for (int r = sub; r < n; r += RPW) {
    float f[8];
    unpack8(*reinterpret_cast<const uint4*>(row + static_cast<size_t>(r) * HD), f);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] += static_cast<double>(f[i]);
  }
#pragma unroll
  for (int o = LPR; o < 32; o <<= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
  if (sub == 0) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = n > 0 ? static_cast<float>(acc[i] / static_cast<double>(n)) : 0.f;
    float4* out = reinterpret_cast<float4*>(p.means + static_cast<size_t>(blk) * HD + c * 8);
    out[0] = make_float4(f[0], f[1], f[2], f[3]);
    out[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
}

// ---------------------------------------------------------------------------------- choice
// Order of fp64 scores as unsigned integers; NaN below every number, both zeros alike.
__device__ __forceinline__ unsigned long long score_key(double s) {
  if (s != s) return 0ull;
  if (s == 0.0) s = 0.0;
  const unsigned long long u = static_cast<unsigned long long>(__double_as_longlong(s));
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

struct TopkParams {
  const __nv_bfloat16* Q;  // [B, H, Nq, d]
  const float* means;      // [B, Hkv, nb, d]
  const int32_t* len;      // [B], nullable
  int32_t* blocks;         // [B, H, GQ, kb]
  int H, Hkv, Nq, Nk, GQ, C, BK, nb, kb;
};

constexpr int kTopkThreads = 256;
constexpr int kTopkMaxBlocks = 24576;  // keys of a row in shared memory: 8 bytes each

// One query block: qbar (mean of its rows), s_j = qbar . kbar_j, the kb largest, ties to the lower j.
// Scores are fp64 (the fp32 means' products are exact there), so that the choice is the definition's
// and not the summation order's.
template <int HD>
__global__ void __launch_bounds__(kTopkThreads) block_topk_kernel(const TopkParams p) {
  extern __shared__ __align__(16) unsigned long long tkeys[];  // nb
  __shared__ double qbar[HD];
  __shared__ int red[kTopkThreads / 32];
  const int t = threadIdx.x, lane = lane_id(), warp = warp_id();
  const int g = blockIdx.x, bh = blockIdx.y;
  const int b = bh / p.H, h = bh - b * p.H;
  const int nq = min(p.C, p.Nq - g * p.C);
  if (t < HD) {
    const __nv_bfloat16* q = p.Q + (static_cast<size_t>(bh) * p.Nq + static_cast<size_t>(g) * p.C) * HD + t;
    double acc = 0.0;
    for (int r = 0; r < nq; ++r) acc += static_cast<double>(__bfloat162float(q[static_cast<size_t>(r) * HD]));
    qbar[t] = static_cast<double>(static_cast<float>(acc / static_cast<double>(nq)));
  }
  __syncthreads();
  const int nv = (valid_rows(p.len, b, p.Nk) + p.BK - 1) / p.BK;  // blocks with a valid key
  const int kk = min(p.kb, nv);
  const float* mk = p.means + (static_cast<size_t>(b) * p.Hkv + h / (p.H / p.Hkv)) * p.nb * HD;
  for (int j = t; j < nv; j += kTopkThreads) {
    double acc = 0.0;
    for (int c = 0; c < HD; ++c) acc = fma(qbar[c], static_cast<double>(mk[static_cast<size_t>(j) * HD + c]), acc);
    tkeys[j] = score_key(acc);
  }
  __syncthreads();
  auto count = [&](unsigned long long cand) {  // keys >= cand
    int n = 0;
    for (int j = t; j < nv; j += kTopkThreads) n += tkeys[j] >= cand ? 1 : 0;
    n = __reduce_add_sync(0xffffffffu, n);
    __syncthreads();
    if (lane == 0) red[warp] = n;
    __syncthreads();
    n = 0;
    for (int i = 0; i < kTopkThreads / 32; ++i) n += red[i];
    return n;
  };
  // the kk-th largest key, bit by bit; `above` = keys larger than it once every bit is fixed
  unsigned long long cut = 0;
  int at_cut = nv;  // keys >= cut
  for (int bit = 63; bit >= 0 && at_cut != kk; --bit) {
    const unsigned long long cand = cut | (1ull << bit);
    const int n = count(cand);
    if (n >= kk) {
      cut = cand;
      at_cut = n;
    }
  }
  // keys above the cut, and of those equal to it the first `ties`
  int ties = kk;
  if (at_cut != kk) ties = kk - (cut == ~0ull ? 0 : count(cut + 1));
  int32_t* out = p.blocks + (static_cast<size_t>(bh) * p.GQ + g) * p.kb;
  int base = 0, eq_base = 0;
  for (int j0 = 0; j0 < nv; j0 += kTopkThreads) {
    const int j = j0 + t;
    const unsigned long long k = j < nv ? tkeys[j] : 0ull;
    const bool eq = j < nv && at_cut != kk && k == cut;
    const bool gt = j < nv && (at_cut != kk ? k > cut : k >= cut);
    // counts of both kinds in the warps before this one, packed in one word
    const unsigned beq = __ballot_sync(0xffffffffu, eq), bgt = __ballot_sync(0xffffffffu, gt);
    __syncthreads();
    if (lane == 0) red[warp] = __popc(bgt) | (__popc(beq) << 16);
    __syncthreads();
    int gt_before = 0, eq_before = 0, gt_all = 0, eq_all = 0;
    for (int i = 0; i < kTopkThreads / 32; ++i) {
      const int v = red[i];
      if (i < warp) gt_before += v & 0xffff, eq_before += v >> 16;
      gt_all += v & 0xffff, eq_all += v >> 16;
    }
    const unsigned lt = (1u << lane) - 1u;
    const int eq_rank = eq_base + eq_before + __popc(beq & lt);     // this key's place among the equal ones
    const int gt_rank = base + gt_before + __popc(bgt & lt);        // chosen keys above the cut before it
    if (gt || (eq && eq_rank < ties)) out[gt_rank + min(eq_rank, ties)] = j;
    base += gt_all;
    eq_base += eq_all;
  }
  for (int i = kk + t; i < p.kb; i += kTopkThreads) out[i] = -1;
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

template <int HD>
__global__ void __launch_bounds__(kCacheThreads) cache_write_kernel(const CacheWriteParams p) {
  constexpr int CG = HD / 16;                       // 16-element pieces of a row
  constexpr int RG = kCacheThreads / CG;            // rows of one pass
  constexpr int NIT = 128 / RG;                     // passes over the largest block
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
  top = __reduce_max_sync(0xffffffffu, top);
  if (lane == 0) wmax[warp] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < WARPS; ++i) top = max(top, wmax[i]);
  const float amax = __uint_as_float(top << 16);
  const float scale = top == 0u ? 1.f : fmaxf(amax / 448.f, 7.8886090522101181e-31f);  // 2^-100
  const size_t blk = static_cast<size_t>(bh) * (p.cap / p.BK) + p.start / p.BK + j;
  if (t == 0) p.scale[which][blk] = scale;
  uint8_t* dst = p.Y[which] + (static_cast<size_t>(bh) * p.cap + p.start + static_cast<size_t>(j) * p.BK) * HD + c * 16;
#pragma unroll
  for (int i = 0; i < NIT; ++i) {
    const int r = r0 + i * RG;
    if (r < rows) {
      float f[16];
      unpack8(u[i][0], f);
      unpack8(u[i][1], f + 8);
      unsigned w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const unsigned lo = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * e] / scale, f[4 * e + 1] / scale), __NV_SATFINITE, __NV_E4M3);
        const unsigned hi = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * e + 2] / scale, f[4 * e + 3] / scale), __NV_SATFINITE, __NV_E4M3);
        w[e] = lo | (hi << 16);
      }
      *reinterpret_cast<uint4*>(dst + static_cast<size_t>(r) * HD) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  if (which == 0 && p.means != nullptr) {
    // the block's mean key, of the values before rounding (fp64 sums as in block_means_kernel)
    double acc[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[e] = 0.0;
#pragma unroll
    for (int i = 0; i < NIT; ++i) {
      float f[16];
      unpack8(u[i][0], f);
      unpack8(u[i][1], f + 8);
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[e] += static_cast<double>(f[e]);
    }
#pragma unroll
    for (int o = CG; o < 32; o <<= 1)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[e] += __shfl_xor_sync(0xffffffffu, acc[e], o);
    if (lane < CG)
#pragma unroll
      for (int e = 0; e < 16; ++e) wsum[warp][c * 16 + e] = acc[e];
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
