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
  int B, H, Hkv, Nq, Nk, C, BK, nb, GQ, kb;
  float scale_log2;         // scale * log2(e)
};

constexpr int kSimpleWarps = 4;

template <bool KV8>
__device__ __forceinline__ void load_kv8(const void* base, size_t at, float* f) {
  if constexpr (KV8) {
    const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(base) + at);
    const __nv_fp8x2_storage_t* w = reinterpret_cast<const __nv_fp8x2_storage_t*>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(w[i], __NV_E4M3)));
      f[2 * i] = v.x;
      f[2 * i + 1] = v.y;
    }
  } else {
    unpack8(*reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + at), f);
  }
}

// One warp per query row: 32 keys at a time (a lane scores one key), then the lanes split the columns.
template <int HD, bool KV8>
__global__ void __launch_bounds__(kSimpleWarps * 32) block_attn_simple_kernel(const BlockAttnParams p) {
  __shared__ float sq[kSimpleWarps][HD];
  const int warp = warp_id(), lane = lane_id();
  const long long row = static_cast<long long>(blockIdx.x) * kSimpleWarps + warp;
  if (row >= static_cast<long long>(p.B) * p.H * p.Nq) return;
  const int bh = static_cast<int>(row / p.Nq), i = static_cast<int>(row - static_cast<long long>(bh) * p.Nq);
  const int b = bh / p.H, g = i / p.C;
  const int bkv = b * p.Hkv + (bh - b * p.H) / (p.H / p.Hkv);
  const int n = valid_rows(p.len, b, p.Nk);
  for (int c = lane; c < HD; c += 32) sq[warp][c] = __bfloat162float(p.Q[static_cast<size_t>(row) * HD + c]) * p.scale_log2;
  __syncwarp();
  constexpr int PER = HD / 32;
  float o[PER], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < PER; ++e) o[e] = 0.f;
  const int32_t* list = p.blocks ? p.blocks + (static_cast<size_t>(bh) * p.GQ + g) * p.kb : nullptr;
  for (int t = 0; t < p.kb; ++t) {
    const int blk = list ? list[t] : t;
    if (blk < 0) break;
    if (blk >= p.nb) {
      raise_status(kStatusBadIndex);
      continue;
    }
    const float ks = KV8 ? p.ks[static_cast<size_t>(bkv) * p.nb + blk] : 1.f;
    const float vs = KV8 ? p.vs[static_cast<size_t>(bkv) * p.nb + blk] : 1.f;
    for (int j0 = blk * p.BK; j0 < min(n, (blk + 1) * p.BK); j0 += 32) {
      const bool live = j0 + lane < n;
      float x = -INFINITY;
      if (live) {
        const size_t at = (static_cast<size_t>(bkv) * p.Nk + j0 + lane) * HD;
        float acc = 0.f;
        for (int c = 0; c < HD; c += 8) {
          float f[8];
          load_kv8<KV8>(p.K, at + c, f);
#pragma unroll
          for (int e = 0; e < 8; ++e) acc = fmaf(sq[warp][c + e], f[e], acc);
        }
        x = acc * ks;
      }
      float mx = x;
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
      const float mn = fmaxf(m, mx);
      const float ref = mn == -INFINITY ? 0.f : mn;
      const float alpha = exp2f(m - ref);
      const float w = live ? exp2f(x - ref) : 0.f;
      m = mn;
      l = l * alpha + w;
#pragma unroll
      for (int e = 0; e < PER; ++e) o[e] *= alpha;
      const int keys = min(32, n - j0);
      for (int k = 0; k < keys; ++k) {
        const float wv = __shfl_sync(0xffffffffu, w, k) * vs;
        const size_t at = (static_cast<size_t>(bkv) * p.Nk + j0 + k) * HD;
#pragma unroll
        for (int e = 0; e < PER; ++e) {
          float v;
          if constexpr (KV8) {
            const __half_raw r = __nv_cvt_fp8_to_halfraw(static_cast<const uint8_t*>(p.V)[at + lane + 32 * e], __NV_E4M3);
            v = __half2float(__half(r));
          } else {
            v = __bfloat162float(static_cast<const __nv_bfloat16*>(p.V)[at + lane + 32 * e]);
          }
          o[e] = fmaf(wv, v, o[e]);
        }
      }
    }
  }
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) l += __shfl_xor_sync(0xffffffffu, l, s);
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int e = 0; e < PER; ++e) {
    const size_t at = static_cast<size_t>(row) * HD + lane + 32 * e;
    float v = o[e] * inv;
    if (p.R != nullptr) v += __bfloat162float(p.R[at]);
    p.out[at] = __float2bfloat16(v);
  }
  if (p.lse != nullptr && lane == 0) p.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

}  // namespace mcs
