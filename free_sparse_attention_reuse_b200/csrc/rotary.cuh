// From a layer's projections to attention-ready tensors in one pass: RMS norm of q and k, rotary
// positions over several axes (time, height, width), and the change from token-major
// [B, N, H, d] views to head-major [B, H, N, d].
//
// Mathematics.  For a q or k row x of d elements (fp32 throughout, one rounding to bf16 at the end):
//   x <- x * rsqrt(mean(x^2) + eps) * w     mean over the row (head norm) or over the token's H rows
//                                           (token norm); left out without a norm
//   a_i = pos[axis(i)] * theta^(-2 j / d_axis)   pair i is the j-th pair of its axis's section
//   (y1, y2) = (x1 cos a_i - x2 sin a_i, x1 sin a_i + x2 cos a_i)
// Pair i is (x[2i], x[2i+1]) (adjacent) or (x[i], x[i + r/2]) (halves, r = sum of the axes' sizes);
// elements from r on are only normalised.  v is copied.
//
// The angle is formed in turns and in fp64 (frequencies come divided by 2 pi from the host), reduced
// to [-1/2, 1/2] turns there, and only then rounded to fp32, so positions far from the origin lose
// nothing: fp32 holds an angle of 10^5 radians to 2^-7 only.
#pragma once

#include "sm100.cuh"

namespace mcs {

constexpr int kRotMaxAxes = 4;
constexpr int kRotThreads = 256;
constexpr int kRotMaxTokens = 16;  // tokens of a CTA

struct RotaryParams {
  const __nv_bfloat16* x[3];  // q, k, v (nullable k, v)
  __nv_bfloat16* y[3];
  const void* w[2];           // norm weights of q and k (nullable), fp32 or bf16
  long long sb[3], sn[3], sh[3];
  int heads[3];
  const void* pos;            // [N, A] or [B, N, A], int32 or fp32
  double turns[64];           // frequency of pair i in turns per unit of position
  unsigned char axis[64];     // its axis
  int B, N, A, half;          // half = number of rotated pairs
  int T, tiles;               // tokens per CTA, CTAs per batch entry
  int pos_float, pos_batch, w_bf16;
  float eps;
};

enum RotaryNorm : int { kNormNone = 0, kNormHead = 1, kNormToken = 2 };

__device__ __forceinline__ void unpack8(const uint4& u, float* f) {
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = __bfloat1622float2(h[i]);
    f[2 * i] = t.x;
    f[2 * i + 1] = t.y;
  }
}
__device__ __forceinline__ uint4 pack8(const float* f) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

// 8 norm weights from element `at` on.
__device__ __forceinline__ void load_w8(const void* w, int bf16, size_t at, float* f) {
  if (bf16) {
    unpack8(*reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(w) + at), f);
  } else {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(w) + at);
    const float4 a = p[0], b = p[1];
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  }
}

// One CTA: T consecutive tokens of one batch entry, all heads of q, k and v; the sines and cosines
// of a token are made once and shared by all its rows.  HD/8 lanes hold a row, 8 elements each.
template <int HD, int NORM, bool HALVES>
__global__ void __launch_bounds__(kRotThreads) rotary_kernel(const __grid_constant__ RotaryParams p) {
  constexpr int LPR = HD / 8;            // lanes per row
  constexpr int RPW = 32 / LPR;          // rows per warp and pass
  constexpr int WARPS = kRotThreads / 32;
  __shared__ float2 cs[kRotMaxTokens * (HD / 2)];
  __shared__ float rs[2][kRotMaxTokens];
  const int b = blockIdx.x / p.tiles, n0 = (blockIdx.x - b * p.tiles) * p.T;
  const int nt = min(p.T, p.N - n0);
  const int warp = warp_id(), lane = lane_id();
  const int c = lane % LPR, sub = lane / LPR;

  for (int i = threadIdx.x; i < nt * p.half; i += kRotThreads) {
    const int t = i / p.half, j = i - t * p.half;
    const size_t at = (static_cast<size_t>(p.pos_batch ? b : 0) * p.N + n0 + t) * p.A + p.axis[j];
    const double x = p.pos_float ? static_cast<double>(static_cast<const float*>(p.pos)[at])
                                 : static_cast<double>(static_cast<const int32_t*>(p.pos)[at]);
    const double a = x * p.turns[j];
    float2 v;
    sincospif(2.f * static_cast<float>(a - rint(a)), &v.y, &v.x);
    cs[t * (HD / 2) + j] = v;
  }
  if (NORM == kNormToken) {
    // 1 / rms of each token's whole q and k: one warp per (tensor, token)
    for (int u = warp; u < 2 * nt; u += WARPS) {
      const int s = u / nt, t = u - s * nt;
      if (p.x[s] == nullptr) continue;
      const __nv_bfloat16* row = p.x[s] + b * p.sb[s] + (n0 + t) * p.sn[s] + c * 8;
      float ss = 0.f;
      for (int h = sub; h < p.heads[s]; h += RPW) {
        float f[8];
        unpack8(*reinterpret_cast<const uint4*>(row + h * p.sh[s]), f);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(f[i], f[i], ss);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (lane == 0) rs[s][t] = rsqrtf(ss / static_cast<float>(p.heads[s] * HD) + p.eps);
    }
  }
  __syncthreads();

  for (int s = 0; s < 3; ++s) {
    if (p.x[s] == nullptr) continue;
    const int rows = p.heads[s] * nt;  // head-major, so that a head's tokens are written together
    for (int r0 = warp * RPW; r0 < rows; r0 += WARPS * RPW) {
      const int r = r0 + sub;
      const bool live = r < rows;
      const int h = live ? r / nt : 0, t = live ? r - h * nt : 0;
      uint4 u = make_uint4(0u, 0u, 0u, 0u);
      if (live)
        u = *reinterpret_cast<const uint4*>(p.x[s] + b * p.sb[s] + (n0 + t) * p.sn[s] + h * p.sh[s] + c * 8);
      if (s < 2) {
        float f[8];
        unpack8(u, f);
        if (NORM != kNormNone) {
          float k;
          if (NORM == kNormHead) {
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(f[i], f[i], ss);
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            k = rsqrtf(ss * (1.f / HD) + p.eps);
          } else {
            k = rs[s][t];
          }
          if (p.w[s] != nullptr) {
            float w[8];
            load_w8(p.w[s], p.w_bf16, (NORM == kNormToken ? static_cast<size_t>(h) * HD : 0) + c * 8, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = f[i] * k * w[i];
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] *= k;
          }
        }
        const float2* ct = cs + t * (HD / 2);
        if (!HALVES) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int j = c * 4 + i;
            if (j < p.half) {
              const float2 v = ct[j];
              const float x1 = f[2 * i], x2 = f[2 * i + 1];
              f[2 * i] = x1 * v.x - x2 * v.y;
              f[2 * i + 1] = x1 * v.y + x2 * v.x;
            }
          }
        } else {
          // the partner elements are the same 8 slots of the lane half/8 further (or back)
          const int hc = p.half / 8;
          const bool lo = c < hc, hi = !lo && c < 2 * hc;
          const int src = lane + (lo ? hc : hi ? -hc : 0);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float o = __shfl_sync(0xffffffffu, f[i], src);
            if (lo || hi) {
              const float2 v = ct[c * 8 + i - (hi ? p.half : 0)];
              f[i] = lo ? f[i] * v.x - o * v.y : o * v.y + f[i] * v.x;
            }
          }
        }
        u = pack8(f);
      }
      if (live)
        *reinterpret_cast<uint4*>(p.y[s] + ((static_cast<size_t>(b) * p.heads[s] + h) * p.N + n0 + t) * HD + c * 8) = u;
    }
  }
}

}  // namespace mcs
