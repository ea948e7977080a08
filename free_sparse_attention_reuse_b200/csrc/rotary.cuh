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
constexpr int kRotRows = 4;  // rows that a group has in flight

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
// A kernel launched as another's dependent starts while that one still runs and waits here for its results
// (at once where it was launched the plain way); the other lets it start with let_dependents_start.
__device__ __forceinline__ void wait_for_results() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_dependents_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// 16 bytes that no one writes during the kernel; loads in a row stay in a row, so that all of them are in
// flight before the first is used.
__device__ __forceinline__ uint4 load16(const void* p) {
  uint4 u;
  asm volatile("ld.global.nc.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "l"(p));
  return u;
}
__device__ __forceinline__ uint4 pack8(const float* f) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

__device__ __forceinline__ uint2 load8(const void* p) {
  uint2 u;
  asm volatile("ld.global.nc.v2.u32 {%0,%1}, [%2];" : "=r"(u.x), "=r"(u.y) : "l"(p));
  return u;
}

// 4 norm weights from element `at` on.
__device__ __forceinline__ void load_w4(const void* w, int bf16, size_t at, float* f) {
  if (bf16) {
    const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(w) + at);
    const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.x));
    const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.y));
    f[0] = a.x, f[1] = a.y, f[2] = b.x, f[3] = b.y;
  } else {
    const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(w) + at);
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
  }
}

// One CTA: T consecutive tokens of one batch entry.  HD / 8 lanes make a group and hold a row, 8 elements
// each; a group keeps to one token, whose sines and cosines stay in its registers, and goes through its
// heads (through a share of them where there are more groups than tokens), kRotRows rows in flight.  With
// pairs in halves a lane holds four elements of the first half and their four partners (two 8-byte
// pieces), so that nothing is exchanged; lanes beyond the halves hold eight that are not turned.
// Bound: device memory (480p clip, head norm: 198 us, 91 % of the copy rate; one row in flight and the sines
// in shared memory left it at 58 %; partners by shuffles left the halves form at 143 us for 403 MB,
// three CTAs an SM instead of four at 117 against 105, five at 137).
template <int HD, int NORM, bool HALVES>
__global__ void __launch_bounds__(kRotThreads, 4) rotary_kernel(const __grid_constant__ RotaryParams p) {
  constexpr int LPR = HD / 8;                 // lanes of a group
  constexpr int GROUPS = kRotThreads / LPR;   // 16 or 32
  __shared__ float part[2][GROUPS];
  const int b = blockIdx.x / p.tiles, n0 = (blockIdx.x - b * p.tiles) * p.T;
  const int group = threadIdx.x / LPR, c = threadIdx.x % LPR;
  const int t = group % p.T, share = group / p.T, shares = GROUPS / p.T;
  const bool live = n0 + t < p.N;
  const int n = live ? n0 + t : p.N - 1;  // (idle groups follow along on the last token and store nothing)

  // this lane's elements: e0 .. e0 + 3 and e1 .. e1 + 3, pairs p0 .. p0 + 3 where it turns any
  int e0 = c * 8, e1 = e0 + 4, p0 = c * 4;
  bool turns = p0 < p.half;
  if (HALVES) {
    turns = c * 4 < p.half;
    e0 = turns ? c * 4 : 2 * p.half + (c - p.half / 4) * 8;
    e1 = turns ? p.half + c * 4 : e0 + 4;
  }
  const bool whole = 2 * p.half == HD;  // every element turns
  float2 cs[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    cs[i] = make_float2(1.f, 0.f);
    if (turns && p0 + i < p.half) {
      const size_t at = (static_cast<size_t>(p.pos_batch ? b : 0) * p.N + n) * p.A + p.axis[p0 + i];
      const double x = p.pos_float ? static_cast<double>(static_cast<const float*>(p.pos)[at])
                                   : static_cast<double>(static_cast<const int32_t*>(p.pos)[at]);
      const double a = x * p.turns[p0 + i];
      sincospif(2.f * static_cast<float>(a - rint(a)), &cs[i].y, &cs[i].x);
    }
  }
  auto source = [&](int s) { return p.x[s] + b * p.sb[s] + n * p.sn[s]; };
  auto load = [&](const __nv_bfloat16* row) {
    if (!HALVES) return load16(row + e0);
    const uint2 x = load8(row + e0), y = load8(row + e1);
    return make_uint4(x.x, x.y, y.x, y.y);
  };
  // 8 norm weights of this lane's elements
  auto load_w = [&](const void* w, size_t at, float* f) {
    load_w4(w, p.w_bf16, at + e0, f);
    load_w4(w, p.w_bf16, at + e1, f + 4);
  };

  float rs[2] = {1.f, 1.f};
  if (NORM == kNormToken) {
    // 1 / rms of the token's whole q and k (the rows are read again below, from L2)
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      float ss = 0.f;
      if (p.x[s] != nullptr) {
        const __nv_bfloat16* row = source(s);
        for (int h0 = share; h0 < p.heads[s]; h0 += 8 * shares) {
          uint4 u[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int h = h0 + k * shares;
            u[k] = h < p.heads[s] ? load16(row + h * p.sh[s] + c * 8) : make_uint4(0u, 0u, 0u, 0u);
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            float f[8];
            unpack8(u[k], f);
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(f[i], f[i], ss);
          }
        }
      }
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (c == 0) part[s][group] = ss;
    }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      float ss = 0.f;
      for (int i = 0; i < shares; ++i) ss += part[s][i * p.T + t];
      rs[s] = rsqrtf(ss / static_cast<float>(p.heads[s] * HD) + p.eps);
    }
  }

  // A row u, normalised with 1 / rms r and weights w, and turned.
  auto turn = [&](uint4& u, float r, const float* w) {
    float f[8];
    unpack8(u, f);
    if (NORM != kNormNone) {
      if (NORM == kNormHead) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(f[i], f[i], ss);
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        r = rsqrtf(ss * (1.f / HD) + p.eps);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = f[i] * r * w[i];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      constexpr int STEP = HALVES ? 1 : 2, PARTNER = HALVES ? 4 : 1;
      const float x1 = f[STEP * i], x2 = f[STEP * i + PARTNER];
      const float y1 = x1 * cs[i].x - x2 * cs[i].y, y2 = x1 * cs[i].y + x2 * cs[i].x;
      if (whole || (turns && p0 + i < p.half)) f[STEP * i] = y1, f[STEP * i + PARTNER] = y2;
    }
    u = pack8(f);
  };

  const size_t step = static_cast<size_t>(p.N) * HD;  // between heads of a target
#pragma unroll
  for (int s = 0; s < 3; ++s) {
    if (p.x[s] == nullptr) continue;
    const __nv_bfloat16* src = source(s);
    __nv_bfloat16* dst = p.y[s] + (static_cast<size_t>(b) * p.heads[s] * p.N + n) * HD;
    float w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 1.f;
    const void* weights = s < 2 ? p.w[s] : nullptr;
    if (NORM == kNormHead && weights != nullptr) load_w(weights, 0, w);
    // as many passes for every group, for the exchanges inside (a group may have no head in the last)
    for (int h0 = share; h0 - share < p.heads[s]; h0 += shares * kRotRows) {
      uint4 u[kRotRows];
#pragma unroll
      for (int k = 0; k < kRotRows; ++k) {
        const int h = h0 + k * shares;
        u[k] = h < p.heads[s] ? load(src + h * p.sh[s]) : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int k = 0; k < kRotRows; ++k) {
        const int h = h0 + k * shares;
        if (NORM == kNormToken && weights != nullptr) load_w(weights, static_cast<size_t>(min(h, p.heads[s] - 1)) * HD, w);
        if (s < 2) turn(u[k], rs[s < 2 ? s : 0], w);
        if (live && h < p.heads[s]) {
          __nv_bfloat16* out = dst + h * step;
          if (HALVES) {
            *reinterpret_cast<uint2*>(out + e0) = make_uint2(u[k].x, u[k].y);
            *reinterpret_cast<uint2*>(out + e1) = make_uint2(u[k].z, u[k].w);
          } else {
            *reinterpret_cast<uint4*>(out + e0) = u[k];
          }
        }
      }
    }
  }
}

}  // namespace mcs
