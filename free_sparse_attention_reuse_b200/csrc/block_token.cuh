// Attention over listed key blocks for few query rows (one token, one token of several heads, up to 16 rows
// of a list): the keys and values are read once from memory and little else happens, so nothing is
// staged in shared memory.  Every warp streams runs of keys straight into the registers of mma.sync
// fragments (16 rows, of which as many count as there are):
//
//   S = Q K^T   contraction over d in an order of our choosing: a lane's 16 consecutive bytes of a key row
//               are its B fragments of two (bf16) or four (e4m3) k steps, Q's fragments follow suit;
//   O = P V     the columns in an order of our choosing: a lane's 16 bytes of four value rows, two rows
//               interleaved, are its B fragments of eight (16) column tiles.
//
// A lane loads 16 bytes at a time and a warp's load covers whole 32-byte sectors; a run's values are
// loaded while its logits are formed, the next run's keys while the softmax runs.  Running maximum and
// sum per row, in fp32 and base 2; a CTA's four warps are merged through shared memory, the CTAs of a
// split list by block_join_kernel.  Bound: device memory.
#pragma once

#include "block_attn.cuh"

namespace mcs {

constexpr int kTokenWarps = 4;

__device__ __forceinline__ void mma_16816(float& c0, float& c1, float& c2, float& c3, uint32_t a0, uint32_t a1,
                                          uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c0), "+f"(c1), "+f"(c2), "+f"(c3)
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same for at most 8 rows: the upper half of A is zero and that of the result is dropped.
__device__ __forceinline__ void mma_8816(float& c0, float& c1, uint32_t a0, uint32_t a2, uint32_t b0, uint32_t b1) {
  [[maybe_unused]] float x, y;
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%5}, {%7,%8}, {%0,%1,%9,%9};"
      : "+f"(c0), "+f"(c1), "=f"(x), "=f"(y)
      : "r"(a0), "r"(0u), "r"(a2), "r"(b0), "r"(b1), "f"(0.f));
}
// Two e4m3 values (low 16 bits) to bf16, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_bf16(uint32_t x) {
  const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(x & 0xffffu), __NV_E4M3)));
  return pack_bf16x2(f.x, f.y);
}

template <int HD, bool KV8, int RT>
__global__ void __launch_bounds__(kTokenWarps * 32, RT == 8 && HD == 64 ? 3 : 2) block_token_kernel(const BlockAttnParams p) {
  constexpr int KC = KV8 || HD == 64 ? 32 : 16;  // keys of a run
  constexpr int NT = KC / 8;                     // key tiles
  constexpr int LB = HD * (KV8 ? 1 : 2) / 64;    // 16-byte loads of a lane per key row (4 lanes a row)
  constexpr int KS = KV8 ? 4 : 2;                // k steps that such a load feeds
  constexpr int VC = KV8 ? HD / 8 : 8;           // columns that a lane loads of a value row at once
  constexpr int VH = HD / (8 * VC);              // such loads per value row
  constexpr int WIDE = RT == 16;
  using Val = typename std::conditional<VC * (KV8 ? 1 : 2) == 16, uint4, uint2>::type;
  __shared__ float sm_m[kTokenWarps][RT], sm_l[kTokenWarps][RT];
  __shared__ __align__(16) float sm_o[kTokenWarps][RT][HD];
  __shared__ int s_end;

  let_dependents_start();
  const int warp = warp_id(), lane = lane_id(), g = lane >> 2, t = lane & 3;
  const int unit = blockIdx.x;
  const int sp = unit % p.splits, tu = unit / p.splits;
  const int bh = tu / p.GQ, gq = tu - bh * p.GQ;
  const int b = bh / p.H, bkv = b * p.Hkv + (bh - b * p.H) / (p.H / p.Hkv);
  const int rows = min(p.C, p.Nq - gq * p.C);
  const size_t row0 = static_cast<size_t>(bh) * p.Nq + static_cast<size_t>(gq) * p.C;
  const int len = valid_rows(p.len, b, p.Nk);
  const int32_t* list = p.blocks != nullptr ? p.blocks + (static_cast<size_t>(bh) * p.GQ + gq) * p.kb : nullptr;

  // entries of the list: up to its first negative one
  int n = list != nullptr ? p.kb : min(p.nb, (len + p.BK - 1) / p.BK);
  if (list != nullptr) {
    if (threadIdx.x == 0) s_end = p.kb;
    __syncthreads();
    int first = p.kb;
    for (int i = threadIdx.x; i < p.kb; i += kTokenWarps * 32) {
      const int id = list[i];
      if (id < 0) {
        first = i;
        break;
      }
    }
    first = __reduce_min_sync(0xffffffffu, first);
    if (lane == 0 && first < p.kb) atomicMin(&s_end, first);
    __syncthreads();
    n = s_end;
  }
  const int rpb = p.BK / KC;  // runs of a block
  const int c_end = static_cast<int>(static_cast<long long>(n) * (sp + 1) / p.splits) * rpb;
  int c = static_cast<int>(static_cast<long long>(n) * sp / p.splits) * rpb + warp - kTokenWarps;
  int key0 = 0, valid = 0, blk = 0;
  // this warp's next run that holds a valid key
  auto advance = [&]() -> bool {
    for (c += kTokenWarps; c < c_end; c += kTokenWarps) {
      const int e = c / rpb;
      blk = list != nullptr ? list[e] : e;
      if (blk >= p.nb) {
        raise_status(kStatusBadIndex);
        continue;
      }
      key0 = blk * p.BK + (c - e * rpb) * KC;
      valid = min(KC, len - key0);
      if (valid > 0) return true;
    }
    return false;
  };

  // Q fragments: row g (and g + 8), the d order of the key loads
  uint32_t qa[LB * KS * 2], qb[WIDE ? LB * KS * 2 : 1];
#pragma unroll
  for (int i = 0; i < LB * KS / 2; ++i) {
    const int d = KV8 ? (i >> 1) * 64 + t * 16 + (i & 1) * 8 : i * 32 + t * 8;
    uint4 u = make_uint4(0u, 0u, 0u, 0u);
    if (g < rows) u = *reinterpret_cast<const uint4*>(p.Q + (row0 + g) * HD + d);
    qa[4 * i] = u.x, qa[4 * i + 1] = u.y, qa[4 * i + 2] = u.z, qa[4 * i + 3] = u.w;
    if constexpr (WIDE) {
      u = make_uint4(0u, 0u, 0u, 0u);
      if (g + 8 < rows) u = *reinterpret_cast<const uint4*>(p.Q + (row0 + g + 8) * HD + d);
      qb[4 * i] = u.x, qb[4 * i + 1] = u.y, qb[4 * i + 2] = u.z, qb[4 * i + 3] = u.w;
    }
  }

  constexpr int ESZ = KV8 ? 1 : 2;
  const uint8_t* Kb = static_cast<const uint8_t*>(p.K) + static_cast<size_t>(bkv) * p.Nk * HD * ESZ;
  const uint8_t* Vb = static_cast<const uint8_t*>(p.V) + static_cast<size_t>(bkv) * p.Nk * HD * ESZ;
  uint4 kr[NT][LB];
  Val vr[NT * 2][VH];
  float ks = 1.f, vs = 1.f;
  auto load_k = [&]() {
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int k = i * 8 + g;
#pragma unroll
      for (int j = 0; j < LB; ++j)
        kr[i][j] = k < valid ? *reinterpret_cast<const uint4*>(Kb + (static_cast<size_t>(key0 + k) * HD * ESZ + j * 64 + t * 16))
                             : make_uint4(0u, 0u, 0u, 0u);
    }
    if (KV8) {
      ks = p.ks[static_cast<size_t>(bkv) * p.nb + blk];
      vs = p.vs[static_cast<size_t>(bkv) * p.nb + blk];
    }
  };
  // value rows 16 i + 2 t + {0, 1, 8, 9}: what the lane's P fragments of 16 keys multiply
  auto load_v = [&]() {
#pragma unroll
    for (int i = 0; i < NT * 2; ++i) {
      const int k = (i >> 2) * 16 + 2 * t + (i & 1) + (i & 2) * 4;
#pragma unroll
      for (int h = 0; h < VH; ++h) {
        vr[i][h] = Val{};
        if (k < valid)
          vr[i][h] = *reinterpret_cast<const Val*>(Vb + (static_cast<size_t>(key0 + k) * HD + h * 64 + g * VC) * ESZ);
      }
    }
  };

  constexpr int OT = HD / 8;  // column tiles
  float o[OT][2], o2[WIDE ? OT : 1][2];
#pragma unroll
  for (int i = 0; i < OT; ++i) o[i][0] = o[i][1] = 0.f;
  if constexpr (WIDE)
#pragma unroll
    for (int i = 0; i < OT; ++i) o2[i][0] = o2[i][1] = 0.f;
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;

  bool more = advance();
  if (more) load_k();
  while (more) {
    load_v();
    float s[NT][2], s2[WIDE ? NT : 1][2];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      s[i][0] = s[i][1] = 0.f;
      if constexpr (WIDE) s2[i][0] = s2[i][1] = 0.f;
#pragma unroll
      for (int j = 0; j < LB; ++j) {
        uint32_t w[2 * KS];
        if constexpr (KV8) {
          e4m3_to_bf16(kr[i][j], w);
        } else {
          w[0] = kr[i][j].x, w[1] = kr[i][j].y, w[2] = kr[i][j].z, w[3] = kr[i][j].w;
        }
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          const int q = (j * KS + k) * 2;
          if constexpr (WIDE) mma_16816(s[i][0], s[i][1], s2[i][0], s2[i][1], qa[q], qb[q], qa[q + 1], qb[q + 1], w[2 * k], w[2 * k + 1]);
          else mma_8816(s[i][0], s[i][1], qa[q], qa[q + 1], w[2 * k], w[2 * k + 1]);
        }
      }
    }
    const int nvalid = valid;
    const float kscale = p.scale_log2 * ks, vscale = vs;
    more = advance();
    if (more) load_k();
    // softmax of the run: the row's running maximum, shared by its four lanes
    auto soften = [&](float (*x)[2], float& m, float& l) -> float {
      float mx = -INFINITY;
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          x[i][e] = i * 8 + 2 * t + e < nvalid ? x[i][e] * kscale : -INFINITY;
          mx = fmaxf(mx, x[i][e]);
        }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      mx = fmaxf(mx, m);
      const float ref = mx == -INFINITY ? 0.f : mx;  // a row without a key of weight yet
      const float alpha = fast_exp2(m - ref);
      m = mx;
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          x[i][e] = fast_exp2(x[i][e] - ref);
          sum += x[i][e];
        }
      l = fmaf(l, alpha, sum);
      return alpha;
    };
    const float al0 = soften(s, m0, l0);
    float al1 = 1.f;
    if constexpr (WIDE) al1 = soften(s2, m1, l1);
    if (__any_sync(0xffffffffu, al0 != 1.f || al1 != 1.f)) {
#pragma unroll
      for (int i = 0; i < OT; ++i) o[i][0] *= al0, o[i][1] *= al0;
      if constexpr (WIDE)
#pragma unroll
        for (int i = 0; i < OT; ++i) o2[i][0] *= al1, o2[i][1] *= al1;
    }
    // O += (P * V scale) V, 16 keys at a time
#pragma unroll
    for (int k = 0; k < NT / 2; ++k) {
      auto frag = [&](const float (*x)[2], int i) {
        return KV8 ? pack_bf16x2(x[i][0] * vscale, x[i][1] * vscale) : pack_bf16x2(x[i][0], x[i][1]);
      };
      const uint32_t a0 = frag(s, 2 * k), a2 = frag(s, 2 * k + 1);
      uint32_t a1 = 0, a3 = 0;
      if constexpr (WIDE) a1 = frag(s2, 2 * k), a3 = frag(s2, 2 * k + 1);
#pragma unroll
      for (int h = 0; h < VH; ++h) {
        const uint32_t* va = reinterpret_cast<const uint32_t*>(&vr[4 * k][h]);
        const uint32_t* vb = reinterpret_cast<const uint32_t*>(&vr[4 * k + 1][h]);
        const uint32_t* vc = reinterpret_cast<const uint32_t*>(&vr[4 * k + 2][h]);
        const uint32_t* vd = reinterpret_cast<const uint32_t*>(&vr[4 * k + 3][h]);
#pragma unroll
        for (int j = 0; j < VC; ++j) {
          uint32_t b0, b1;
          if constexpr (KV8) {  // bytes j of both rows side by side, then widened
            const uint32_t sel = (j & 3) | ((4 + (j & 3)) << 4);
            b0 = e4m3x2_to_bf16(__byte_perm(va[j / 4], vb[j / 4], sel));
            b1 = e4m3x2_to_bf16(__byte_perm(vc[j / 4], vd[j / 4], sel));
          } else {
            const uint32_t sel = (j & 1) ? 0x7632u : 0x5410u;
            b0 = __byte_perm(va[j / 2], vb[j / 2], sel);
            b1 = __byte_perm(vc[j / 2], vd[j / 2], sel);
          }
          const int i = h * VC + j;
          if constexpr (WIDE) mma_16816(o[i][0], o[i][1], o2[i][0], o2[i][1], a0, a1, a2, a3, b0, b1);
          else mma_8816(o[i][0], o[i][1], a0, a2, b0, b1);
        }
      }
    }
  }

  // merge the warps: column of tile h * VC + j, place n: 64 h + n * VC + j
  auto spill = [&](const float (*x)[2], float m, float l, int row) {
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    if (t == 0) sm_m[warp][row] = m, sm_l[warp][row] = l;
#pragma unroll
    for (int h = 0; h < VH; ++h)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int j = 0; j < VC; j += 4)
          *reinterpret_cast<float4*>(&sm_o[warp][row][64 * h + (2 * t + e) * VC + j]) =
              make_float4(x[h * VC + j][e], x[h * VC + j + 1][e], x[h * VC + j + 2][e], x[h * VC + j + 3][e]);
  };
  spill(o, m0, l0, g);
  if constexpr (WIDE) spill(o2, m1, l1, g + 8);
  __syncthreads();
  constexpr int Q4 = HD / 4;
  for (int i = threadIdx.x; i < rows * Q4; i += kTokenWarps * 32) {
    const int r = i / Q4, cc = (i - r * Q4) * 4;
    float m = -INFINITY;
#pragma unroll
    for (int w = 0; w < kTokenWarps; ++w) m = fmaxf(m, sm_m[w][r]);
    const float mz = m == -INFINITY ? 0.f : m;
    float l = 0.f, v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kTokenWarps; ++w) {
      const float a = fast_exp2(sm_m[w][r] - mz);
      const float4 x = *reinterpret_cast<const float4*>(&sm_o[w][r][cc]);
      l = fmaf(a, sm_l[w][r], l);
      v[0] = fmaf(a, x.x, v[0]);
      v[1] = fmaf(a, x.y, v[1]);
      v[2] = fmaf(a, x.z, v[2]);
      v[3] = fmaf(a, x.w, v[3]);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const float l2 = l == 0.f ? -INFINITY : mz + log2f(l);
    const size_t row = row0 + r;
    if (p.splits > 1) {
      const size_t prow = static_cast<size_t>(sp) * p.B * p.H * p.Nq + row;
      *reinterpret_cast<float4*>(p.part + prow * HD + cc) = make_float4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
      if (cc == 0) p.plse[prow] = l2;
      continue;
    }
    float add[4] = {0.f, 0.f, 0.f, 0.f};
    if (p.R != nullptr) {
      const uint2 u = *reinterpret_cast<const uint2*>(p.R + row * HD + cc);
      const float2 x = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.x));
      const float2 y = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.y));
      add[0] = x.x, add[1] = x.y, add[2] = y.x, add[3] = y.y;
    }
    uint2 u;
    u.x = pack_bf16x2(fmaf(v[0], inv, add[0]), fmaf(v[1], inv, add[1]));
    u.y = pack_bf16x2(fmaf(v[2], inv, add[2]), fmaf(v[3], inv, add[3]));
    *reinterpret_cast<uint2*>(p.out + row * HD + cc) = u;
    if (p.lse != nullptr && cc == 0) p.lse[row] = l2 * 0.69314718055994531f;
  }
}

}  // namespace mcs
