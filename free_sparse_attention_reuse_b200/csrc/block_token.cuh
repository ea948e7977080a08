// Attention over listed key blocks for few query rows (one token, one token of several heads, up to 16 rows
// of a list): the keys and values are read once from memory and little else happens.  A list's runs of 16 or
// 32 keys, which lie one behind the other in memory, are shared out over four warps; each warp keeps a
// ring of runs in flight with bulk copies (its loads straight into registers reached 3.1 TB/s: too few
// bytes under way for the registers they took) and multiplies with mma.sync (16 rows, of which as
// many count as there are):
//
//   S = Q K^T   contraction over d in an order of our choosing: a lane's 16 consecutive bytes of a key row
//               are its B fragments of two (bf16) or four (e4m3) k steps, Q's fragments follow suit;
//   O = P V     the columns in an order of our choosing: a lane's 16 bytes of four value rows, two rows
//               interleaved, are its B fragments of eight (16) column tiles.
//
// Running maximum and sum per row, in fp32 and base 2; a CTA's four warps are merged through shared memory,
// the CTAs of a split list by block_join_kernel.  Bound: device memory.
#pragma once

#include "block_attn.cuh"

namespace mcs {

constexpr int kTokenWarps = 4;

// C += A B for 16 rows (F16: fp16 operands, else bf16), and for at most 8: the upper half of A is zero
// and that of the result is dropped.
template <bool F16>
__device__ __forceinline__ void mma_16816(float& c0, float& c1, float& c2, float& c3, uint32_t a0, uint32_t a1,
                                          uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c0), "+f"(c1), "+f"(c2), "+f"(c3)
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c0), "+f"(c1), "+f"(c2), "+f"(c3)
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <bool F16>
__device__ __forceinline__ void mma_8816(float& c0, float& c1, uint32_t a0, uint32_t a2, uint32_t b0, uint32_t b1) {
  [[maybe_unused]] float x, y;
  if constexpr (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%5}, {%7,%8}, {%0,%1,%9,%9};"
        : "+f"(c0), "+f"(c1), "=f"(x), "=f"(y)
        : "r"(a0), "r"(0u), "r"(a2), "r"(b0), "r"(b1), "f"(0.f));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%5}, {%7,%8}, {%0,%1,%9,%9};"
        : "+f"(c0), "+f"(c1), "=f"(x), "=f"(y)
        : "r"(a0), "r"(0u), "r"(a2), "r"(b0), "r"(b1), "f"(0.f));
}
// D = A B for fp16.
__device__ __forceinline__ void mma_16816_zero(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                               uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// A row of Q as fp16 fragments: times the power of two that brings its largest element into [2^14, 2^15); returned
// is the one that takes it back.  Exact for elements down to 2^-28 of the largest, off by at most 2^-39 of
// it below (half of fp16's 2^-24 steps).  The exponent is kept where both powers are normal numbers: a row whose
// largest element is below 2^-107 is brought up by 2^121, and its elements are off by at most 2^-146.  (A row with
// infinities or NaN gives NaN either way.)
template <int N>
__device__ __forceinline__ float q_to_f16(uint32_t* q) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&q[i]));
    top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
  }
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
  const int e = min(max(static_cast<int>(__float_as_uint(top) >> 23), 20), 254) - 127;
  const float up = __uint_as_float(static_cast<uint32_t>(14 - e + 127) << 23);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&q[i]));
    q[i] = pack_f16x2(f.x * up, f.y * up);
  }
  return __uint_as_float(static_cast<uint32_t>(e - 14 + 127) << 23);
}

template <int HD, bool KV8>
struct TokenSmem {
  static constexpr int KC = KV8 || HD == 64 ? 32 : 16;             // keys of a run
  static constexpr uint32_t ROW = HD * (KV8 ? 1 : 2);              // bytes of a row
  static constexpr uint32_t RUN = KC * ROW;                        // of a run's keys, or values
  static constexpr int RING = 16384 / (2 * RUN);                   // runs that a warp has in hand: 2 or 4
  static constexpr uint32_t WARP = RING * 2 * RUN;                 // 16 KB
  static constexpr uint32_t BYTES = kTokenWarps * WARP;            // the warps' results lie over it at the end
  static_assert(kTokenWarps * 16 * HD * 4 <= BYTES, "results fit");
};

template <int HD, bool KV8, int RT>
__global__ void __launch_bounds__(kTokenWarps * 32, RT == 8 ? 3 : 2) block_token_kernel(const BlockAttnParams p) {
  using L = TokenSmem<HD, KV8>;
  constexpr int KC = L::KC, RING = L::RING;
  constexpr int NT = KC / 8;                     // key tiles
  constexpr int LB = HD * (KV8 ? 1 : 2) / 64;    // 16-byte loads of a lane per key row (4 lanes a row)
  constexpr int KS = KV8 ? 4 : 2;                // k steps that such a load feeds
  constexpr int VC = KV8 ? HD / 8 : 8;           // columns that a lane loads of a value row at once
  constexpr int VH = HD / (8 * VC);              // such loads per value row
  constexpr int WIDE = RT == 16;
  constexpr uint32_t VB = VC * (KV8 ? 1 : 2);    // their bytes: 16, or 8
  extern __shared__ __align__(128) uint8_t ring_mem[];
  __shared__ float sm_m[kTokenWarps][RT], sm_l[kTokenWarps][RT];
  __shared__ __align__(8) uint64_t sm_full[kTokenWarps][RING];
  __shared__ int sm_valid[kTokenWarps][RING];
  __shared__ float sm_scale[kTokenWarps][RING][2];
  __shared__ int s_end, s_abort;
  constexpr bool QS = RT == 8 && HD == 128;  // Q's fragments in shared memory: three CTAs an SM instead of two
  __shared__ __align__(16) uint4 sm_q[QS ? LB * KS / 2 : 1][32];
  float (*sm_o)[RT][HD] = reinterpret_cast<float (*)[RT][HD]>(ring_mem);

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

  if (threadIdx.x == 0) s_abort = 0;
  if (lane < RING) mbar_init(&sm_full[warp][lane], KV8 ? 3 : 1);
  fence_mbar_init();
  __syncthreads();

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

  // 8-bit rows are widened to fp16 (one instruction for two values; bf16 takes four), so Q is fp16 as well,
  // and P.  fp16 ends at 2^-24 and is rounded coarser from 2^-14 down, while a key of little weight may have
  // the largest value: P, at most 1, is multiplied by 2^15, so that it is off by at most 2^-11 of itself down to
  // 2^-29 of the row's largest and by 2^-40 of that below.  The V scale is applied to a run's products in
  // fp32, and takes the 2^15 back.
  constexpr float kPUp = 32768.f;
  float qs0 = 1.f, qs1 = 1.f;
  if constexpr (KV8) {
    qs0 = q_to_f16<LB * KS * 2>(qa);
    if constexpr (WIDE) qs1 = q_to_f16<LB * KS * 2>(qb);
  }

  if constexpr (QS) {
    if (warp == 0)
#pragma unroll
      for (int i = 0; i < LB * KS / 2; ++i) sm_q[i][lane] = make_uint4(qa[4 * i], qa[4 * i + 1], qa[4 * i + 2], qa[4 * i + 3]);
    __syncthreads();
  }
  const uint32_t qbase = smem_u32(&sm_q[0][lane]);

  const uint8_t* Kb = static_cast<const uint8_t*>(p.K) + static_cast<size_t>(bkv) * p.Nk * L::ROW;
  const uint8_t* Vb = static_cast<const uint8_t*>(p.V) + static_cast<size_t>(bkv) * p.Nk * L::ROW;
  const uint32_t ring = smem_u32(ring_mem) + warp * L::WARP;
  uint64_t* full = sm_full[warp];
  volatile int* abort_flag = &s_abort;
  uint32_t issued = 0;
  // the run that advance() found into the ring's next slot, which this warp has read before
  auto issue = [&]() {
    const uint32_t slot = issued % RING, dst = ring + slot * 2 * L::RUN;
    ++issued;
    // masked keys weigh 0, but 0 times what lies in their value rows need not be 0; a later run's copy into these
    // rows must not pass the stores by
    if (valid < KC) {
      for (int k = valid; k < KC; ++k)
        for (uint32_t e = lane * 16; e < L::ROW; e += 512)
          asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(dst + L::RUN + k * L::ROW + e), "r"(0u) : "memory");
      fence_proxy_async_smem();
    }
    if (KV8 && lane < 2) {
      const float* src = (lane == 0 ? p.ks : p.vs) + static_cast<size_t>(bkv) * p.nb + blk;
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(&sm_scale[warp][slot][lane])), "l"(src) : "memory");
      cp_async_arrive(full + slot);
    }
    if (lane == 0) {
      sm_valid[warp][slot] = valid;
      const uint32_t bytes = valid * L::ROW;
      const size_t at = static_cast<size_t>(key0) * L::ROW;
      mbar_arrive_expect_tx(full + slot, 2 * bytes);
      bulk_load(dst, Kb + at, bytes, full + slot);
      bulk_load(dst + L::RUN, Vb + at, bytes, full + slot);
    }
    __syncwarp();
  };

  constexpr int OT = HD / 8;  // column tiles
  float o[OT][2], o2[WIDE ? OT : 1][2];
#pragma unroll
  for (int i = 0; i < OT; ++i) o[i][0] = o[i][1] = 0.f;
  if constexpr (WIDE)
#pragma unroll
    for (int i = 0; i < OT; ++i) o2[i][0] = o2[i][1] = 0.f;
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;

  bool more = true;
#pragma unroll 1
  for (int i = 0; i < RING - 1 && more; ++i) {
    more = advance();
    if (more) issue();
  }
#pragma unroll 1
  for (uint32_t done = 0; done < issued; ++done) {
    if (more) more = advance();
    if (more) issue();  // into the slot of the run before this one
    const uint32_t slot = done % RING;
    if (!mbar_wait_warp(full + slot, (done / RING) & 1, abort_flag, p.wait_ns)) {
      for (; done < issued; ++done) mbar_drain(full + done % RING, (done / RING) & 1);  // copies under way land
      break;
    }
    const uint32_t kbase = ring + slot * 2 * L::RUN, vbase = kbase + L::RUN;
    const int nvalid = sm_valid[warp][slot];
    const float ks = KV8 ? sm_scale[warp][slot][0] : 1.f, vscale = KV8 ? sm_scale[warp][slot][1] * (1.f / kPUp) : 1.f;
    const float ks0 = p.scale_log2 * ks * qs0, ks1 = p.scale_log2 * ks * qs1;
    float s[NT][2], s2[WIDE ? NT : 1][2];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      s[i][0] = s[i][1] = 0.f;
      if constexpr (WIDE) s2[i][0] = s2[i][1] = 0.f;
    }
    // key tiles innermost: their chains of products overlap
#pragma unroll
    for (int j = 0; j < LB; ++j) {
      uint4 kr[NT];
#pragma unroll
      for (int i = 0; i < NT; ++i) kr[i] = lds16(kbase + (i * 8 + g) * L::ROW + j * 64 + t * 16);
      uint32_t qf[2 * KS];  // Q's fragments of this load's k steps
#pragma unroll
      for (int k = 0; k < KS / 2; ++k) {
        const int q = j * KS * 2 + 4 * k;
        if constexpr (QS) {
          const uint4 u = lds16(qbase + (q / 4) * 512);
          qf[4 * k] = u.x, qf[4 * k + 1] = u.y, qf[4 * k + 2] = u.z, qf[4 * k + 3] = u.w;
        } else {
          qf[4 * k] = qa[q], qf[4 * k + 1] = qa[q + 1], qf[4 * k + 2] = qa[q + 2], qf[4 * k + 3] = qa[q + 3];
        }
      }
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const int q = (j * KS + k) * 2;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          const uint32_t in[4] = {kr[i].x, kr[i].y, kr[i].z, kr[i].w};
          uint32_t b0, b1;
          if constexpr (KV8) e4m3x4_to_f16(in[k], b0, b1);
          else b0 = in[2 * k], b1 = in[2 * k + 1];
          if constexpr (WIDE) mma_16816<KV8>(s[i][0], s[i][1], s2[i][0], s2[i][1], qf[2 * k], qb[q], qf[2 * k + 1], qb[q + 1], b0, b1);
          else mma_8816<KV8>(s[i][0], s[i][1], qf[2 * k], qf[2 * k + 1], b0, b1);
        }
      }
    }
    // softmax of the run: the row's running maximum, shared by its four lanes
    auto soften = [&](float (*x)[2], float kscale, float& m, float& l) -> float {
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
    const float al0 = soften(s, ks0, m0, l0);
    float al1 = 1.f;
    if constexpr (WIDE) al1 = soften(s2, ks1, m1, l1);
    uint32_t pa[NT / 2][4];
#pragma unroll
    for (int k = 0; k < NT / 2; ++k) {
      auto frag = [&](const float* x) { return KV8 ? pack_f16x2(x[0] * kPUp, x[1] * kPUp) : pack_bf16x2(x[0], x[1]); };
      pa[k][0] = frag(s[2 * k]), pa[k][2] = frag(s[2 * k + 1]);
      pa[k][1] = pa[k][3] = 0;
      if constexpr (WIDE) pa[k][1] = frag(s2[2 * k]), pa[k][3] = frag(s2[2 * k + 1]);
    }
    if (!KV8 && __any_sync(0xffffffffu, al0 != 1.f || al1 != 1.f)) {
#pragma unroll
      for (int i = 0; i < OT; ++i) o[i][0] *= al0, o[i][1] *= al0;
      if constexpr (WIDE)
#pragma unroll
        for (int i = 0; i < OT; ++i) o2[i][0] *= al1, o2[i][1] *= al1;
    }
    // O += P V, 16 keys at a time; 8-bit: O = alpha O + V scale (P V)
#pragma unroll
    for (int h = 0; h < VH; ++h) {
      // value rows 16 k + 2 t + {0, 1, 8, 9}: what the lane's P fragments of 16 keys multiply; 8-bit rows eight
      // columns at a time
      auto row_at = [&](int i) {
        const int k = (i >> 2) * 16 + 2 * t + (i & 1) + (i & 2) * 4;
        return vbase + k * L::ROW + h * 8 * VB + g * VB;
      };
      if constexpr (KV8) {
#pragma unroll
        for (int j8 = 0; j8 < VC; j8 += 8) {
          uint32_t vr[NT * 2][2];
#pragma unroll
          for (int i = 0; i < NT * 2; ++i)
            asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(vr[i][0]), "=r"(vr[i][1]) : "r"(row_at(i) + j8));
#pragma unroll
          for (int j = 0; j < 8; j += 2) {
            const int i = h * VC + j8 + j;
            float c[2][4];
            // bytes j and j + 1 of two rows side by side, then widened: tiles j and j + 1
            constexpr uint32_t kSel[2] = {0x5140u, 0x7362u};
            const uint32_t sel = kSel[(j & 2) >> 1];
#pragma unroll
            for (int k = 0; k < NT / 2; ++k) {
              uint32_t b00, b01, b10, b11;
              e4m3x4_to_f16(__byte_perm(vr[4 * k][j / 4], vr[4 * k + 1][j / 4], sel), b00, b10);
              e4m3x4_to_f16(__byte_perm(vr[4 * k + 2][j / 4], vr[4 * k + 3][j / 4], sel), b01, b11);
              if (k == 0) {
                mma_16816_zero(c[0], pa[k][0], pa[k][1], pa[k][2], pa[k][3], b00, b01);
                mma_16816_zero(c[1], pa[k][0], pa[k][1], pa[k][2], pa[k][3], b10, b11);
              } else if constexpr (WIDE) {
                mma_16816<true>(c[0][0], c[0][1], c[0][2], c[0][3], pa[k][0], pa[k][1], pa[k][2], pa[k][3], b00, b01);
                mma_16816<true>(c[1][0], c[1][1], c[1][2], c[1][3], pa[k][0], pa[k][1], pa[k][2], pa[k][3], b10, b11);
              } else {
                mma_8816<true>(c[0][0], c[0][1], pa[k][0], pa[k][2], b00, b01);
                mma_8816<true>(c[1][0], c[1][1], pa[k][0], pa[k][2], b10, b11);
              }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              o[i + e][0] = fmaf(c[e][0], vscale, o[i + e][0] * al0), o[i + e][1] = fmaf(c[e][1], vscale, o[i + e][1] * al0);
              if constexpr (WIDE)
                o2[i + e][0] = fmaf(c[e][2], vscale, o2[i + e][0] * al1), o2[i + e][1] = fmaf(c[e][3], vscale, o2[i + e][1] * al1);
            }
          }
        }
      } else {
        uint32_t vr[NT * 2][4];
#pragma unroll
        for (int i = 0; i < NT * 2; ++i) {
          const uint4 u = lds16(row_at(i));
          vr[i][0] = u.x, vr[i][1] = u.y, vr[i][2] = u.z, vr[i][3] = u.w;
        }
#pragma unroll
        for (int j = 0; j < VC; ++j) {
          const int i = h * VC + j;
          const uint32_t sel = (j & 1) ? 0x7632u : 0x5410u;
#pragma unroll
          for (int k = 0; k < NT / 2; ++k) {
            const uint32_t b0 = __byte_perm(vr[4 * k][j / 2], vr[4 * k + 1][j / 2], sel);
            const uint32_t b1 = __byte_perm(vr[4 * k + 2][j / 2], vr[4 * k + 3][j / 2], sel);
            if constexpr (WIDE) mma_16816<false>(o[i][0], o[i][1], o2[i][0], o2[i][1], pa[k][0], pa[k][1], pa[k][2], pa[k][3], b0, b1);
            else mma_8816<false>(o[i][0], o[i][1], pa[k][0], pa[k][2], b0, b1);
          }
        }
      }
    }
    __syncwarp();  // every lane has read the slot
  }
  __syncthreads();  // the results lie over the rings

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
