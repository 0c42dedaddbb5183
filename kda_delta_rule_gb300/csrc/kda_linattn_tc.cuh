// Linear attention with one decay for each head over packed sequences, bf16, on the tensor cores.
//
//   S_t = e^(g_t) S_(t-1) + k_t v_t^T,   o_t = scale S_t^T q_t
//
// in chunks of 128 tokens; with b_i the log decays summed from a chunk's start, inclusive, and S the state before it,
//
//   O  = scale (P V + e^b Q S),  P_ij = (q_i . k_j) e^(b_i - b_j) for j <= i
//   S' = e^(b_C) S + (e^(b_C - b) K)^T V
//
// Decays.  They are summed as fixed-point numbers, exactly.  e^(b_i - b_j) is never the quotient of two exponentials, which
// could leave fp32's range: for tokens of different blocks of 32 it is e^(b_i - b_J) e^(b_J - b_j) with b_J the sum at the end of
// j's block, both factors at most 1; within a block it is the exponential of the difference.
//
// Precision.  P, and the copy of S that the chunk's outputs read, are rounded to bf16 for their products (o is rounded to bf16
// as well); the state itself is fp32 in registers, and what is added to it has to be as good: the decayed keys, which are no bf16
// numbers, go in as two (hi + lo, 16 bits of significand), one product each.
//
// One CTA per (segment of a sequence, head), chunk after chunk; roles by warp:
//   0-7   state: decayed keys of a chunk (hi over the keys in place, lo beside them); S' = e^(b_C) S + sum; S as the next chunk's
//         bf16 operand
//   8-11  scores: the decays of the next chunk; P from the scores, Q S scaled by its rows' decays in place; the outputs, through the value tile
//         to whole rows in memory
//   12    copies (TMA): q one tile, k and v two
//   13    products: Q K^T, Q S, hi and lo (V^T K), P V (P from tensor memory)
// The state's product is taken as V^T K (rows are value channels), so that a warp's threads hold 32 neighbouring
// columns of S and its reads and writes of fp32 states are whole lines, and any dk is a number of columns.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/kda.h"
#include "kda_common.cuh"
#include "kda_linattn.h"
#include "kda_mla.cuh"
#include "kda_mla_tc.cuh"
#include "kda_tc.cuh"
#include "kda_tmap.h"

namespace kda {
namespace {

using namespace tc;

constexpr int kC = kLinChunk;
constexpr uint32_t kAtom = kC * 128;              // 64 channels of a chunk's rows

template <int DK, int DV>
struct LinTc {
  static constexpr int AK = (DK + 63) / 64, AV = (DV + 63) / 64;   // atoms of a tile; heads of 32 channels come with their neighbour's
  static constexpr int MS = DV == 128 ? 128 : 64;                  // rows of the state's product
  static constexpr uint32_t Q = 0, K = Q + AK * kAtom, V = K + 2 * AK * kAtom, LO = V + 2 * AV * kAtom, SB = LO + AK * kAtom;
  static constexpr uint32_t MISC = SB + AK * DV * 128, SMEM = MISC + 2560;
  // of the first pass: keys, values and lo twice each
  static constexpr uint32_t LK = 0, LV = LK + 2 * AK * kAtom, LLO = LV + 2 * AV * kAtom, LMISC = LLO + 2 * AK * kAtom, LSMEM = LMISC + 2560;
  static_assert(SMEM <= 232448 && LSMEM <= 232448, "shared memory of a CTA");
};

// A operand in tensor memory (rows are lanes, two bf16 per column), issued by one lane of a converged warp
__device__ __forceinline__ void mma_ts_w(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{ .reg .pred p, e; .reg .b32 r; elect.sync r|e, 0xffffffff; setp.ne.b32 p, %4, 0; "
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }"
      :: "r"(d_tmem), "r"(a_tmem), "l"(b), "r"(idesc), "r"(acc) : "memory");
}
__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
      :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
         "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 x = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&x);
}
__device__ __forceinline__ uint4 pack8(const float* v) {
  return make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
}
template <int N>
__device__ __forceinline__ void bar_sync(int id) { asm volatile("barrier.cta.sync %0, %1;" :: "r"(id), "n"(N) : "memory"); }
// one arrival per warp, after what its lanes did before
__device__ __forceinline__ void arrive_w(uint32_t mbar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(mbar);
}
__device__ __forceinline__ bool wait_w(uint32_t mbar, int phase, volatile int* abort) { return wait_phase_w(mbar, (uint32_t)phase & 1u, abort); }

// inclusive sum over the warp's lanes
__device__ __forceinline__ int64_t warp_scan(int64_t x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t up = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += up;
  }
  return x;
}
// f as two bf16 numbers, the first in the low half
__device__ __forceinline__ uint32_t split2(float f) {
  const __nv_bfloat16 hi = __float2bfloat16_rn(f);
  const __nv_bfloat16 lo = __float2bfloat16_rn(f - __bfloat162float(hi));
  return (uint32_t)__bfloat16_as_ushort(hi) | ((uint32_t)__bfloat16_as_ushort(lo) << 16);
}

// The decayed keys of a tile (256 threads): k f = hi + lo with f = f1 + f2.  hi = k f1 rounded, whose error is a
// bf16 number, found by one fused multiply-add, which k f2 joins.  Rows of 8 threads, whatever their order of channels, so the swizzle does not matter.
// Rows from n on are cleared, in the value tile as well: they are another sequence's.
template <int AK, int AV>
__device__ __forceinline__ void decay_keys(unsigned char* k, unsigned char* lo, unsigned char* v, const uint32_t* f, int tid, int n) {
#pragma unroll
  for (int i = 0; i < kC / 32; ++i) {
    const int row = (tid >> 3) + 32 * i;
    const uint32_t w = f[row];
    const uint32_t w1 = __byte_perm(w, w, 0x1010), w2 = __byte_perm(w, w, 0x3232);
    const __nv_bfloat162 f1 = *reinterpret_cast<const __nv_bfloat162*>(&w1), f2 = *reinterpret_cast<const __nv_bfloat162*>(&w2);
#pragma unroll
    for (int a = 0; a < AK; ++a) {
      const uint32_t at = a * kAtom + row * 128 + (tid & 7) * 16;
      uint4 x = *reinterpret_cast<const uint4*>(k + at);
      uint32_t* xs = reinterpret_cast<uint32_t*>(&x);
      uint32_t ys[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 kk = *reinterpret_cast<const __nv_bfloat162*>(&xs[j]);
        const __nv_bfloat162 hi = __hmul2_rn(kk, f1);
        const __nv_bfloat162 l = __hfma2(kk, f2, __hfma2(kk, f1, __hneg2(hi)));
        xs[j] = *reinterpret_cast<const uint32_t*>(&hi);
        ys[j] = *reinterpret_cast<const uint32_t*>(&l);
      }
      if (row >= n) {
        x = make_uint4(0, 0, 0, 0);
        ys[0] = ys[1] = ys[2] = ys[3] = 0;
      }
      *reinterpret_cast<uint4*>(k + at) = x;
      *reinterpret_cast<uint4*>(lo + at) = make_uint4(ys[0], ys[1], ys[2], ys[3]);
    }
    if (row >= n) {
#pragma unroll
      for (int a = 0; a < AV; ++a) *reinterpret_cast<uint4*>(v + a * kAtom + row * 128 + (tid & 7) * 16) = make_uint4(0, 0, 0, 0);
    }
  }
}

// The state's product, V^T (hi + lo): rows value channels, columns key channels
template <int DK, int DV>
__device__ __forceinline__ void mma_state(uint32_t d, uint32_t v, uint32_t hi, uint32_t lo, bool add) {
  constexpr uint32_t ID = idesc_bf16(LinTc<DK, DV>::MS, DK, true, true);
  const uint64_t dv = desc_mn(v, kC, 0), dh = desc_mn(hi, kC, 0), dl = desc_mn(lo, kC, 0);
#pragma unroll
  for (int j = 0; j < kC / 16; ++j) mma_w(d, dv + (uint64_t)(128 * j), dh + (uint64_t)(128 * j), ID, add || j > 0);
#pragma unroll
  for (int j = 0; j < kC / 16; ++j) mma_w(d, dv + (uint64_t)(128 * j), dl + (uint64_t)(128 * j), ID, 1);
}

// TMEM -> registers, N consecutive columns of this warp's lanes
template <int N>
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, float* v) {
  if constexpr (N == 16) {
    float x[16];
    tmem_ld16(taddr, x);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = x[i];
  } else {
    float x[32];
    tmem_ld32(taddr, x);
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = x[i];
  }
}

template <int DK, int DV>
__global__ void __launch_bounds__(448, 1)
kda_linattn_tc_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                      const LinPrefillArgs a, const __grid_constant__ LinSched sched) {
  using L = LinTc<DK, DV>;
  constexpr int AK = L::AK, AV = L::AV;
  extern __shared__ __align__(1024) unsigned char sm[];
  unsigned char* misc = sm + L::MISC;
  const uint32_t base = smem_u32(sm), bars = smem_u32(misc);
  const uint32_t full_q = bars, full_k = bars + 8, full_v = bars + 24, qkd = bars + 40, qsd = bars + 56, kvd = bars + 64, pvd = bars + 80,
                 p_ready = bars + 88, o_free = bars + 96, s_ready = bars + 104, kbar = bars + 112, gate = bars + 120, v_free = bars + 136;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(misc + 160);
  volatile int* abort = reinterpret_cast<volatile int*>(misc + 164);
  float* s_end = reinterpret_cast<float*>(misc + 168);                  // [2]: e^(b_C)
  int64_t* s_blk = reinterpret_cast<int64_t*>(misc + 176);              // [4]: the blocks' decays
  float* s_near = reinterpret_cast<float*>(misc + 256);                 // [128]: log2 decays from the block's start
  float* s_col = reinterpret_cast<float*>(misc + 768);                  // [128]: 2^(decay to the block's end)
  uint32_t* s_f = reinterpret_cast<uint32_t*>(misc + 1280);             // [2][128]: 2^(decay to the chunk's end) as two bf16

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h = blockIdx.y, hk = h / a.share;
  if (base & 1023) {                                        // the swizzled tiles need it
    if (tid == 0) atomicOr(&g_kda_device_error, kDevErrWait);
    return;
  }
  if (tid == 0) {
    mbar_init(full_q, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(full_k + 8 * i, 1);
      mbar_init(full_v + 8 * i, 1);
      mbar_init(qkd + 8 * i, 1);
      mbar_init(kvd + 8 * i, 1);
      mbar_init(gate + 8 * i, 4);
      mbar_init(v_free + 8 * i, 4);
    }
    mbar_init(qsd, 1);
    mbar_init(pvd, 1);
    mbar_init(p_ready, 4);
    mbar_init(o_free, 4);
    mbar_init(s_ready, 8);
    mbar_init(kbar, 8);
    *abort = 0;
    mbar_init_fence();
  }
  if (warp == 13) tmem_alloc(smem_u32(tslot), 512);
  const LinItem it = lin_item(sched, blockIdx.x);
  const int nch = (it.n + kC - 1) / kC;
  mla_grid_wait();
  mla_grid_next();
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *tslot;
  const uint32_t t_o = tmem, t_kv = tmem + 256;             // scores of chunk c: tmem + 128 + 256 (c & 1)

  if (warp == 12) {
    if (lane == 0) {
      int nq = 0, nkv = 0;                                  // tiles asked for
      for (int c = 0; c < nch; ++c) {
        const int s = c & 1, y = (int)(it.t0 + (int64_t)c * kC);
        if (c >= 2 && !wait_phase(kvd + 8 * s, ((c - 2) >> 1) & 1, abort)) break;
        if (c >= 2 && !wait_phase(v_free + 8 * s, ((c - 2) >> 1) & 1, abort)) break;
        mbar_expect_tx(full_k + 8 * s, AK * kAtom);
        for (int i = 0; i < AK; ++i) tma_load_2d(base + L::K + (s * AK + i) * kAtom, &mk, hk * DK + 64 * i, y, full_k + 8 * s);
        mbar_expect_tx(full_v + 8 * s, AV * kAtom);
        for (int i = 0; i < AV; ++i) tma_load_2d(base + L::V + (s * AV + i) * kAtom, &mv, h * DV + 64 * i, y, full_v + 8 * s);
        nkv = c + 1;
        if (c >= 1 && !wait_phase(qsd, (c - 1) & 1, abort)) break;
        mbar_expect_tx(full_q, AK * kAtom);
        for (int i = 0; i < AK; ++i) tma_load_2d(base + L::Q + i * kAtom, &mq, hk * DK + 64 * i, y, full_q);
        nq = c + 1;
      }
      // no copy is left under way into this CTA's shared memory (bounded waits; a completed phase returns at once)
      if (nq) mbar_wait(full_q, (nq - 1) & 1);
      for (int c = max(0, nkv - 2); c < nkv; ++c) {
        mbar_wait(full_k + 8 * (c & 1), (c >> 1) & 1);
        mbar_wait(full_v + 8 * (c & 1), (c >> 1) & 1);
      }
    }
    __syncwarp();
  } else if (warp == 13) {
    const uint64_t dq = desc_k(base + L::Q, kC, 0), ds = desc_k(base + L::SB, DV, 0);
    constexpr uint32_t ID_QK = idesc_bf16(128, 128, false, false), ID_QS = idesc_bf16(128, DV, false, false), ID_PV = idesc_bf16(128, DV, false, true);
    const auto scores = [&](int c) {
      if (!wait_w(full_q, c, abort) || !wait_w(full_k + 8 * (c & 1), c >> 1, abort)) return false;
      fence_after();
      const uint64_t dk = desc_k(base + L::K + (c & 1) * AK * kAtom, kC, 0);
#pragma unroll
      for (int j = 0; j < DK / 16; ++j) {
        const uint64_t step = (uint64_t)((j >> 2) * (kAtom >> 4) + (j & 3) * 2);
        mma_w(tmem + 128 + 256 * (c & 1), dq + step, dk + step, ID_QK, j > 0);
      }
      mma_commit_w(qkd + 8 * (c & 1));
      return true;
    };
    bool on = nch > 0 && scores(0);
    for (int c = 0; on && c < nch; ++c) {
      const int s = c & 1;
      if (!wait_w(s_ready, c, abort) || (c > 0 && !wait_w(o_free, c - 1, abort))) break;
      fence_after();
#pragma unroll
      for (int j = 0; j < DK / 16; ++j)
        mma_w(t_o, dq + (uint64_t)((j >> 2) * (kAtom >> 4) + (j & 3) * 2), ds + (uint64_t)((j >> 2) * (DV * 8) + (j & 3) * 2), ID_QS, j > 0);
      mma_commit_w(qsd);
      if (!wait_w(kbar, c, abort) || !wait_w(full_v + 8 * s, c >> 1, abort)) break;
      fence_after();
      mma_state<DK, DV>(t_kv, base + L::V + s * AV * kAtom, base + L::K + s * AK * kAtom, base + L::LO, false);
      mma_commit_w(kvd + 8 * s);
      if (!wait_w(p_ready, c, abort)) break;
      fence_after();
      const uint64_t dv = desc_mn(base + L::V + s * AV * kAtom, kC, 0);
#pragma unroll
      for (int j = 0; j < kC / 16; ++j) mma_ts_w(t_o, tmem + 128 + 256 * s + 8 * j, dv + (uint64_t)(128 * j), ID_PV, 1);
      mma_commit_w(pvd);
      if (c + 1 < nch) on = scores(c + 1);
    }
  } else if (warp < 8) {
    // ---- state: thread = column j of S (a lane of the product), rows i0 .. i0 + NC - 1
    constexpr int NC = DK / 2, LD = NC < 32 ? NC : 32;
    const int qd = warp & 3, i0 = NC * (warp >> 2);
    const int j = L::MS == 128 ? 32 * qd + lane : 16 * qd + lane;
    const bool mine = (L::MS == 128 || lane < 16) && j < DV;
    const int64_t hstate = (int64_t)DK * DV, at = (int64_t)i0 * DV + j;
    float S[NC];
    {
      const float* src = nullptr;
      if (it.nth > 0) src = a.seg_state + ((int64_t)lin_slot(sched, it.place, it.nth - 1) * a.H + h) * hstate;
      else if (a.S0) src = a.S0 + ((int64_t)it.seq * a.H + h) * hstate;
#pragma unroll
      for (int e = 0; e < NC; ++e) S[e] = src && mine ? src[at + e * DV] : 0.f;
    }
    const auto publish = [&] {                              // S as the operand of the next chunk's outputs
      if (mine) {
#pragma unroll
        for (int e = 0; e < NC; e += 8) *reinterpret_cast<uint4*>(sm + L::SB + off_k(j, i0 + e, DV)) = pack8(S + e);
      }
      fence_async_smem();
      fence_before();
      arrive_w(s_ready, lane);
    };
    const auto store = [&](float* dst) {
      if (mine) {
#pragma unroll
        for (int e = 0; e < NC; ++e) dst[at + e * DV] = S[e];
      }
    };
    if (nch > 0) publish();
    for (int c = 0; c < nch; ++c) {
      const int s = c & 1, n = min(kC, it.n - c * kC);
      bool ok = wait_w(gate + 8 * s, c >> 1, abort) && wait_w(full_k + 8 * s, c >> 1, abort) && wait_w(qkd + 8 * s, c >> 1, abort);
      if (n < kC) ok = ok && wait_w(full_v + 8 * s, c >> 1, abort);
      fence_after();
      if (ok) decay_keys<AK, AV>(sm + L::K + s * AK * kAtom, sm + L::LO, sm + L::V + s * AV * kAtom, s_f + 128 * s, tid, n);
      fence_async_smem();
      fence_before();
      arrive_w(kbar, lane);
      ok = wait_w(kvd + 8 * s, c >> 1, abort);
      fence_after();
      const float f = s_end[s];
#pragma unroll
      for (int e = 0; e < NC; e += LD) {
        float x[LD];
        tmem_ld_cols<LD>(t_kv + ((uint32_t)(32 * qd) << 16) + i0 + e, x);
#pragma unroll
        for (int i = 0; i < LD; ++i) S[e + i] = fmaf(f, S[e + i], x[i]);
      }
      const int pos = it.nth * sched.seg_len + c * kC + n;
      if (ok && a.ckpt_stride > 0 && pos % a.ckpt_stride == 0) {
        const int64_t ck = (int64_t)sched.ckpt_base[it.place] + pos / a.ckpt_stride - 1;
        if (ck < a.num_ckpt) {
          float* page = reinterpret_cast<float*>(a.pages + (int64_t)a.ckpt_page_ids[ck] * a.page_bytes);
          store(page + h * hstate);
          if (h == 0) {
            for (int64_t e = a.H * hstate + tid; e < a.page_bytes / 4; e += 256) page[e] = 0.f;
            if (tid == 0 && a.ckpt_pos) a.ckpt_pos[ck] = pos;
          }
        }
      }
      if (c + 1 < nch) {
        wait_w(qsd, c, abort);                              // the product that reads the operand's last value
        publish();
      }
    }
    if (it.last && !*abort) store(a.S_final + ((int64_t)it.seq * a.H + h) * hstate);
  } else {
    // ---- scores: thread = row i of the chunk
    const int w = warp - 8, i = 32 * w + lane;
    const uint32_t lane_at = (uint32_t)(32 * w) << 16;
    const float* g = a.g + h;
    __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(a.o) + (int64_t)h * DV;
    float near = 0.f, far[3] = {0.f, 0.f, 0.f}, all = 0.f;   // log2 decay from the block's start; factors from the ends of earlier blocks, from the chunk's start
    float next = i < it.n ? g[(it.t0 + i) * a.g_stride] : 0.f;
    const auto decays = [&](int c) {
      const int n = min(kC, it.n - c * kC);
      bool bad = false;
      const int64_t sum = warp_scan(lin_fixed(i < n ? next : 0.f, &bad), lane);
      if (bad) atomicOr(&g_kda_device_error, kDevErrGate);
      const int64_t t = (int64_t)(c + 1) * kC + i;
      next = t < it.n ? g[(it.t0 + t) * a.g_stride] : 0.f;
      if (lane == 31) s_blk[w] = sum;
      near = lin_float(sum);
      bar_sync<128>(1);
      int64_t before = 0, total = 0;
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        if (b < w) before += s_blk[b];
        total += s_blk[b];
      }
      int64_t since = before;
#pragma unroll
      for (int b = 0; b < 3; ++b) {
        since -= s_blk[b];
        far[b] = a.scale * exp2f(lin_float(since + sum));   // used for b < w
      }
      all = a.scale * exp2f(lin_float(before + sum));
      s_near[i] = near;
      s_col[i] = exp2f(lin_float(s_blk[w] - sum));
      s_f[128 * (c & 1) + i] = i < n ? split2(exp2f(lin_float(total - before - sum))) : 0u;
      if (tid == 256) s_end[c & 1] = exp2f(lin_float(total));
      arrive_w(gate + 8 * (c & 1), lane);
    };
    if (nch > 0) decays(0);
    for (int c = 0; c < nch; ++c) {
      const int s = c & 1, n = min(kC, it.n - c * kC);
      const uint32_t t_p = tmem + 128 + 256 * s + lane_at;
      wait_w(gate + 8 * s, c >> 1, abort);
      bool ok = wait_w(qkd + 8 * s, c >> 1, abort);
      fence_after();
#pragma unroll
      for (int b = 0; b < 4; ++b) {                         // columns 32 b .. of P, over the scores already read
        uint32_t p[16];
        if (b <= w) {
          float x[32];
          tmem_ld32(t_p + 32 * b, x);
          if (b < w) {
            const float f = b == 0 ? far[0] : b == 1 ? far[1] : far[2];
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
              const float4 cf = *reinterpret_cast<const float4*>(s_col + 32 * b + j);
              p[j / 2] = pack2(x[j] * (f * cf.x), x[j + 1] * (f * cf.y));
              p[j / 2 + 1] = pack2(x[j + 2] * (f * cf.z), x[j + 3] * (f * cf.w));
            }
          } else {
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
              const float4 lj = *reinterpret_cast<const float4*>(s_near + 32 * b + j);
              const float y0 = j <= lane ? x[j] * (a.scale * ex2(near - lj.x)) : 0.f, y1 = j + 1 <= lane ? x[j + 1] * (a.scale * ex2(near - lj.y)) : 0.f;
              const float y2 = j + 2 <= lane ? x[j + 2] * (a.scale * ex2(near - lj.z)) : 0.f, y3 = j + 3 <= lane ? x[j + 3] * (a.scale * ex2(near - lj.w)) : 0.f;
              p[j / 2] = pack2(y0, y1);
              p[j / 2 + 1] = pack2(y2, y3);
            }
          }
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j) p[j] = 0;
        }
        tmem_st16u(t_p + 16 * b, p);
      }
      ok = wait_w(qsd, c, abort) && ok;
      fence_after();
#pragma unroll
      for (int e = 0; e < DV; e += 32) {                    // e^b Q S
        float x[32];
        uint32_t y[16];
        tmem_ld32(t_o + lane_at + e, x);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
#pragma unroll
          for (int j = 0; j < 16; ++j) y[j] = __float_as_uint(all * x[16 * half + j]);
          tmem_st16u(t_o + lane_at + e + 16 * half, y);
        }
      }
      tmem_st_wait();
      fence_before();
      arrive_w(p_ready, lane);
      if (c + 1 < nch) decays(c + 1);
      ok = wait_w(pvd, c, abort) && ok;
      ok = wait_w(kvd + 8 * s, c >> 1, abort) && ok;        // the value tile's last reader: the rows go through it
      fence_after();
      unsigned char* tile = sm + L::V + s * AV * kAtom;
      const auto place = [](int row, int ch) { return row * (DV * 2) + ((ch ^ (DV >= 64 ? row & 7 : (row >> 1) & 3)) << 4); };
#pragma unroll
      for (int e = 0; e < DV; e += 32) {
        float x[32];
        tmem_ld32(t_o + lane_at + e, x);
        if (e + 32 == DV) {
          fence_before();
          arrive_w(o_free, lane);
        }
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) *reinterpret_cast<uint4*>(tile + place(i, e / 8 + ch)) = pack8(x + 8 * ch);
      }
      __syncwarp();
      const int64_t row0 = it.t0 + (int64_t)c * kC;
#pragma unroll
      for (int e = 0; e < DV / 8; ++e) {
        const int at = lane + 32 * e, r = 32 * w + at / (DV / 8), ch = at % (DV / 8);
        const uint4 y = *reinterpret_cast<const uint4*>(tile + place(r, ch));
        if (ok && r < n) *reinterpret_cast<uint4*>(o + (row0 + r) * ((int64_t)a.H * DV) + 8 * ch) = y;
      }
      fence_async_smem();
      arrive_w(v_free + 8 * s, lane);
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == 13) tmem_dealloc(tmem, 512);
}

// First pass: a segment's state from zero, (e^(B - b) K)^T V with B the segment's whole decay.  The chunks go backwards, so that the decay
// from a chunk's end to the segment's end is known, and one accumulator in tensor memory takes them all.
// Warps 0-7 decay the keys, 8 copies, 9 issues the products.
template <int DK, int DV>
__global__ void __launch_bounds__(320, 1)
kda_linattn_tc_local_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv, const LinPrefillArgs a,
                            const __grid_constant__ LinSched sched) {
  using L = LinTc<DK, DV>;
  constexpr int AK = L::AK, AV = L::AV;
  extern __shared__ __align__(1024) unsigned char sm[];
  unsigned char* misc = sm + L::LMISC;
  const uint32_t base = smem_u32(sm), bars = smem_u32(misc);
  const uint32_t full_k = bars, full_v = bars + 16, kvd = bars + 32, kbar = bars + 48;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(misc + 160);
  volatile int* abort = reinterpret_cast<volatile int*>(misc + 164);
  int64_t* s_blk = reinterpret_cast<int64_t*>(misc + 176);
  uint32_t* s_f = reinterpret_cast<uint32_t*>(misc + 1280);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h = blockIdx.y, hk = h / a.share;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(full_k + 8 * i, 1);
      mbar_init(full_v + 8 * i, 1);
      mbar_init(kvd + 8 * i, 1);
    }
    mbar_init(kbar, 8);
    *abort = 0;
    mbar_init_fence();
  }
  if (warp == 9) tmem_alloc(smem_u32(tslot), 128);
  int lo = 0, hi = sched.n_seqs - 1;                        // slot -> segment: every sequence's last one has none
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (sched.item_base[mid] - mid <= (int)blockIdx.x) lo = mid; else hi = mid - 1;
  }
  const LinItem it = lin_item(sched, blockIdx.x + lo);
  const int nch = it.n / kC;                                // whole chunks: only last segments end elsewhere
  mla_grid_wait();
  mla_grid_next();
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *tslot;
  if (warp == 8) {
    if (lane == 0) {
      int asked = 0;
      for (int c = 0; c < nch; ++c) {
        const int s = c & 1, y = (int)(it.t0 + (int64_t)(nch - 1 - c) * kC);
        if (c >= 2 && !wait_phase(kvd + 8 * s, ((c - 2) >> 1) & 1, abort)) break;
        mbar_expect_tx(full_k + 8 * s, AK * kAtom);
        for (int i = 0; i < AK; ++i) tma_load_2d(base + L::LK + (s * AK + i) * kAtom, &mk, hk * DK + 64 * i, y, full_k + 8 * s);
        mbar_expect_tx(full_v + 8 * s, AV * kAtom);
        for (int i = 0; i < AV; ++i) tma_load_2d(base + L::LV + (s * AV + i) * kAtom, &mv, h * DV + 64 * i, y, full_v + 8 * s);
        asked = c + 1;
      }
      for (int c = max(0, asked - 2); c < asked; ++c) {
        mbar_wait(full_k + 8 * (c & 1), (c >> 1) & 1);
        mbar_wait(full_v + 8 * (c & 1), (c >> 1) & 1);
      }
    }
    __syncwarp();
  } else if (warp == 9) {
    for (int c = 0; c < nch; ++c) {
      const int s = c & 1;
      if (!wait_w(kbar, c, abort) || !wait_w(full_v + 8 * s, c >> 1, abort)) break;
      fence_after();
      mma_state<DK, DV>(tmem, base + L::LV + s * AV * kAtom, base + L::LK + s * AK * kAtom, base + L::LLO + s * AK * kAtom, c > 0);
      mma_commit_w(kvd + 8 * s);
    }
  } else {
    const float* g = a.g + h;
    int64_t behind = 0;                                     // decay of the chunks behind this one
    float next = tid < kC ? g[(it.t0 + (int64_t)(nch - 1) * kC + tid) * a.g_stride] : 0.f;
    bool ok = true;
    for (int c = 0; c < nch; ++c) {
      const int s = c & 1;
      int64_t sum = 0;
      if (tid < kC) {
        bool bad = false;
        sum = warp_scan(lin_fixed(next, &bad), lane);
        if (bad) atomicOr(&g_kda_device_error, kDevErrGate);
        if (c + 1 < nch) next = g[(it.t0 + (int64_t)(nch - 2 - c) * kC + tid) * a.g_stride];
        if (lane == 31) s_blk[4 * s + warp] = sum;
      }
      bar_sync<256>(1);
      int64_t to_end = behind;                              // from the end of this thread's block of 32
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int64_t x = s_blk[4 * s + b];
        if (b >= warp) to_end += x;
        if (behind > kLinLeast) behind += x;
      }
      if (tid < kC) s_f[128 * s + tid] = split2(exp2f(lin_float(to_end - sum)));
      bar_sync<256>(1);
      ok = wait_w(full_k + 8 * s, c >> 1, abort) && ok;     // the copy has waited for the products of chunk c - 2, which read lo, too
      if (ok) decay_keys<AK, AV>(sm + L::LK + s * AK * kAtom, sm + L::LLO + s * AK * kAtom, sm + L::LV + s * AV * kAtom, s_f + 128 * s, tid, kC);
      fence_async_smem();
      fence_before();
      arrive_w(kbar, lane);
    }
    const int last = nch - 1;
    ok = wait_w(kvd + 8 * (last & 1), last >> 1, abort) && ok;
    fence_after();
    constexpr int NC = DK / 2, LD = NC < 32 ? NC : 32;
    const int qd = warp & 3, i0 = NC * (warp >> 2);
    const int j = L::MS == 128 ? 32 * qd + lane : 16 * qd + lane;
    const bool mine = ok && (L::MS == 128 || lane < 16) && j < DV;
    const int64_t at = (int64_t)blockIdx.x * a.H + h;
    float* dst = a.seg_state + at * ((int64_t)DK * DV) + (int64_t)i0 * DV + j;
#pragma unroll
    for (int e = 0; e < NC; e += LD) {
      float x[LD];
      tmem_ld_cols<LD>(tmem + ((uint32_t)(32 * qd) << 16) + i0 + e, x);
      if (mine) {
#pragma unroll
        for (int i = 0; i < LD; ++i) dst[(e + i) * DV] = x[i];
      }
    }
    if (tid == 0) a.seg_decay[at] = behind;
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == 9) tmem_dealloc(tmem, 128);
}

template <int DK, int DV>
cudaError_t run_tc(const LinPrefillArgs& a, const LinSched& sched, cudaStream_t s) {
  using L = LinTc<DK, DV>;
  static std::atomic<uint64_t> allowed{0}, allowed_local{0};
  CUtensorMap mq, mk, mv;
  const int64_t H_k = a.H / a.share;
  if (!make_map_rows(&mq, a.q, a.T, H_k * DK, a.q_stride, 64, kC) || !make_map_rows(&mk, a.k, a.T, H_k * DK, a.k_stride, 64, kC) ||
      !make_map_rows(&mv, a.v, a.T, (int64_t)a.H * DV, a.v_stride, 64, kC))
    return cudaErrorInvalidValue;
  const auto kern = kda_linattn_tc_kernel<DK, DV>;
  if (const cudaError_t e = mla_allow_smem(kern, L::SMEM, allowed)) return e;
  const int local = sched.n_items - sched.n_seqs;
  if (local > 0) {
    const auto first = kda_linattn_tc_local_kernel<DK, DV>;
    if (const cudaError_t e = mla_allow_smem(first, L::LSMEM, allowed_local)) return e;
    if (const cudaError_t e = mla_launch(first, dim3((unsigned)local, (unsigned)a.H), 320, L::LSMEM, s, mk, mv, a, sched)) return e;
    if (const cudaError_t e = launch_linattn_scan(a, sched, s)) return e;
  }
  return mla_launch(kern, dim3((unsigned)sched.n_items, (unsigned)a.H), 448, L::SMEM, s, mq, mk, mv, a, sched);
}

int read_and_clear_errors_here(int* flags) {
  int word = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&word, g_kda_device_error, sizeof(int));
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_kda_device_error, &zero, sizeof(int));
  *flags |= word;
  return (int)e;
}

}  // namespace
}  // namespace kda
