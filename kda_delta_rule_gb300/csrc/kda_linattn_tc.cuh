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
// as well); the state itself is fp32, and what is added to it has to be as good: the decayed keys, which are no bf16
// numbers, go in as the sum of three (hi + lo + least, 24 bits of significand), one product each.
//
// One CTA per (segment of a sequence, head), chunk after chunk; roles by warp:
//   0-7   state (in tensor memory): S' = e^(b_C) S + sum, the factor as two numbers; S as the next chunk's bf16 operand; checkpoints
//   8-15  scores, two warps for 32 rows: P from the scores, Q S scaled by its rows' decays in place
//   16-23 decayed keys, 32 tokens at a time: hi over the keys in place, lo and least beside them (two slots)
//   24-27 outputs, through the value tile to memory
//   28    copies (TMA): q one tile, k and v two; the decays, a chunk ahead
//   29    products Q K^T, Q S, P V (P from tensor memory)
//   30    products (least + lo + hi)^T V (two warps issue: 48 products a chunk take one some 7000 clocks)
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
  static constexpr int OC = DV < 64 ? DV : 64;                     // columns of an output tile's part that one copy takes
  static constexpr uint32_t Q = 0, K = Q + AK * kAtom, V = K + 2 * AK * kAtom, LO = V + 2 * AV * kAtom, SB = LO + AK * kAtom;
  static constexpr uint32_t SLOT = AK * 4096;                      // lo or least of 32 tokens: two pairs of them
  static constexpr uint32_t MISC = SB + AK * DV * 128, SMEM = MISC + 2592;
  // of the first pass, in steps of 64 tokens: stages of keys and values
  static constexpr int LS = 6;
  static constexpr uint32_t HK = AK * kAtom / 2, HV = AV * kAtom / 2, STAGE = HK + HV, LMISC = LS * STAGE, LSMEM = LMISC + 256 + LS * 256;
  static_assert(SMEM <= 232448 && LSMEM <= 232448, "shared memory of a CTA");
};

// low word of a descriptor whose atoms of 64 rows or columns are `stride` bytes apart (MN-major)
__device__ __forceinline__ uint32_t lo_mn(uint32_t base, uint32_t stride) { return (base >> 4) | ((stride >> 4) << 16); }
// A operand in tensor memory (rows are lanes, two bf16 per column), issued by the lane for which `el` is not zero
__device__ __forceinline__ void mma_ts_e(uint32_t el, uint32_t d_tmem, uint32_t a_tmem, uint32_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{ .reg .pred p, e; .reg .b64 db; setp.ne.b32 e, %5, 0; setp.ne.b32 p, %4, 0; mov.b64 db, {%2, %6}; "
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p; }"
      :: "r"(d_tmem), "r"(a_tmem), "r"(b), "r"(idesc), "r"(acc), "r"(el), "r"(kDescHi) : "memory");
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float (&v)[8]) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\t"
               "tcgen05.wait::ld.sync.aligned;"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]) : "r"(taddr) : "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
      :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
         "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, int x, int y, uint32_t src) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" :: "l"(map), "r"(x), "r"(y), "r"(src) : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const float (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
               :: "r"(taddr), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]) : "memory");
}
__device__ __forceinline__ void tmem_st8u(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
               :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]) : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 x = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&x);
}
__device__ __forceinline__ uint4 pack8(const float* v) {
  return make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
}
// a value's leading 16 bits
__device__ __forceinline__ float lead(float x) { return __uint_as_float(__float_as_uint(x) & 0xffff0000u); }
// the registers of a warp's role; all warps of a group of four call one of these, with the same number
template <int N> __device__ __forceinline__ void regs_less() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(N)); }
template <int N> __device__ __forceinline__ void regs_more() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(N)); }
// one arrival per warp, after what its lanes did before
__device__ __forceinline__ void arrive_w(uint32_t mbar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(mbar);
}
// A warp waits for a phase.  It sleeps in the barrier for up to a millisecond at a time; a wait that has not ended after about a
// second, or that meets another role's giving up, returns false and tells the other roles.
__device__ __forceinline__ bool wait_w(uint32_t mbar, int phase, volatile int* abort) {
  const auto sleep = [&] {
    uint32_t done;
    asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3; selp.u32 %0, 1, 0, p; }"
                 : "=r"(done) : "r"(mbar), "r"((uint32_t)phase & 1u), "r"(1000000u) : "memory");
    return __all_sync(0xffffffffu, done != 0);
  };
  if (sleep()) return true;
  const long long t0 = clock64();
#pragma unroll 1
  while (!sleep()) {
    const bool late = clock64() - t0 > (1LL << 31);
    if (__any_sync(0xffffffffu, late || *abort)) {
      if (late) atomicOr(&g_kda_device_error, kDevErrWait);
      *abort = 1;
      return false;
    }
  }
  return true;
}

// inclusive sum over the warp's lanes
__device__ __forceinline__ int64_t warp_scan(int64_t x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t up = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += up;
  }
  return x;
}
// Two decayed keys: x = k f in fp32, whose leading 16 bits are a bf16 number (hi), of what they leave, which is exact, again
// (lo), and the rest rounded (least).  (bf16 arithmetic with products split by fused multiply-adds takes 12 instructions at half rate,
// this 13: 235 against 186 clocks for 8 warps' pieces.)
__device__ __forceinline__ void split_two(float2 k, float2 f, uint32_t& hi, uint32_t& lo, uint32_t& least) {
  const float2 p = __fmul2_rn(k, f);
  hi = __byte_perm(__float_as_uint(p.x), __float_as_uint(p.y), 0x7632);
  const float2 y = __fadd2_rn(p, make_float2(-lead(p.x), -lead(p.y)));
  lo = __byte_perm(__float_as_uint(y.x), __float_as_uint(y.y), 0x7632);
  const float2 z = __fadd2_rn(y, make_float2(-lead(y.x), -lead(y.y)));
  least = pack2(z.x, z.y);
}
// of eight channels of a token
__device__ __forceinline__ void split_keys(const uint4& k, float f, uint4& hi, uint4& lo, uint4& least) {
  const uint32_t w[4] = {k.x, k.y, k.z, k.w};
  uint32_t h[4], l[4], r[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    split_two(make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u)), make_float2(f, f), h[j], l[j], r[j]);
  hi = make_uint4(h[0], h[1], h[2], h[3]);
  lo = make_uint4(l[0], l[1], l[2], l[3]);
  least = make_uint4(r[0], r[1], r[2], r[3]);
}

// The state's product over 32 tokens, V^T (least + lo + hi): rows value channels, columns key channels; operands as low words of
// their descriptors.  The tensor core drops what does not fit the accumulator's 24 bits at every step
// of 16 tokens, so the small parts come first, and few of the steps lose bits of the whole (over 2048 tokens on one
// accumulator, in any order, the state was off by 4e-6).
template <int DK, int DV>
__device__ __forceinline__ void mma_state(uint32_t el, uint32_t d, uint32_t v, uint32_t hi, uint32_t lo, uint32_t least, bool add) {
  constexpr uint32_t ID = idesc_bf16(LinTc<DK, DV>::MS, DK, true, true);
#pragma unroll
  for (int j = 0; j < 2; ++j) mma_e(el, d, v + 128 * j, least + 128 * j, ID, add || j > 0);
#pragma unroll
  for (int j = 0; j < 2; ++j) mma_e(el, d, v + 128 * j, lo + 128 * j, ID, 1);
#pragma unroll
  for (int j = 0; j < 2; ++j) mma_e(el, d, v + 128 * j, hi + 128 * j, ID, 1);
}

// Four neighbouring tokens' log decays per lane of one warp, summed from each block of 32 tokens' start (near) and, exactly, from the
// chunk's start to the blocks' starts (before) and its end (all).
struct ChunkDecays {
  int64_t sum[4], before, block, all;                       // block: the whole of this lane's block
};
__device__ __forceinline__ ChunkDecays chunk_decays(const float (&g)[4], int lane) {
  bool bad = false;
  ChunkDecays d;
#pragma unroll
  for (int i = 0; i < 4; ++i) d.sum[i] = lin_fixed(g[i], &bad) + (i ? d.sum[i - 1] : 0);
  if (bad) atomicOr(&g_kda_device_error, kDevErrGate);
  int64_t x = d.sum[3];
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {                         // over the 8 lanes of a block
    const int64_t up = __shfl_up_sync(0xffffffffu, x, o, 8);
    if ((lane & 7) >= o) x += up;
  }
  const int64_t first = x - d.sum[3];
#pragma unroll
  for (int i = 0; i < 4; ++i) d.sum[i] += first;
  d.before = d.all = 0;
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const int64_t t = __shfl_sync(0xffffffffu, x, 8 * b + 7);
    if (b < (lane >> 3)) d.before += t;
    if (b == (lane >> 3)) d.block = t;
    d.all += t;
  }
  return d;
}

template <int DK, int DV>
__global__ void __launch_bounds__(1024, 1)
kda_linattn_tc_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                      const __grid_constant__ CUtensorMap mo, const LinPrefillArgs a, const __grid_constant__ LinSched sched) {
  using L = LinTc<DK, DV>;
  constexpr int AK = L::AK, AV = L::AV, OC = L::OC;
  extern __shared__ __align__(1024) unsigned char sm[];
  unsigned char* misc = sm + L::MISC;
  const uint32_t base = smem_u32(sm), bars = smem_u32(misc);
  const uint32_t full_q = bars, full_k = bars + 8, full_v = bars + 24, qkd = bars + 40, qsd = bars + 56, kvd = bars + 64, pvd = bars + 80,
                 p_ready = bars + 88, o_free = bars + 96, s_ready = bars + 104, kv_read = bars + 112, gate = bars + 120, v_free = bars + 136,
                 keys = bars + 152, slot_free = bars + 168, cleared = bars + 184;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(misc + 192);
  volatile int* abort = reinterpret_cast<volatile int*>(misc + 196);
  float* s_end = reinterpret_cast<float*>(misc + 200);                  // [2]: log2 decay of the chunk
  float* s_gap = reinterpret_cast<float*>(misc + 256);                  // [2][4][4]: log2 decay from block y's end to block x's start; [x][3]: from the chunk's start
  float* s_near = reinterpret_cast<float*>(misc + 512);                 // [2][128]: log2 decays from the block's start
  float* s_col = reinterpret_cast<float*>(misc + 1536);                 // [2][128]: 2^(decay to the block's end)
  float* s_tail = reinterpret_cast<float*>(misc + 2560);                // [2][4]: 2^(decay from the block's end to the chunk's end)

  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;   // warp: known to be the same for its lanes
  const int item = blockIdx.x / (unsigned)a.H, h = blockIdx.x - item * a.H, hk = h / a.share;   // the heads of a row together
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
      mbar_init(gate + 8 * i, 1);
      mbar_init(v_free + 8 * i, 4);
      mbar_init(keys + 8 * i, 8);
      mbar_init(slot_free + 8 * i, 1);
    }
    mbar_init(qsd, 1);
    mbar_init(pvd, 1);
    mbar_init(p_ready, 8);
    mbar_init(o_free, 4);
    mbar_init(s_ready, 8);
    mbar_init(kv_read, 8);
    mbar_init(cleared, 8);
    *abort = 0;
    mbar_init_fence();
  }
  if (warp == 29) tmem_alloc(smem_u32(tslot), 512);
  const LinItem it = lin_item(sched, item);
  const int nch = (it.n + kC - 1) / kC;
  mla_grid_wait();
  mla_grid_next();
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *tslot;
  const uint32_t t_o = tmem, t_qk = tmem + 128, t_kv = tmem + 256, t_s = tmem + 384;

  // Registers by role, of the 64 a thread that the block starts with (32 warps): 8 x 48 + 8 x 96 + 8 x 64 + 8 x 48 = 32 x 64.
  if (warp == 28) {
    regs_less<48>();
    // ---- copies, by lane 0; decays, four tokens per lane
    const float* g = a.g + h;
    const auto fetch = [&](int c, float (&x)[4]) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = c * kC + 4 * lane + i;
        x[i] = t < it.n ? g[(it.t0 + t) * a.g_stride] : 0.f;
      }
    };
    const auto load_v = [&](int c) {
      const int s = c & 1;
      if (lane == 0) {
        mbar_expect_tx(full_v + 8 * s, AV * kAtom);
        for (int i = 0; i < AV; ++i)
          tma_load_2d(base + L::V + (s * AV + i) * kAtom, &mv, h * DV + 64 * i, (int)(it.t0 + (int64_t)c * kC), full_v + 8 * s);
      }
    };
    float x[4], next[4];
    int nq = 0, nk = 0, nv = 0;                             // tiles asked for
    if (nch > 0) fetch(0, x);
    for (int c = 0; c < nch; ++c) {
      const int s = c & 1, y = (int)(it.t0 + (int64_t)c * kC);
      if (c + 1 < nch) fetch(c + 1, next);
      const ChunkDecays d = chunk_decays(x, lane);
      float near[4], col[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        near[i] = lin_float(d.sum[i]);
        col[i] = exp2f(lin_float(d.block - d.sum[i]));
      }
      // the gaps: from the end of block y to the start of block x > y, and the start of the chunk
      float gap[4];
      int64_t since = d.before;
#pragma unroll
      for (int b = 0; b < 3; ++b) {
        since -= __shfl_sync(0xffffffffu, d.block, 8 * b);
        gap[b] = lin_float(since);
      }
      gap[3] = lin_float(d.before);
      const float tail = exp2f(lin_float(d.all - d.before - d.block)), end = lin_float(d.all);
      if (c >= 2 && !wait_w(kvd + 8 * s, (c - 2) >> 1, abort)) break;
      if (lane == 0) {
        mbar_expect_tx(full_k + 8 * s, AK * kAtom);
        for (int i = 0; i < AK; ++i) tma_load_2d(base + L::K + (s * AK + i) * kAtom, &mk, hk * DK + 64 * i, y, full_k + 8 * s);
      }
      nk = c + 1;
      if (c >= 1 && !wait_w(qsd, c - 1, abort)) break;
      if (lane == 0) {
        mbar_expect_tx(full_q, AK * kAtom);
        for (int i = 0; i < AK; ++i) tma_load_2d(base + L::Q + i * kAtom, &mq, hk * DK + 64 * i, y, full_q);
      }
      nq = c + 1;
      // the value tile comes free last: the outputs of chunk c - 2 leave through it, and are read when P of chunk c - 1 is done
      if (c >= 2 && !wait_w(v_free + 8 * s, (c - 2) >> 1, abort)) break;
      load_v(c);
      nv = c + 1;
      // the same places' readers of chunk c - 2 are done: its keys and P (its value tile was waited for), its state (Q S of c - 1 was)
      *reinterpret_cast<float4*>(s_near + 128 * s + 4 * lane) = make_float4(near[0], near[1], near[2], near[3]);
      *reinterpret_cast<float4*>(s_col + 128 * s + 4 * lane) = make_float4(col[0], col[1], col[2], col[3]);
      if ((lane & 7) == 0) *reinterpret_cast<float4*>(s_gap + 16 * s + 4 * (lane >> 3)) = make_float4(gap[0], gap[1], gap[2], gap[3]);
      if ((lane & 7) == 0) s_tail[4 * s + (lane >> 3)] = tail;
      if (lane == 0) s_end[s] = end;
      arrive_w(gate + 8 * s, lane);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = next[i];
    }
    // no copy is left under way into this CTA's shared memory (bounded waits; a completed phase returns at once)
    if (nq) mbar_wait(full_q, (nq - 1) & 1);
    for (int c = max(0, nk - 2); c < nk; ++c) mbar_wait(full_k + 8 * (c & 1), (c >> 1) & 1);
    for (int c = max(0, nv - 2); c < nv; ++c) mbar_wait(full_v + 8 * (c & 1), (c >> 1) & 1);
    __syncwarp();
  } else if (warp == 29) {
    regs_less<48>();
    // ---- products of the outputs
    const uint32_t el = elect_one();
    const uint32_t dq = desc_lo_k(base + L::Q), ds = desc_lo_k(base + L::SB), dk = desc_lo_k(base + L::K), dv = lo_mn(base + L::V, kAtom);
    constexpr uint32_t ID_QK = idesc_bf16(128, 128, false, false), ID_QS = idesc_bf16(128, DV, false, false), ID_PV = idesc_bf16(128, DV, false, true);
    constexpr uint32_t KS = AK * (kAtom >> 4), VS = AV * (kAtom >> 4);   // a stage in descriptor units
    const auto scores = [&](int c) {                        // over P of the chunk before, which P V has read
      if (!wait_w(full_k + 8 * (c & 1), c >> 1, abort) || !wait_w(full_q, c, abort)) return false;
      fence_after();
      const uint32_t k = dk + (c & 1) * KS;
#pragma unroll
      for (int j = 0; j < DK / 16; ++j) {
        const uint32_t step = (j >> 2) * (kAtom >> 4) + (j & 3) * 2;
        mma_e(el, t_qk, dq + step, k + step, ID_QK, j > 0);
      }
      commit_e(el, qkd + 8 * (c & 1));
      return true;
    };
    bool on = nch > 0 && scores(0);
    for (int c = 0; on && c < nch; ++c) {
      if ((c > 0 && !wait_w(o_free, c - 1, abort)) || !wait_w(s_ready, c, abort)) break;
      fence_after();
#pragma unroll
      for (int j = 0; j < DK / 16; ++j)
        mma_e(el, t_o, dq + (j >> 2) * (kAtom >> 4) + (j & 3) * 2, ds + (j >> 2) * (DV * 8) + (j & 3) * 2, ID_QS, j > 0);
      commit_e(el, qsd);
      // rows past the sequence's end are cleared in the value tile before the chunk's first keys
      if (c + 1 == nch && !wait_w(cleared, 0, abort)) break;
      if (!wait_w(full_v + 8 * (c & 1), c >> 1, abort) || !wait_w(p_ready, c, abort)) break;
      fence_after();
      const uint32_t v = dv + (c & 1) * VS;
#pragma unroll
      for (int j = 0; j < kC / 16; ++j) mma_ts_e(el, t_o, t_qk + 8 * j, v + 128 * j, ID_PV, 1);
      commit_e(el, pvd);
      if (c + 1 < nch) on = scores(c + 1);
    }
    __syncwarp();
  } else if (warp == 30) {
    regs_less<48>();
    // ---- products of the state, a quarter of a chunk at a time
    const uint32_t el = elect_one();
    const uint32_t dv = lo_mn(base + L::V, kAtom), dhi = lo_mn(base + L::K, kAtom), dlo = lo_mn(base + L::LO, 4096);
    bool on = true;
    for (int c = 0; on && c < nch; ++c) {
      const int s = c & 1;
      if ((c > 0 && !wait_w(kv_read, c - 1, abort)) || !wait_w(full_v + 8 * s, c >> 1, abort)) break;
      const uint32_t v = dv + s * (AV * (kAtom >> 4)), hi = dhi + s * (AK * (kAtom >> 4));
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        on = on && wait_w(keys + 8 * (u & 1), 2 * c + (u >> 1), abort);
        if (!on) break;
        fence_after();
        const uint32_t lo = dlo + (u & 1) * (L::SLOT >> 3);
        mma_state<DK, DV>(el, t_kv, v + 256 * u, hi + 256 * u, lo, lo + (L::SLOT >> 4), u > 0);
        commit_e(el, slot_free + 8 * (u & 1));
      }
      if (on) commit_e(el, kvd + 8 * s);
    }
    __syncwarp();
  } else if (warp == 31) {
    regs_less<48>();
  } else if (warp >= 24) {
    regs_less<48>();
    // ---- outputs: thread = row
    const int w = warp & 3;
    for (int c = 0; c < nch; ++c) {
      const int s = c & 1, n = min(kC, it.n - c * kC);
      bool ok = wait_w(pvd, c, abort);
      ok = wait_w(kvd + 8 * s, c >> 1, abort) && ok;        // the value tile's last reader: the rows go through it
      fence_after();
      unsigned char* tile = sm + L::V + s * AV * kAtom + 32 * w * (OC * 2);   // parts of OC columns, 32 rows of each, swizzled as the store's map says
      const auto place = [](int row, int ch) { return row * (OC * 2) + ((ch ^ (OC == 64 ? row & 7 : (row >> 1) & 3)) << 4); };
#pragma unroll
      for (int e = 0; e < DV; e += 16) {
        float x[16];
        tmem_ld16(t_o + ((uint32_t)(32 * w) << 16) + e, x);
#pragma unroll
        for (int ch = 0; ch < 2; ++ch)
          *reinterpret_cast<uint4*>(tile + e / OC * kAtom + place(lane, e % OC / 8 + ch)) = pack8(x + 8 * ch);
      }
      fence_before();
      arrive_w(o_free, lane);
      fence_async_smem();
      __syncwarp();
      const int64_t row0 = it.t0 + (int64_t)c * kC + 32 * w;
      if (ok && 32 * w + 32 <= n) {
        if (lane == 0) {
#pragma unroll
          for (int e = 0; e < DV; e += OC) tma_store_2d(&mo, h * DV + e, (int)row0, smem_u32(tile + e / OC * kAtom));
          bulk_commit();
          bulk_wait_read_all();
        }
      } else if (ok) {                                      // the sequence ends inside: what follows is another one's
        __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(a.o) + row0 * ((int64_t)a.H * DV) + h * DV;
        for (int e = lane; e < 32 * (DV / 8); e += 32) {
          const int r = e / (DV / 8), col = e % (DV / 8) * 8;
          if (32 * w + r < n)
            *reinterpret_cast<uint4*>(o + r * ((int64_t)a.H * DV) + col) = *reinterpret_cast<const uint4*>(tile + col / OC * kAtom + place(r, col % OC / 8));
        }
      }
      arrive_w(v_free + 8 * s, lane);
    }
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  } else if (warp >= 16) {
    // ---- decayed keys
    const int t = tid - 512;
    const uint32_t at0 = (t >> 3) * 128 + (t & 7) * 16;
    for (int c = 0; c < nch; ++c) {
      const int s = c & 1, n = min(kC, it.n - c * kC);
      unsigned char* k = sm + L::K + s * AK * kAtom + at0;
      bool ok = wait_w(gate + 8 * s, c >> 1, abort) && wait_w(full_k + 8 * s, c >> 1, abort) && wait_w(qkd + 8 * s, c >> 1, abort);
      if (n < kC) {                                         // what follows the sequence's end is another one's
        ok = ok && wait_w(full_v + 8 * s, c >> 1, abort);
        for (int e = t; e < AV * kC * 8; e += 256)
          if (ok && ((e >> 3) & (kC - 1)) >= n) *reinterpret_cast<uint4*>(sm + L::V + s * AV * kAtom + e * 16) = make_uint4(0, 0, 0, 0);
        fence_async_smem();
      }
      if (c + 1 == nch) arrive_w(cleared, lane);
      // a quarter's loads are under way while the one before is worked on
      uint4 x[AK];
      float f;
      const auto load = [&](int u) {
        f = s_tail[4 * s + u] * s_col[128 * s + 32 * u + (t >> 3)];
#pragma unroll
        for (int e = 0; e < AK; ++e) x[e] = *reinterpret_cast<const uint4*>(k + e * kAtom + u * 4096);
      };
      load(0);
#pragma unroll 1
      for (int u = 0; u < 4; ++u) {
        const int i = 4 * c + u;
        unsigned char* lo = sm + L::LO + (i & 1) * 2 * L::SLOT + at0;
        uint4 hi[AK], l[AK], r[AK];
        if (32 * u + (t >> 3) >= n) {                       // +-0 for them, whatever they hold
#pragma unroll
          for (int e = 0; e < AK; ++e) x[e] = make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int e = 0; e < AK; ++e) split_keys(x[e], f, hi[e], l[e], r[e]);
        if (u < 3) load(u + 1);
#pragma unroll
        for (int e = 0; e < AK; ++e) *reinterpret_cast<uint4*>(k + e * kAtom + u * 4096) = hi[e];
        if (i >= 2) ok = wait_w(slot_free + 8 * (i & 1), (i - 2) >> 1, abort) && ok;
#pragma unroll
        for (int e = 0; e < AK; ++e) {
          *reinterpret_cast<uint4*>(lo + e * 4096) = l[e];
          *reinterpret_cast<uint4*>(lo + L::SLOT + e * 4096) = r[e];
        }
        fence_async_smem();
        arrive_w(keys + 8 * (i & 1), lane);
      }
    }
  } else if (warp < 8) {
    regs_less<48>();
    // ---- state: thread = column j of S (a lane of the product), rows i0 .. i0 + NC - 1, eight at a time
    constexpr int NC = DK / 2;
    const int qd = warp & 3, i0 = NC * (warp >> 2);
    const int j = L::MS == 128 ? 32 * qd + lane : 16 * qd + lane;
    const bool mine = (L::MS == 128 || lane < 16) && j < DV;
    const int64_t hstate = (int64_t)DK * DV, at = (int64_t)i0 * DV + j;
    const uint32_t here = ((uint32_t)(32 * qd) << 16) + i0;
    const auto put = [&](int e, const float (&x)[8]) {      // into the operand of the next chunk's outputs
      if (mine) *reinterpret_cast<uint4*>(sm + L::SB + off_k(j, i0 + e, DV)) = pack8(x);
    };
    const auto store = [&](float* dst) {
#pragma unroll 2
      for (int e = 0; e < NC; e += 8) {
        float x[8];
        tmem_ld8(t_s + here + e, x);
        if (mine) {
#pragma unroll
          for (int i = 0; i < 8; ++i) dst[at + (e + i) * DV] = x[i];
        }
      }
    };
    {
      const float* src = nullptr;
      if (it.nth > 0) src = a.seg_state + ((int64_t)lin_slot(sched, it.place, it.nth - 1) * a.H + h) * hstate;
      else if (a.S0) src = a.S0 + ((int64_t)it.seq * a.H + h) * hstate;
#pragma unroll 4
      for (int e = 0; e < NC; e += 8) {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = src && mine ? src[at + (e + i) * DV] : 0.f;
        tmem_st8(t_s + here + e, x);
        put(e, x);
      }
      tmem_st_wait();
      fence_async_smem();
      arrive_w(s_ready, lane);
    }
    for (int c = 0; c < nch; ++c) {
      const int s = c & 1;
      wait_w(gate + 8 * s, c >> 1, abort);
      const float2 f = lin_factor_near(s_end[s]);
      wait_w(qsd, c, abort);                                // the product that reads the operand's last value
      wait_w(kvd + 8 * s, c >> 1, abort);
      fence_after();
#pragma unroll 2
      for (int e = 0; e < NC; e += 8) {
        float x[8], y[8];
        tmem_ld8(t_s + here + e, x);
        tmem_ld8(t_kv + here + e, y);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = fmaf(f.x, x[i], fmaf(f.y, x[i], y[i]));
        tmem_st8(t_s + here + e, x);
        put(e, x);
      }
      tmem_st_wait();
      fence_before();
      arrive_w(kv_read, lane);
      fence_async_smem();
      arrive_w(s_ready, lane);
      const int pos = it.nth * sched.seg_len + min(it.n, (c + 1) * kC);
      if (a.ckpt_stride > 0 && pos % a.ckpt_stride == 0 && !*abort) {
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
    }
    if (it.last && !*abort) store(a.S_final + ((int64_t)it.seq * a.H + h) * hstate);
  } else {
    regs_more<96>();
    // ---- scores: a row i of the chunk for two threads, of warps w and w + 4
    const int w = warp & 3, half = (warp - 8) >> 2, i = 32 * w + lane;
    const uint32_t lane_at = (uint32_t)(32 * w) << 16;
    constexpr int OH = DV == 128 ? 64 : 32;                 // columns of Q S to scale: heads of 32 value channels, the first warp's alone
    for (int c = 0; c < nch; ++c) {
      const int s = c & 1;
      const uint32_t t_p = t_qk + lane_at;
      wait_w(gate + 8 * s, c >> 1, abort);
      const float near = s_near[128 * s + i];
      const float4 gap = *reinterpret_cast<const float4*>(s_gap + 16 * s + 4 * w);
      const float far[3] = {a.scale * ex2(near + gap.x), a.scale * ex2(near + gap.y), a.scale * ex2(near + gap.z)};   // used for blocks before w
      const float all = a.scale * ex2(near + gap.w), whole = s_near[128 * s + 32 * w + 31];   // the own block's decay
      wait_w(qkd + 8 * s, c >> 1, abort);
      fence_after();
      // Columns 32 b .. of P, bf16, over the scores' first half.  The first warp takes its rows' own block and, of the last
      // rows, the one before; a block is written over columns of blocks at or before its own, so the warps read all they need,
      // meet, and write.
      uint32_t p[2][16];
      const int b0 = half == 0 ? w : 0, b1 = half == 0 ? (w == 3 ? 2 : -1) : (w >= 2 ? 1 : -1);   // this warp's blocks (-1: none)
      const bool first = half == 0 || w > 0;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int b = u == 0 ? (first ? b0 : -1) : b1;
        if (b < 0) {
#pragma unroll
          for (int j = 0; j < 16; ++j) p[u][j] = 0;
          continue;
        }
        float x[32];
        tmem_ld32(t_p + 32 * b, x);
        const bool own = u == 0 && half == 0;
        if (own && whole < -100.f) {                        // the factors of the form below would leave fp32's range
          const float* nj = s_near + 128 * s + 32 * w;
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const float2 lj = *reinterpret_cast<const float2*>(nj + j);
            p[u][j / 2] = pack2(x[j] * (a.scale * ex2(fminf(near - lj.x, 0.f))), x[j + 1] * (a.scale * ex2(fminf(near - lj.y, 0.f))));
          }
        } else {
          // from the block's end, where that comes before the row; from behind it, 2^(near - whole) >= 1, for its own
          const float f = own ? a.scale * ex2(near - whole) : b == 0 ? far[0] : b == 1 ? far[1] : far[2];
          const float* cj = s_col + 128 * s + 32 * b;
          const float2 f2 = make_float2(f, f);
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            const float4 cf = *reinterpret_cast<const float4*>(cj + j);
            const float2 y = __fmul2_rn(__fmul2_rn(make_float2(cf.x, cf.y), f2), make_float2(x[j], x[j + 1]));
            const float2 z = __fmul2_rn(__fmul2_rn(make_float2(cf.z, cf.w), f2), make_float2(x[j + 2], x[j + 3]));
            p[u][j / 2] = pack2(y.x, y.y);
            p[u][j / 2 + 1] = pack2(z.x, z.y);
          }
        }
        if (own) {                                          // columns behind the row: nothing, whatever they held
#pragma unroll
          for (int j = 0; j < 16; ++j) p[u][j] = lane > 2 * j ? p[u][j] : lane == 2 * j ? p[u][j] & 0xffffu : 0u;
        }
      }
      // the two warps of these rows: all scores are read
      fence_before();
      asm volatile("barrier.cta.sync %0, 64;" :: "r"(1 + w) : "memory");
      fence_after();
      // written blocks: the first warp its own (w) and the last (3, zeros unless w = 3 or block 2 of w = 3); the second the rest
      if (half == 0) {
        tmem_st16u(t_p + 16 * w, p[0]);
        if (w == 3) {
          tmem_st16u(t_p + 16 * 2, p[1]);
        } else {
#pragma unroll
          for (int b = 1; b < 4; ++b)
            if (b > w && (b & 1)) {
              const uint32_t zero[16] = {};
              tmem_st16u(t_p + 16 * b, zero);
            }
        }
      } else {
        if (w > 0) tmem_st16u(t_p, p[0]);
        if (w >= 2) tmem_st16u(t_p + 16, p[1]);
#pragma unroll
        for (int b = 1; b < 4; ++b)
          if (b > w && !(b & 1)) {
            const uint32_t zero[16] = {};
            tmem_st16u(t_p + 16 * b, zero);
          }
      }
      wait_w(qsd, c, abort);
      fence_after();
      if (OH * half < DV) {
#pragma unroll
        for (int e = 0; e < OH; e += 32) {                  // e^b Q S
          float x[32];
          uint32_t y[16];
          tmem_ld32(t_o + lane_at + OH * half + e, x);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
              const float2 z = __fmul2_rn(make_float2(x[16 * q + j], x[16 * q + j + 1]), make_float2(all, all));
              y[j] = __float_as_uint(z.x);
              y[j + 1] = __float_as_uint(z.y);
            }
            tmem_st16u(t_o + lane_at + OH * half + e + 16 * q, y);
          }
        }
      }
      tmem_st_wait();
      fence_before();
      arrive_w(p_ready, lane);
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == 29) tmem_dealloc(tmem, 512);
}

// First pass: a segment's state from zero, (e^(B - b) K)^T V with B the segment's whole decay, in steps of 64 tokens.  The steps go backwards,
// so that the decay from a step's end to the segment's end is known; the products of two steps each (two accumulators in turn) are summed in
// registers.  The decayed keys' three parts are the product's A operand in tensor memory (two steps of them), a lane per key channel: through
// shared memory, written once and read by the products, they took most of its bandwidth.  Warps 0-7 decay the keys of the even steps, 8-15 of
// the odd ones, 32 tokens of 32 channels each: what bounds the pass is a warp's own chain of waits (200 to 400 clocks each, also
// for phases long past) and accesses, of which this has two waits in two steps' time.  All of them sum; 16 works out the decays, 17
// copies, 18 issues the products.
template <int DK, int DV>
__global__ void __launch_bounds__(608, 1)
kda_linattn_tc_local_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv, const LinPrefillArgs a,
                            const __grid_constant__ LinSched sched) {
  using L = LinTc<DK, DV>;
  constexpr int AK = L::AK, AV = L::AV, R = kC / 2, NS = L::LS;
  extern __shared__ __align__(1024) unsigned char sm[];
  unsigned char* misc = sm + L::LMISC;
  const uint32_t base = smem_u32(sm), bars = smem_u32(misc);
  const uint32_t full_k = bars, full_v = bars + 8 * NS, kvd = bars + 16 * NS, kbar = bars + 24 * NS;   // [NS] each
  uint32_t* tslot = reinterpret_cast<uint32_t*>(misc + 32 * NS);
  volatile int* abort = reinterpret_cast<volatile int*>(misc + 32 * NS + 4);
  float* s_f = reinterpret_cast<float*>(misc + 256);                    // [NS][R]
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;   // warp: known to be the same for its lanes
  const int item = blockIdx.x / (unsigned)a.H, h = blockIdx.x - item * a.H, hk = h / a.share;   // the heads of a row together
  if (base & 1023) {                                        // the swizzled tiles need it
    if (tid == 0) atomicOr(&g_kda_device_error, kDevErrWait);
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(full_k + 8 * i, 2);                         // the copy and the decays
      mbar_init(full_v + 8 * i, 1);
      mbar_init(kvd + 8 * i, 1);
      mbar_init(kbar + 8 * i, 8);
    }
    *abort = 0;
    mbar_init_fence();
  }
  int lo = 0, hi = sched.n_seqs - 1;                        // slot -> segment: every sequence's last one has none
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (sched.item_base[mid] - mid <= item) lo = mid; else hi = mid - 1;
  }
  const LinItem it = lin_item(sched, item + lo);
  const int n = it.n / R;                                   // whole steps, an even number: only last segments end elsewhere
  const int64_t at = blockIdx.x;
  mla_grid_wait();
  if (warp == 18) tmem_alloc(smem_u32(tslot), 512);
  mla_grid_next();
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *tslot;
  const auto acc_at = [&](int c) { return tmem + 128 * (c >> 1 & 1); };
  const auto key_at = [&](int c) { return tmem + 256 + 96 * (c & 1); };   // hi, lo, least: 32 columns each
  if (warp == 17) {
    int asked = 0;
    Ring r;
    for (int c = 0; c < n; ++c, r.step(NS)) {
      const int s = r.slot, y = (int)(it.t0 + (int64_t)(n - 1 - c) * R);
      if (c >= NS && !wait_w(kvd + 8 * s, r.phase ^ 1, abort)) break;
      if (lane == 0) {
        mbar_expect_tx(full_k + 8 * s, L::HK);
        for (int i = 0; i < AK; ++i) tma_load_2d(base + s * L::STAGE + i * R * 128, &mk, hk * DK + 64 * i, y, full_k + 8 * s);
        mbar_expect_tx(full_v + 8 * s, L::HV);
        for (int i = 0; i < AV; ++i) tma_load_2d(base + s * L::STAGE + L::HK + i * R * 128, &mv, h * DV + 64 * i, y, full_v + 8 * s);
      }
      asked = c + 1;
    }
    for (int c = max(0, asked - NS); c < asked; ++c) {      // no copy is left under way
      mbar_wait(full_k + 8 * (c % NS), (c / NS) & 1);
      mbar_wait(full_v + 8 * (c % NS), (c / NS) & 1);
    }
    __syncwarp();
  } else if (warp == 18) {
    constexpr uint32_t ID = idesc_bf16(128, DV, false, true);   // rows past the key channels are not read
    Ring r;
    const uint32_t el = elect_one();
    for (int c = 0; c < n; ++c, r.step(NS)) {
      const int s = r.slot;
      if (!wait_w(kbar + 8 * s, r.phase, abort) || !wait_w(full_v + 8 * s, r.phase, abort)) break;
      fence_after();
      const uint32_t v = lo_mn(base + s * L::STAGE + L::HK, R * 128);
#pragma unroll
      for (int part = 2; part >= 0; --part) {               // the small parts first
#pragma unroll
        for (int j = 0; j < R / 16; ++j) mma_ts_e(el, acc_at(c), key_at(c) + 32 * part + 8 * j, v + 128 * j, ID, (c & 1) || part < 2 || j > 0);
      }
      commit_e(el, kvd + 8 * s);
    }
  } else if (warp == 16) {
    constexpr int AT = 4;                                   // steps whose decays are asked for together, while the ones before are worked out
    const float* g = a.g + h;
    int64_t behind = 0;                                     // decay of the steps behind this one
    float x[AT][2], next[AT][2];
    const auto fetch = [&](int c, float (&to)[AT][2]) {
#pragma unroll
      for (int u = 0; u < AT; ++u)
#pragma unroll
        for (int i = 0; i < 2; ++i) to[u][i] = c + u < n ? g[(it.t0 + (int64_t)(n - 1 - c - u) * R + 2 * lane + i) * a.g_stride] : 0.f;
    };
    fetch(0, x);
    Ring r;
    for (int c0 = 0; c0 < n; c0 += AT) {
      fetch(c0 + AT, next);
#pragma unroll
      for (int u = 0; u < AT; ++u) {
        const int c = c0 + u;
        if (c >= n) break;
        bool bad = false;
        const int64_t one = lin_fixed(x[u][0], &bad), two = lin_fixed(x[u][1], &bad);
        if (bad) atomicOr(&g_kda_device_error, kDevErrGate);
        const int64_t sum = warp_scan(one + two, lane), all = __shfl_sync(0xffffffffu, sum, 31);
        const float f0 = exp2f(lin_float(behind + all - (sum - two))), f1 = exp2f(lin_float(behind + all - sum));
        if (behind > kLinLeast) behind += all;
        if (c >= NS) wait_w(kbar + 8 * r.slot, r.phase ^ 1, abort);
        *reinterpret_cast<float2*>(s_f + R * r.slot + 2 * lane) = make_float2(f0, f1);
        arrive_w(full_k + 8 * r.slot, lane);
        r.step(NS);
      }
#pragma unroll
      for (int u = 0; u < AT; ++u) {
        x[u][0] = next[u][0];
        x[u][1] = next[u][1];
      }
    }
    if (lane == 0) a.seg_decay[at] = lin_factor(behind);
  } else {
    constexpr int NC = DV / 4;                              // columns of the state per thread, of row `ch`
    const int qd = warp & 3, cols = NC * (warp >> 2), half = warp >> 2 & 1, ch = 32 * qd + lane;
    const bool mine = 32 * qd < DK;                         // the same for a warp
    const uint32_t lane_at = (uint32_t)(32 * qd) << 16;
    float S[NC];
#pragma unroll
    for (int e = 0; e < NC; ++e) S[e] = 0.f;
    bool ok = true;
    int added = 0;                                          // pairs of steps
    const auto add = [&] {                                  // the next pair's products, which are done
      if (mine) {
#pragma unroll
        for (int e = 0; e < NC; e += 8) {
          float x[8];
          tmem_ld8(acc_at(2 * added) + lane_at + cols + e, x);
#pragma unroll
          for (int i = 0; i < 8; ++i) S[e + i] += x[i];
        }
      }
      ++added;
    };
    // this channel's values of token 32 half + t: 64 channels of a token are a row of 128 bytes, its 16-byte pieces in an order of the row's own
    const uint32_t at_k = (ch >> 6) * (R * 128) + 32 * half * 128 + (ch & 7) * 2, piece = (ch & 63) >> 3;
    Ring r, two;                                            // this step's stage, that of the last but one
    for (int i = 0; i < warp >> 3; ++i) {
      r.step(NS);
      two.step(NS);
    }
    for (int c = warp >> 3; c < n; c += 2) {
      const int s = r.slot;
      // the copy has waited for the products that read this stage before
      ok = wait_w(full_k + 8 * s, r.phase, abort) && ok;
      uint32_t w[2][3][8];
      if (mine) {
        const unsigned char* k = sm + s * L::STAGE + at_k;
        const float* f = s_f + R * s + 32 * half;
#pragma unroll
        for (int t = 0; t < 32; t += 4) {
          const float4 f4 = *reinterpret_cast<const float4*>(f + t);
          float x[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            x[i] = __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t*>(k + (t + i) * 128 + ((piece ^ ((t + i) & 7)) << 4)) << 16);
          auto& to = w[t / 16];
          const int j = t % 16 / 2;
          split_two(make_float2(x[0], x[1]), make_float2(f4.x, f4.y), to[0][j], to[1][j], to[2][j]);
          split_two(make_float2(x[2], x[3]), make_float2(f4.z, f4.w), to[0][j + 1], to[1][j + 1], to[2][j + 1]);
        }
      }
      if (c >= 2) {                                         // the products of the step before last have read this operand's place
        ok = wait_w(kvd + 8 * two.slot, two.phase, abort) && ok;
        fence_after();
        two.step(NS);
        two.step(NS);
      }
      if (mine) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int p = 0; p < 3; ++p) tmem_st8u(key_at(c) + lane_at + 32 * p + 16 * half + 8 * u, w[u][p]);
      }
      // The pair that those products (an odd step's) or the ones before them (an even step's) ended.  It is the last but one before this step's
      // pair, whose accumulator it has: read here, before the arrival, by both kinds of warps (the odd steps' a step earlier).
      if (c >= 3) add();
      tmem_st_wait();
      fence_before();
      arrive_w(kbar + 8 * s, lane);
      r.step(NS);
      r.step(NS);
    }
    ok = wait_w(kvd + 8 * ((n - 1) % NS), (n - 1) / NS, abort) && ok;
    fence_after();
    while (added < n / 2) add();
    if (ok && mine) {
      float* dst = a.seg_state + at * ((int64_t)DK * DV) + (int64_t)ch * DV + cols;
#pragma unroll
      for (int e = 0; e < NC; e += 4) *reinterpret_cast<float4*>(dst + e) = make_float4(S[e], S[e + 1], S[e + 2], S[e + 3]);
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == 18) tmem_dealloc(tmem, 512);
}

template <int DK, int DV>
cudaError_t run_tc(const LinPrefillArgs& a, const LinSched& sched, cudaStream_t s) {
  using L = LinTc<DK, DV>;
  static std::atomic<uint64_t> allowed{0}, allowed_local{0};
  CUtensorMap mq, mk, mv, mo;
  const int64_t H_k = a.H / a.share;
  if (!make_map_rows(&mq, a.q, a.T, H_k * DK, a.q_stride, 64, kC) || !make_map_rows(&mk, a.k, a.T, H_k * DK, a.k_stride, 64, kC) ||
      !make_map_rows(&mv, a.v, a.T, (int64_t)a.H * DV, a.v_stride, 64, kC) ||
      !make_map_rows(&mo, a.o, a.T, (int64_t)a.H * DV, (int64_t)a.H * DV, L::OC, 32))
    return cudaErrorInvalidValue;
  const auto kern = kda_linattn_tc_kernel<DK, DV>;
  if (const cudaError_t e = mla_allow_smem(kern, L::SMEM, allowed)) return e;
  const int local = sched.n_items - sched.n_seqs;
  if (local > 0) {
    const auto first = kda_linattn_tc_local_kernel<DK, DV>;
    if (const cudaError_t e = mla_allow_smem(first, L::LSMEM, allowed_local)) return e;
    CUtensorMap hk, hv;                                     // half a chunk's rows
    if (!make_map_rows(&hk, a.k, a.T, H_k * DK, a.k_stride, 64, kC / 2) || !make_map_rows(&hv, a.v, a.T, (int64_t)a.H * DV, a.v_stride, 64, kC / 2))
      return cudaErrorInvalidValue;
    if (const cudaError_t e = mla_launch(first, (unsigned)(local * a.H), 608, L::LSMEM, s, hk, hv, a, sched)) return e;
    if (const cudaError_t e = launch_linattn_scan(a, sched, s)) return e;
  }
  return mla_launch(kern, (unsigned)(sched.n_items * a.H), 1024, L::SMEM, s, mq, mk, mv, mo, a, sched);
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
