// Device pieces that the two tensor-core kernels of the latent page cache share.
#pragma once

#include "kda_tc.cuh"

namespace kda {
namespace tc {

constexpr int kMlaSoft = 8;            // softmax warps
constexpr float kLazy = 8.f;           // log2 units a row's maximum may exceed its reference by
// Reference of a row without a score yet: fp32's lowest, which any score above it outgrows (the
// difference of two finite numbers is at worst infinite, never NaN as with -infinity).
constexpr float kNone = -3.402823466e38f;

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t mbar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
      :: "r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(mbar) : "memory");
}
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t e;
  asm volatile("{ .reg .pred p; .reg .b32 r; elect.sync r|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(e));
  return e;
}
// The low words of operand descriptors (kda_tc.cuh: address and leading offset); the high
// word, stride 1024 and the 128-byte swizzle, is the same for all.  Kept apart so that a step
// along an operand is one 32-bit addition.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo_k(uint32_t base) { return (base >> 4) | (1u << 16); }
__device__ __forceinline__ uint32_t desc_lo_mn(uint32_t base) { return (base >> 4) | ((8192u >> 4) << 16); }
// A product issued by the lane for which `el` is not zero, of a converged warp.
__device__ __forceinline__ void mma_e(uint32_t el, uint32_t d_tmem, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{ .reg .pred p, e; .reg .b64 da, db; setp.ne.b32 e, %5, 0; setp.ne.b32 p, %4, 0; "
      "mov.b64 da, {%1, %6}; mov.b64 db, {%2, %6}; "
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p; }"
      :: "r"(d_tmem), "r"(a), "r"(b), "r"(idesc), "r"(acc), "r"(el), "r"(kDescHi) : "memory");
}
__device__ __forceinline__ void commit_e(uint32_t el, uint32_t mbar) {
  asm volatile("{ .reg .pred e; setp.ne.b32 e, %1, 0; "
               "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0]; }"
               :: "r"(mbar), "r"(el) : "memory");
}
// barrier of the softmax warps; true if `x` held in any of their threads
__device__ __forceinline__ bool vote(bool x) {
  uint32_t r;
  asm volatile("{ .reg .pred p, q; setp.ne.b32 p, %1, 0; barrier.cta.red.or.pred q, 1, %2, p; selp.u32 %0, 1, 0, q; }"
               : "=r"(r) : "r"((uint32_t)x), "n"(32 * kMlaSoft) : "memory");
  return r != 0;
}
// 16 lanes x 32 columns: v[4 i + c] of a thread is row lane / 4 + 8 (c / 2) and column
// 8 i + 2 (lane % 4) + c % 2
__device__ __forceinline__ void tmem_ld_16x32(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr) : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float (&v)[16]) {
  uint32_t r[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(v[i]);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n\t"
      "tcgen05.wait::st.sync.aligned;"
      :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
         "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Wait for a phase; a wait that gives up (after about a second) or meets another role's
// giving up returns false and tells the other roles.
__device__ __forceinline__ bool wait_phase(uint32_t mbar, uint32_t parity, volatile int* abort) {
#pragma unroll 1
  for (int i = 0; i < 64; ++i)
    if (mbar_test(mbar, parity)) return true;
  if (mbar_wait_or_abort(mbar, parity, abort)) return true;
  *abort = 1;
  return false;
}
// The same by a whole warp, which then agrees on the outcome.
__device__ __forceinline__ bool wait_phase_w(uint32_t mbar, uint32_t parity, volatile int* abort) {
  return __all_sync(0xffffffffu, wait_phase(mbar, parity, abort));
}

// Phases that the lanes of a warp wait for, one each (the lanes with `wants`): have they
// all completed; and the wait for it.  PAIR: arrivals may come from the pair's other CTA.
template <bool PAIR = false>
__device__ __forceinline__ bool lanes_done(bool wants, uint32_t mbar, uint32_t parity) {
  uint32_t done = 1;
  if (wants) {
    if constexpr (PAIR)
      asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
                   : "=r"(done) : "r"(mbar), "r"(parity) : "memory");
    else
      done = mbar_test(mbar, parity);
  }
  return __all_sync(0xffffffffu, done != 0);
}
template <bool PAIR = false>
__device__ __forceinline__ bool lanes_wait(bool wants, uint32_t mbar, uint32_t parity, volatile int* abort) {
  const long long t0 = clock64();
#pragma unroll 1
  for (int i = 1;; ++i) {
    if (lanes_done<PAIR>(wants, mbar, parity)) return true;
    if (i % 64 == 0) {
      const bool late = clock64() - t0 > (1LL << 31);   // about a second
      if (__any_sync(0xffffffffu, late || *abort)) {
        if (late) atomicOr(&g_kda_device_error, kDevErrWait);
        *abort = 1;
        return false;
      }
    }
  }
}

// Which of the lanes' phases have completed (never suspends).
__device__ __forceinline__ uint32_t lanes_poll(uint32_t mbar, uint32_t parity) {
  uint32_t done;
  asm volatile("{ .reg .pred p; mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
               : "=r"(done) : "r"(mbar), "r"(parity) : "memory");
  return __ballot_sync(0xffffffffu, done != 0);
}

// box of columns (64 or 128, as slabs), rows, a page
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int y, int slab, int z, uint32_t mbar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
      :: "r"(dst), "l"(map), "r"(0), "r"(y), "r"(slab), "r"(z), "r"(mbar) : "memory");
}

// A ring position: slot and phase parity advance together.
struct Ring {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void step(int n) {
    if (++slot == n) { slot = 0; phase ^= 1; }
  }
};

}  // namespace tc
}  // namespace kda
