// bf16 attention over the latent page cache on the tensor cores (kda_mla.cuh has the
// division of work, kda_mla_decode.cu the formulas and the merge).
//
// One CTA per SM walks its piece of the line of tiles.  An item is NR query rows (the
// heads and draft positions that read the same tokens); a tile is 64 tokens, staged
// once by TMA as column slabs [64 tokens][64 values] and used twice, since c is both
// key and value:
//   S = Q K^T      M = 64 rows (NR live), N = 64 tokens, K = d_c + d_r:  a thread of the
//                  16x256b TMEM load holds 2 rows x 8 tokens, so a row's maximum takes two
//                  shuffles and one exchange between two warps;
//   O^T += C^T P^T M = 128 channels, N = NR rows, K = 64 tokens: the slabs, read MN-major,
//                  are the A operand, and the accumulator of NR x d_c floats takes
//                  NR d_c / 128 columns of TMEM (256 of 512 at NR = 64, d_c = 512), which
//                  the other orientation (512 columns for 64 rows on half the lanes) would
//                  not leave room for beside S.
// Warps 0-7 do the softmax and write results (warps w and w + 4 share TMEM lanes and take
// half of a tile's tokens each), warp 8 issues the copies, warp 9 the products.  S is
// double-buffered: S of the next tile runs during the softmax of this one whenever its
// slabs have arrived; when they have not, O of this tile goes first so that its slabs are
// free for the copies.
//
// The running reference m of a row moves only when the maximum rises more than 2^8
// above it (weights then stay below 2^8, far inside bf16's and fp32's range), so O in
// TMEM is rescaled rarely.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <numeric>

#include "../../include/kda.h"
#include "kda_common.cuh"
#include "kda_mla.cuh"
#include "kda_tc.cuh"
#include "kda_tmap.h"

namespace kda {
namespace {

using namespace tc;

constexpr int kSoft = 8;               // softmax warps, two per quarter of the TMEM lanes
constexpr int kThreads = 32 * (kSoft + 2);
constexpr int kPairBytes = 16384;      // two column slabs: [64 tokens][64 values] each
constexpr int kSlabBytes = 8192;
constexpr float kLazy = 8.f;           // log2 units the maximum may exceed the reference by

template <int NR> struct Cfg {
  static constexpr int kPBytes = NR * 128;
  static constexpr int kPBufs = NR == 64 ? 1 : 2;    // P tiles: at 64 rows the second's room goes to a position slab
  static constexpr int kPairs = NR == 64 ? 8 : 10;   // ring of slab pairs
  static constexpr int kRopes = 2;                   // ring of position slabs
  // Q slabs, P tiles, the rings; an M = 64 product reads 64 rows of a 32-row Q slab,
  // the last of them 4 KB into P
  static constexpr int smem(int slabs) {
    return 1024 + slabs * NR * 128 + kPBufs * kPBytes + kPairs * kPairBytes + kRopes * kSlabBytes;
  }
  static_assert(smem(9) + 2048 <= 232448, "2 KB are left for the static shared memory");
  static constexpr uint32_t kCols = NR == 64 ? 512 : 256;   // TMEM: 4 NR of O, 128 of S
};

struct Bars {
  uint64_t pair_full[10], pair_empty[10];
  uint64_t rope_full[2], rope_empty[2];
  uint64_t q_full, q_empty;
  uint64_t s_full[2], p_full[2], pv_done[2];
  uint64_t o_free, drain;
};

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t mbar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
      :: "r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(mbar) : "memory");
}
// has this phase completed (never suspends the thread)
__device__ __forceinline__ bool mbar_poll(uint32_t mbar, uint32_t parity) {
  uint32_t done;
  asm volatile("{ .reg .pred p; mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
               : "=r"(done) : "r"(mbar), "r"(parity) : "memory");
  return done != 0;
}
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{ .reg .pred p; .reg .b32 r; elect.sync r|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(e));
  return e != 0;
}
// barrier of the softmax warps; true if `x` held in any of their threads
__device__ __forceinline__ bool vote(bool x) {
  uint32_t r;
  asm volatile("{ .reg .pred p, q; setp.ne.b32 p, %1, 0; barrier.cta.red.or.pred q, 1, %2, p; selp.u32 %0, 1, 0, q; }"
               : "=r"(r) : "r"((uint32_t)x), "n"(32 * kSoft) : "memory");
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

// A ring position: slot and phase parity advance together.
struct Ring {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void step(int n) {
    if (++slot == n) { slot = 0; phase ^= 1; }
  }
};

template <int NR>
__global__ void __launch_bounds__(kThreads, 1)
kda_mla_tc_kernel(const MlaArgs a, const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_qr,
                  const __grid_constant__ CUtensorMap map_kv, const int box_rows) {
  using C = Cfg<NR>;
  extern __shared__ unsigned char dyn[];
  __shared__ Bars bars;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  // per row: the tile's maximum in each half (by parity of the tile), the reference, and
  // the rescale factor, at a segment's end the sum
  __shared__ float row_x[2][2][64], row_m[64], row_f[64];
  const int lane = threadIdx.x & 31;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  const int np = a.d_c / 128;                          // slab pairs per tile
  const bool rope = a.d_r > 0;
  const int slabs = 2 * np + (rope ? 1 : 0);
  const uint32_t q_smem = (smem_u32(dyn) + 1023u) & ~1023u;
  const uint32_t p_smem = q_smem + slabs * NR * 128;
  const uint32_t pair_smem = p_smem + C::kPBufs * C::kPBytes;
  const uint32_t rope_smem = pair_smem + C::kPairs * kPairBytes;
  const uint32_t bb = smem_u32(&bars);
#define BAR(x) (bb + (uint32_t)offsetof(Bars, x))
#define BARI(x, i) (bb + (uint32_t)offsetof(Bars, x) + 8u * (uint32_t)(i))
  volatile int* abort = &abort_flag;

  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int i = 0; i < C::kPairs; ++i) { mbar_init(BARI(pair_full, i), 1); mbar_init(BARI(pair_empty, i), 1); }
    for (int i = 0; i < 2; ++i) {
      mbar_init(BARI(rope_full, i), 1); mbar_init(BARI(rope_empty, i), 1);
      mbar_init(BARI(s_full, i), 1); mbar_init(BARI(p_full, i), kSoft); mbar_init(BARI(pv_done, i), 1);
    }
    mbar_init(BAR(q_full), 1); mbar_init(BAR(q_empty), 1); mbar_init(BAR(o_free), kSoft); mbar_init(BAR(drain), 1);
    mbar_init_fence();
  }
  if (threadIdx.x < 64) row_m[threadIdx.x] = -INFINITY;
  if (warp == kSoft + 1) tmem_alloc(smem_u32(&tmem_slot), C::kCols);
  fence_before();
  MlaWalk walk = mla_plan<kThreads>(a, blockIdx.x, gridDim.x);   // ends in a block barrier
  fence_after();
  const uint32_t tm = __shfl_sync(0xffffffffu, *(volatile uint32_t*)&tmem_slot, 0);
  const uint32_t tm_o = tm, tm_s = tm + 4 * NR;
  MlaSeg s;

  if (warp == kSoft) {
    // ---- copies ----------------------------------------------------------------
    Ring pr, rr;
    uint32_t pairs_sent = 0, ropes_sent = 0;
    int seg = 0;
    bool bad = false, live = true;
    const int nbox = kMlaTile / box_rows;
    while (live && walk.next(a, s)) {
      if (seg > 0 && !wait_phase_w(BAR(q_empty), (seg - 1) & 1, abort)) break;
      if (lane == 0) {
        mbar_expect_tx(BAR(q_full), (uint32_t)slabs * NR * 128);
        for (int i = 0; i < 2 * np; ++i) tma_load_2d(q_smem + i * NR * 128, &map_q, 64 * i, (int)s.row0, BAR(q_full));
        if (rope) tma_load_2d(q_smem + 2 * np * NR * 128, &map_qr, 0, (int)s.row0, BAR(q_full));
      }
      ++seg;
      for (int tile = s.tile0; tile < s.tile1; ++tile) {
        // lane (slab s, box i) copies box i of slab s of each pair; boxes past the
        // item's tokens come from beyond the last page, that is as zeros
        const int sl = lane / nbox, box = lane % nbox;
        const int t = tile * kMlaTile + box * box_rows;
        int z = (int)a.n_pages, y = 0;
        if (t < s.tokens) {
          const int64_t page = mla_page(a, s.b, t, &bad);
          if (page >= 0) z = (int)page;
          y = t % a.page_tokens;
        }
        for (int j = 0; j < np; ++j) {
          if (pairs_sent >= C::kPairs && !wait_phase_w(BARI(pair_empty, pr.slot), pr.phase ^ 1, abort)) { live = false; break; }
          const uint32_t bar = BARI(pair_full, pr.slot);
          if (lane == 0) mbar_expect_tx(bar, kPairBytes);
          __syncwarp();
          if (sl < 2)
            tma_load_3d(pair_smem + pr.slot * kPairBytes + sl * kSlabBytes + box * box_rows * 128, &map_kv,
                        128 * j + 64 * sl, y, z, bar);
          pr.step(C::kPairs);
          ++pairs_sent;
        }
        if (!live) break;
        if (rope) {
          if (ropes_sent >= C::kRopes && !wait_phase_w(BARI(rope_empty, rr.slot), rr.phase ^ 1, abort)) { live = false; break; }
          const uint32_t bar = BARI(rope_full, rr.slot);
          if (lane == 0) mbar_expect_tx(bar, kSlabBytes);
          __syncwarp();
          if (sl == 0) tma_load_3d(rope_smem + rr.slot * kSlabBytes + box * box_rows * 128, &map_kv, a.d_c, y, z, bar);
          rr.step(C::kRopes);
          ++ropes_sent;
        }
      }
    }
    if (bad) atomicOr(&g_kda_device_error, KDA_DEVERR_INDEX);
    // every copy has landed before the CTA may end (after a wait that gave up, too)
    if (seg > 0) mbar_wait(BAR(q_full), (seg - 1) & 1);
    for (int i = 0; i < C::kPairs && i < (int)pairs_sent; ++i) {
      const uint32_t uses = (pairs_sent - 1 - i) / C::kPairs;       // earlier copies into slot i
      mbar_wait(BARI(pair_full, i), uses & 1);
    }
    for (int i = 0; i < C::kRopes && i < (int)ropes_sent; ++i) mbar_wait(BARI(rope_full, i), ((ropes_sent - 1 - i) / C::kRopes) & 1);
  } else if (warp == kSoft + 1) {
    // ---- products --------------------------------------------------------------
    // The whole warp runs this and one elected lane issues: operand descriptors then stay
    // in uniform registers (an issue costs ~10 clocks; from a single thread's registers ~70).
    constexpr uint32_t id_s = idesc_bf16(64, 64, false, false), id_o = idesc_bf16(128, NR, true, false);
    Ring sp, vp, rr;                                     // pairs as keys, pairs as values, position slabs
    uint32_t gt = 0;                                     // tiles so far
    int seg = 0, pend_seg = 0;
    bool pend = false, pend_first = false, live = true;

    auto values = [&]() -> bool {                        // O^T += C^T P^T of tile gt - 1
      const uint32_t u = gt - 1;
      if (!wait_phase_w(BARI(p_full, u & 1), (u >> 1) & 1, abort)) return false;
      if (pend_first && pend_seg > 0 && !wait_phase_w(BAR(o_free), (pend_seg - 1) & 1, abort)) return false;
      fence_after();
      const uint32_t pb = __shfl_sync(0xffffffffu, p_smem + (u % C::kPBufs) * C::kPBytes, 0);
      const uint32_t more = __shfl_sync(0xffffffffu, pend_first ? 0 : 1, 0);
      for (int j = 0; j < np; ++j) {
        const uint32_t base = __shfl_sync(0xffffffffu, pair_smem + vp.slot * kPairBytes, 0);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          mma_w(tm_o + j * NR, desc_mn(base, 64, ks), desc_k(pb, NR, ks), id_o, ks == 0 ? more : 1);
        mma_commit_w(BARI(pair_empty, vp.slot));
        vp.step(C::kPairs);
      }
      mma_commit_w(BARI(pv_done, u & 1));
      pend = false;
      return true;
    };

    while (live && walk.next(a, s)) {
      for (int tile = s.tile0; tile < s.tile1; ++tile) {
        const bool first = tile == s.tile0;
        if (pend) {
          // keys of this tile not all here: the last tile's values go first
          const int e = sp.slot + np - 1;
          const int last = e >= C::kPairs ? e - C::kPairs : e;
          bool here = mbar_poll(BARI(pair_full, last), sp.phase ^ (e >= C::kPairs ? 1u : 0u));
          if (rope) here &= mbar_poll(BARI(rope_full, rr.slot), rr.phase);
          if (first) here &= mbar_poll(BAR(q_full), seg & 1);
          if (!__all_sync(0xffffffffu, here) && !values()) { live = false; break; }
        }
        if (first && !wait_phase_w(BAR(q_full), seg & 1, abort)) { live = false; break; }
        const uint32_t sd = __shfl_sync(0xffffffffu, tm_s + (gt & 1) * 64, 0);
        for (int j = 0; j < np; ++j) {
          if (!wait_phase_w(BARI(pair_full, sp.slot), sp.phase, abort)) { live = false; break; }
          fence_after();
          const uint32_t base = __shfl_sync(0xffffffffu, pair_smem + sp.slot * kPairBytes, 0);
          const uint32_t qb = q_smem + 2 * j * NR * 128;
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)
            mma_w(sd, desc_k(qb, NR, ks), desc_k(base, 64, ks), id_s, ks > 0 || j > 0);
          sp.step(C::kPairs);
        }
        if (live && rope) {
          if (!wait_phase_w(BARI(rope_full, rr.slot), rr.phase, abort)) { live = false; break; }
          const uint32_t base = __shfl_sync(0xffffffffu, rope_smem + rr.slot * kSlabBytes, 0);
          const uint32_t qb = q_smem + 2 * np * NR * 128;
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) mma_w(sd, desc_k(qb, NR, ks), desc_k(base, 64, ks), id_s, 1);
          mma_commit_w(BARI(rope_empty, rr.slot));
          rr.step(C::kRopes);
        }
        if (!live) break;
        mma_commit_w(BARI(s_full, gt & 1));
        if (tile + 1 == s.tile1) mma_commit_w(BAR(q_empty));
        if (pend && !values()) { live = false; break; }
        pend = true;
        pend_first = first;
        pend_seg = seg;
        ++gt;
      }
      ++seg;
    }
    if (live && pend) values();
    mma_commit_w(BAR(drain));                            // no product outlives the CTA's memory
    mbar_wait(BAR(drain), 0);
    __syncwarp();
  } else {
    // ---- softmax and results ---------------------------------------------------
    uint32_t gt = 0;
    bool dead = false;
    Ring vp;                                             // first pair of the tile
    const int quarter = warp & 3, half = warp >> 2;
    const uint32_t quad = (uint32_t)quarter << 21;       // TMEM lanes 32 quarter ..
    const bool rows_here = 16 * quarter < NR;            // S rows 16 quarter .. of the item
    const int r0 = 16 * quarter + (lane >> 2);           // this thread's rows: r0 and r0 + 8
    const bool leader = rows_here && (lane & 3) == 0;
    while (!dead && walk.next(a, s)) {
      const int lim0 = mla_row_limit(a, s, r0), lim1 = mla_row_limit(a, s, r0 + 8);
      float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
      for (int tile = s.tile0; tile < s.tile1; ++tile, ++gt) {
        const uint32_t buf = gt & 1;
        const int t0 = tile * kMlaTile;
        dead |= !wait_phase(BARI(s_full, buf), (gt >> 1) & 1, abort);
        fence_after();
        float v[16];
        if (rows_here) {
          tmem_ld_16x32(tm_s + buf * 64 + 32 * half + quad, v);
          const int c0 = t0 + 32 * half + 2 * (lane & 3);
          if (t0 + kMlaTile > min(lim0, lim1)) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                if (c0 + 8 * i + e >= lim0) v[4 * i + e] = -INFINITY;
                if (c0 + 8 * i + e >= lim1) v[4 * i + 2 + e] = -INFINITY;
              }
          }
          float x0 = fmaxf(v[0], v[1]), x1 = fmaxf(v[2], v[3]);
#pragma unroll
          for (int i = 1; i < 4; ++i) {
            x0 = fmaxf(x0, fmaxf(v[4 * i], v[4 * i + 1]));
            x1 = fmaxf(x1, fmaxf(v[4 * i + 2], v[4 * i + 3]));
          }
#pragma unroll
          for (int o = 1; o < 4; o <<= 1) {
            x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, o));
            x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, o));
          }
          if (leader) {
            row_x[buf][half][r0] = x0 * a.scale_log2;
            row_x[buf][half][r0 + 8] = x1 * a.scale_log2;
          }
        }
        if (vote(dead)) { dead = true; break; }
        // every warp looks at all rows, so all agree whether some reference has to move
        bool up = false, again = false;
#pragma unroll
        for (int r = lane; r < NR; r += 32) {
          const float m = row_m[r], x = fmaxf(row_x[buf][0][r], row_x[buf][1][r]);
          const bool u = x > m + kLazy;                  // m = -inf: the row's first finite maximum
          up |= u;
          again |= u && m != -INFINITY;
        }
        if (__any_sync(0xffffffffu, up)) {
          again = __any_sync(0xffffffffu, again);
          float f0 = 1.f, f1 = 1.f;
          if (rows_here) {
            const float x0 = fmaxf(row_x[buf][0][r0], row_x[buf][1][r0]);
            const float x1 = fmaxf(row_x[buf][0][r0 + 8], row_x[buf][1][r0 + 8]);
            if (x0 > m0 + kLazy) { f0 = ex2(m0 - x0); m0 = x0; }   // from -inf: times 0, of nothing yet
            if (x1 > m1 + kLazy) { f1 = ex2(m1 - x1); m1 = x1; }
            l0 *= f0;
            l1 *= f1;
          }
          vote(false);                                   // all have read row_m
          if (leader && half == 0) {
            row_m[r0] = m0; row_m[r0 + 8] = m1;
            row_f[r0] = f0; row_f[r0 + 8] = f1;
          }
          vote(false);
          if (again) {
            // O holds every earlier tile of the segment once the last of them is done
            dead |= !wait_phase(BARI(pv_done, buf ^ 1), ((gt - 1) >> 1) & 1, abort);
            fence_after();
            for (int j = 0; j < np; ++j)
#pragma unroll
              for (int c = 0; c < NR / 2; c += 16) {
                float o[16];
                const int col = half * (NR / 2) + c;
                const uint32_t at = tm_o + j * NR + col + quad;
                tmem_ld16(at, o);
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] *= row_f[col + i];
                tmem_st16(at, o);
              }
          }
        }
        // the tile's tokens past the item's end: whatever the page holds there must not
        // meet the zero weights as NaN or infinity
        const int past = s.tokens - t0;
        if (past < kMlaTile) {
          Ring p = vp;
          for (int j = 0; j < np; ++j) {
            for (int i = threadIdx.x; i < 2 * (kMlaTile - past) * 8; i += 32 * kSoft) {
              const int sl = i / ((kMlaTile - past) * 8), k = i % ((kMlaTile - past) * 8);
              const uint32_t at = pair_smem + p.slot * kPairBytes + sl * kSlabBytes + past * 128 + k * 16;
              asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" :: "r"(at), "r"(0) : "memory");
            }
            p.step(C::kPairs);
          }
        }
        vp.slot += np;
        if (vp.slot >= C::kPairs) vp.slot -= C::kPairs;
        uint32_t pk[8];
        if (rows_here) {
          const float b0 = m0 == -INFINITY ? 0.f : m0, b1 = m1 == -INFINITY ? 0.f : m1;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float p0 = ex2(fmaf(v[4 * i], a.scale_log2, -b0)), p1 = ex2(fmaf(v[4 * i + 1], a.scale_log2, -b0));
            const float p2 = ex2(fmaf(v[4 * i + 2], a.scale_log2, -b1)), p3 = ex2(fmaf(v[4 * i + 3], a.scale_log2, -b1));
            l0 += p0 + p1;                               // fp32 weights; the product takes them as bf16
            l1 += p2 + p3;
            const __nv_bfloat162 u = __floats2bfloat162_rn(p0, p1), w = __floats2bfloat162_rn(p2, p3);
            pk[2 * i] = *reinterpret_cast<const uint32_t*>(&u);
            pk[2 * i + 1] = *reinterpret_cast<const uint32_t*>(&w);
          }
        }
        // the P tile's last reader
        if (gt >= C::kPBufs) {
          const uint32_t u = gt - C::kPBufs;
          dead |= !wait_phase(BARI(pv_done, u & 1), (u >> 1) & 1, abort);
        }
        if (rows_here) {
          const uint32_t pb = p_smem + (gt % C::kPBufs) * C::kPBytes + r0 * 128 + (lane & 3) * 4;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t at = pb + ((uint32_t)((4 * half + i) ^ (r0 & 7)) << 4);   // r0 and r0 + 8 share r % 8
            asm volatile("st.shared.b32 [%0], %1;" :: "r"(at), "r"(pk[2 * i]) : "memory");
            asm volatile("st.shared.b32 [%0], %1;" :: "r"(at + 1024), "r"(pk[2 * i + 1]) : "memory");
          }
        }
        fence_async_smem();
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(BARI(p_full, buf));
      }
      if (dead) break;
      // results of the segment
      dead |= !wait_phase(BARI(pv_done, (gt - 1) & 1), ((gt - 1) >> 1) & 1, abort);
      const bool whole = mla_whole(a, s);
      const int64_t slot = (s.item + blockIdx.x) * a.nr;
      if (threadIdx.x == 0) mla_note_item(a, s, blockIdx.x);
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, o);
        l1 += __shfl_xor_sync(0xffffffffu, l1, o);
      }
      if (leader && half == 1) { row_f[r0] = l0; row_f[r0 + 8] = l1; }   // every P, so every use of row_f, is done
      if (vote(dead)) { dead = true; break; }
      fence_after();
      if (leader && half == 0) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int r = r0 + 8 * k;
          const float m = k ? m1 : m0, l = (k ? l1 : l0) + row_f[r];
          row_f[r] = l > 0.f ? 1.f / l : 0.f;
          row_m[r] = -INFINITY;                          // for the next segment
          if (r < s.nrows) {
            if (!whole) a.part_ml[slot + r] = make_float2(m, l);
            else if (a.lse) a.lse[s.row0 + r] = 0.6931471805599453f * (m + log2f(l));
          }
        }
      }
      vote(false);
      for (int j = 0; j < np; ++j)
#pragma unroll
        for (int c = 0; c < NR / 2; c += 16) {
          float o[16];
          const int col = half * (NR / 2) + c;
          tmem_ld16(tm_o + j * NR + col + quad, o);
          const int e = 128 * j + 32 * quarter + lane;
          if (whole) {
            __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(a.o) + s.row0 * a.d_c + e;
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (col + i < s.nrows) out[(int64_t)(col + i) * a.d_c] = __float2bfloat16_rn(o[i] * row_f[col + i]);
          } else {
            float* out = a.part_o + slot * a.d_c + e;
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (col + i < s.nrows) out[(int64_t)(col + i) * a.d_c] = o[i];
          }
        }
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(o_free));
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == kSoft + 1) tmem_dealloc(tm, C::kCols);
#undef BAR
#undef BARI
}

template <int NR>
cudaError_t run(const MlaArgs& a, const CUtensorMap& mq, const CUtensorMap& mr, const CUtensorMap& mk, int box_rows, int ctas,
                cudaStream_t s) {
  const int smem = Cfg<NR>::smem(2 * (a.d_c / 128) + (a.d_r > 0));
  cudaError_t e = cudaFuncSetAttribute(kda_mla_tc_kernel<NR>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kda_mla_tc_kernel<NR><<<ctas, kThreads, smem, s>>>(a, mq, mr, mk, box_rows);
  return cudaGetLastError();
}

}  // namespace

// Rows per item: 32 when no item could have more, which leaves shared memory for more
// tiles in flight; else 64.
int mla_tc_row_tile(int seq_rows, int64_t prefix_len) { return prefix_len == 0 && seq_rows <= 32 ? 32 : 64; }

cudaError_t launch_mla_tc(const MlaArgs& a, int ctas, cudaStream_t s) {
  const int64_t rows = (int64_t)a.B * a.seq_rows;
  const int d = a.d_c + a.d_r, box_rows = std::gcd(a.page_tokens, kMlaTile);
  CUtensorMap mq, mr{}, mk;
  if (!make_map_2d(&mq, a.q, rows, a.d_c, 2, 64, a.nr, true)) return cudaErrorInvalidValue;
  if (a.d_r > 0 && !make_map_2d(&mr, a.q_pe, rows, a.d_r, 2, 64, a.nr, true)) return cudaErrorInvalidValue;
  if (!make_map_pages(&mk, a.pages, a.n_pages, a.page_bytes, a.page_tokens, d, 64, box_rows)) return cudaErrorInvalidValue;
  return a.nr == 32 ? run<32>(a, mq, mr, mk, box_rows, ctas, s) : run<64>(a, mq, mr, mk, box_rows, ctas, s);
}

int read_and_clear_mla_tc_errors(int* flags) {
  int word = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&word, g_kda_device_error, sizeof(int));
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_kda_device_error, &zero, sizeof(int));
  *flags |= word;
  return (int)e;
}

}  // namespace kda
