// bf16 attention over the latent page cache where more than 64 rows read the same tokens
// (the shared prefix; many heads or long drafts): pairs of CTAs (kda_mla.cuh has the
// division of work, kda_mla_decode.cu the formulas and the merge).
//
// The latent accumulator is d_c floats a row, so one SM's TMEM holds 64 rows of O (256 of
// 512 columns) and one CTA's products are half size: M = 64 runs at half the tensor
// rate.  A pair of CTAs works on 128 rows instead, 64 in each, with two-CTA products of
// M = 128: each CTA supplies its rows of the A operand and half of the B operand, and its
// TMEM gets its 64 rows, the first half of the columns in lanes 0-63 and the second in
// lanes 64-127.  Per tile of 128 tokens:
//   S = Q K^T  N = 128 tokens, K = d_c + d_r: CTA r stages the keys of tokens 64 r ..;
//   O += P C   N = 256 channels (d_c / 256 times; a last one of 128 when d_c is an odd
//              multiple of that), K = 128 tokens: CTA r stages half r of each
//              product's channels, all tokens.
// So a tile is staged once as keys and once as values, each CTA half of either: 272 KB
// into the pair for 128 rows, against 147 KB into each CTA for 64 rows alone.  Per CTA and
// tile the products take 2176 clocks at the tensor rate, and their operands and the copies
// 3008 clocks of shared-memory bandwidth (128 B each), which is the kernel's bound; the
// one-CTA form needs 5000 for the same work.  4096 rows on 16384 tokens, d_c = 512, d_r = 64:
// 106 us, 1.37 PFLOP/s (72% of the measured tensor peak), 2990-3070 clocks per tile.
//
// Roles per CTA: warps 0-7 softmax and results, warp 8 copies queries and keys, warp 9
// values, warp 10 issues the products (in the first CTA only, for both).  Order of the
// products: S of the next tile, then O of this one, so that the softmax runs beside them.
// The weights are rounded to bf16 for O (kda_mla_tc.cu has what that costs).
// Keys and values have a ring of four 16 KB units each, refilled unit by unit as the
// products leave them, each by a warp of its own: with one ring and one copying warp a
// unit's turn came late (4450 clocks per tile).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <numeric>

#include "../../include/kda.h"
#include "kda_common.cuh"
#include "kda_mla.cuh"
#include "kda_mla_tc.cuh"
#include "kda_tc.cuh"
#include "kda_tmap.h"

namespace kda {
namespace {

using namespace tc;

constexpr int kRows = 64;              // rows of one CTA
constexpr int kTile = 128;             // tokens per tile
constexpr int kSoft = kMlaSoft;
constexpr int kThreads = 32 * (kSoft + 3);
constexpr int kUnits = 4;              // ring of keys, ring of values
constexpr int kUnitBytes = 16384;      // two slabs
constexpr int kSlabBytes = 8192;       // [64 tokens][64 values]
constexpr int kPBytes = kRows * kTile * 2;
constexpr int kTails = 4;              // barriers of values that are cleared before use, in turn
constexpr uint32_t kCols = 512;        // TMEM: 256 of O, 2 x 64 of S

int smem_bytes(int slabs) { return 1024 + slabs * kSlabBytes + kPBytes + 2 * kUnits * kUnitBytes + kSlabBytes; }

struct Bars {
  // full: the first CTA's, for both CTAs' copies
  uint64_t k_full[kUnits], k_empty[kUnits], v_full[kUnits], v_empty[kUnits];
  uint64_t rope_full, rope_empty;
  uint64_t q_full, q_empty;
  uint64_t s_full[2], p_full[2], pv_done[2];
  uint64_t o_free, tail[kTails], drain;
};

__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// a shared-memory address of the pair's first CTA
__device__ __forceinline__ uint32_t in_first(uint32_t addr) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// tiled loads into this CTA, counted on a barrier of the pair's first CTA
__device__ __forceinline__ void tma2_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t mbar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
      :: "r"(dst), "l"(map), "r"(x), "r"(y), "r"(mbar) : "memory");
}
// box of columns (64 or 128, as slabs), rows, a page
__device__ __forceinline__ void tma2_load_4d(uint32_t dst, const CUtensorMap* map, int y, int slab, int z, uint32_t mbar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
      :: "r"(dst), "l"(map), "r"(0), "r"(y), "r"(slab), "r"(z), "r"(mbar) : "memory");
}
__device__ __forceinline__ void tma2_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t mbar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
      :: "r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(mbar) : "memory");
}
__device__ __forceinline__ void mma2_e(uint32_t el, uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{ .reg .pred p, e; setp.ne.b32 e, %5, 0; setp.ne.b32 p, %4, 0; "
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p; }"
      :: "r"(d_tmem), "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(el) : "memory");
}
// completion of the products so far, on this barrier of both CTAs
__device__ __forceinline__ void commit2_e(uint32_t el, uint32_t mbar) {
  asm volatile("{ .reg .pred e; setp.ne.b32 e, %1, 0; "
               "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %2; }"
               :: "r"(mbar), "r"(el), "h"((uint16_t)3) : "memory");
}
// An arrival on a barrier of the pair's first CTA.  What it announces (weights in shared memory,
// TMEM that has been read) stays in this CTA and is used by this CTA's half of a product, and
// was ordered before it by every writer's proxy or tcgen05 fence and the softmax warps' barrier;
// so the arrival need not release anything to the other CTA.  (PTX's memory model alone does not promise
// it: it rests on each CTA's half of a product being read by its own SM.)  With .release.cluster it took
// 1400 clocks and the kernel 6% longer.
__device__ __forceinline__ void arrive_first(uint32_t mbar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" :: "r"(in_first(mbar)) : "memory");
}

// ODD: d_c is an odd multiple of 128 (its tests would cost the even kernel 2.5%)
template <bool ODD>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
kda_mla_pair_kernel(const MlaArgs a, const MlaPart w, const __grid_constant__ CUtensorMap map_q,
                    const __grid_constant__ CUtensorMap map_qr, const __grid_constant__ CUtensorMap map_c, const __grid_constant__ CUtensorMap map_r,
                    const int box_rows) {
  extern __shared__ unsigned char dyn[];
  __shared__ Bars bars;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  __shared__ float row_x[4][kRows];                    // per row: the tile's maximum, or the sum, of each quarter
  const int lane = threadIdx.x & 31;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  const int rank = (int)cta_rank(), pair = blockIdx.x >> 1, n_pairs = gridDim.x >> 1;
  const int nu = a.d_c / 128;                          // units of a tile's keys, and of its values
  const bool rope = a.d_r > 0;
  const int slabs = 2 * nu + (rope ? 1 : 0);
  const uint32_t q_smem = (smem_u32(dyn) + 1023u) & ~1023u;
  const uint32_t p_smem = q_smem + slabs * kSlabBytes;
  const uint32_t k_ring = p_smem + kPBytes, v_ring = k_ring + kUnits * kUnitBytes;
  const uint32_t rope_smem = v_ring + kUnits * kUnitBytes;
  const uint32_t bb = smem_u32(&bars);
#define BAR(x) (bb + (uint32_t)offsetof(Bars, x))
#define BARI(x, i) (bb + (uint32_t)offsetof(Bars, x) + 8u * (uint32_t)(i))
  volatile int* abort = &abort_flag;

  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int i = 0; i < kUnits; ++i) {
      mbar_init(BARI(k_full, i), 1); mbar_init(BARI(k_empty, i), 1);
      mbar_init(BARI(v_full, i), 1); mbar_init(BARI(v_empty, i), 1);
    }
    mbar_init(BAR(rope_full), 1); mbar_init(BAR(rope_empty), 1);
    mbar_init(BAR(q_full), 1); mbar_init(BAR(q_empty), 1);
    for (int i = 0; i < 2; ++i) { mbar_init(BARI(s_full, i), 1); mbar_init(BARI(p_full, i), 2); mbar_init(BARI(pv_done, i), 1); }
    mbar_init(BAR(o_free), 2); mbar_init(BAR(drain), 1);
    for (int i = 0; i < kTails; ++i) mbar_init(BARI(tail, i), 1);
    mbar_init_fence();
  }
  if (warp == kSoft + 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" :: "r"(smem_u32(&tmem_slot)), "r"(kCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  fence_before();
  mla_grid_enter(w);
  MlaWalk walk = mla_plan<kThreads>(a, w, pair, n_pairs);
  cluster_sync();                                      // both CTAs' barriers stand
  fence_after();
  const uint32_t tm = __shfl_sync(0xffffffffu, *(volatile uint32_t*)&tmem_slot, 0);
  const uint32_t tm_o = tm, tm_s = tm + 256;
  MlaSeg s;

  if (warp == kSoft) {
    // ---- queries and keys --------------------------------------------------------
    uint32_t units = 0, tiles = 0;                       // sent so far
    int seg = 0;
    bool bad = false, live = true;
    const bool lead = rank == 0 && lane == 0;
    // lane (slab, box); with boxes of 64 rows one copy brings both slabs
    const int nb = 64 / box_rows, sl = lane / nb, box = lane % nb;
    const bool copies = lane < (nb == 1 ? 1 : 2 * nb);
    while (live && walk.next(a, w, s)) {
      if (seg > 0 && !wait_phase_w(BAR(q_empty), (seg - 1) & 1, abort)) break;
      if (lead) mbar_expect_tx(BAR(q_full), 2u * slabs * kSlabBytes);
      __syncwarp();
      if (lane == 0) {
        const int row = (int)(s.row0 + kRows * rank);
        tma2_load_3d(q_smem, &map_q, 0, row, 0, in_first(BAR(q_full)));
        if (rope) tma2_load_2d(q_smem + 2 * nu * kSlabBytes, &map_qr, 0, row, in_first(BAR(q_full)));
      }
      ++seg;
      for (int tile = s.tile0; tile < s.tile1; ++tile, ++tiles) {
        // this CTA's 64 tokens; boxes past the item's end come from beyond the last page,
        // that is as zeros
        const MlaTile at = mla_tile(a, w, s, tile);
        const int t = at.t0 + 64 * rank + box * box_rows;
        int z = (int)a.n_pages, y = 0;
        if (t < at.tokens) {
          const int64_t page = mla_page(a, at.b, t, &bad);
          if (page >= 0) z = (int)page;
          y = t % a.page_tokens;
        }
        for (int j = 0; j < nu; ++j, ++units) {
          const int slot = units % kUnits;
          if (units >= kUnits && !wait_phase_w(BARI(k_empty, slot), ((units / kUnits) & 1) ^ 1, abort)) { live = false; break; }
          if (lead) mbar_expect_tx(BARI(k_full, slot), 2 * kUnitBytes);
          __syncwarp();
          if (copies)
            tma2_load_4d(k_ring + slot * kUnitBytes + sl * kSlabBytes + box * box_rows * 128, &map_c, y, 2 * j + sl, z,
                         in_first(BARI(k_full, slot)));
        }
        if (live && rope) {
          if (tiles > 0 && !wait_phase_w(BAR(rope_empty), (tiles - 1) & 1, abort)) { live = false; break; }
          if (lead) mbar_expect_tx(BAR(rope_full), 2 * kSlabBytes);
          __syncwarp();
          if (lane < nb) tma2_load_3d(rope_smem + box * box_rows * 128, &map_r, a.d_c, y, z, in_first(BAR(rope_full)));
        }
        if (!live) break;
      }
    }
    if (bad) atomicOr(&g_kda_device_error, KDA_DEVERR_INDEX);
    // every copy has landed before the pair may end
    if (rank == 0) {
      if (seg > 0) mbar_wait(BAR(q_full), (seg - 1) & 1);
      for (uint32_t i = 0; i < kUnits && i < units; ++i) mbar_wait(BARI(k_full, i), ((units - 1 - i) / kUnits) & 1);
      if (rope && tiles > 0) mbar_wait(BAR(rope_full), (tiles - 1) & 1);
    }
  } else if (warp == kSoft + 1) {
    // ---- values ------------------------------------------------------------------
    uint32_t units = 0, tails = 0;                       // sent so far
    bool bad = false, live = true;
    const bool lead = rank == 0 && lane == 0;
    const int nb = 64 / box_rows, sl = lane / nb, box = lane % nb;
    const bool copies = lane < (nb == 1 ? 1 : 2 * nb);
    while (live && walk.next(a, w, s)) {
      for (int tile = s.tile0; tile < s.tile1 && live; ++tile) {
        int z0 = (int)a.n_pages, z1 = z0, y0 = 0, y1 = 0;   // of the tile's two halves
        const MlaTile at = mla_tile(a, w, s, tile);
        const int t = at.t0 + box * box_rows;
        if (t < at.tokens) {
          const int64_t page = mla_page(a, at.b, t, &bad);
          if (page >= 0) z0 = (int)page;
          y0 = t % a.page_tokens;
        }
        if (t + 64 < at.tokens) {
          const int64_t page = mla_page(a, at.b, t + 64, &bad);
          if (page >= 0) z1 = (int)page;
          y1 = (t + 64) % a.page_tokens;
        }
        // A tile that its tokens end in is cleared past them by the softmax warps first, so it
        // lands on a barrier of this CTA's own and the ring's barrier only keeps count.  The ring of
        // four units admits a tile's values only when the products with those of four tiles
        // before are done, so of four such barriers in turn each is idle when its turn comes.
        const bool tail = at.tokens - at.t0 < kTile;
        const uint32_t own = BARI(tail, tails % kTails);
        for (int j = 0; j < nu; ++j, ++units) {
          // unit 2 g + h: this CTA's 128 channels of the 256 of product g, tokens 64 h ..; an odd
          // last unit: its 64 channels of 128, and `sl` is the half of the tokens
          const bool odd = ODD && j == nu - 1;
          const int slot = units % kUnits, slab = odd ? 2 * j + rank : 4 * (j >> 1) + 2 * rank + sl;
          const int h = odd ? sl : j & 1, z = h ? z1 : z0, y = h ? y1 : y0;
          if (units >= kUnits && !wait_phase_w(BARI(v_empty, slot), ((units / kUnits) & 1) ^ 1, abort)) { live = false; break; }
          const uint32_t dst = v_ring + slot * kUnitBytes + sl * kSlabBytes + box * box_rows * 128;
          if (!tail) {
            if (lead) mbar_expect_tx(BARI(v_full, slot), 2 * kUnitBytes);
            __syncwarp();
            if (odd) {
              if (lane < 2 * nb) tma2_load_3d(dst, &map_r, 64 * slab, y, z, in_first(BARI(v_full, slot)));
            } else if (copies) {
              tma2_load_4d(dst, &map_c, y, slab, z, in_first(BARI(v_full, slot)));
            }
          } else {
            if (j == 0 && lane == 0) mbar_expect_tx(own, nu * kUnitBytes);
            if (lead) mbar_arrive(BARI(v_full, slot));
            __syncwarp();
            if (odd) {
              if (lane < 2 * nb) tma_load_3d(dst, &map_r, 64 * slab, y, z, own);
            } else if (copies) {
              tma_load_4d(dst, &map_c, y, slab, z, own);
            }
          }
        }
        if (tail) ++tails;
      }
    }
    if (bad) atomicOr(&g_kda_device_error, KDA_DEVERR_INDEX);
    for (uint32_t i = 0; i < kTails && i < tails; ++i) mbar_wait(BARI(tail, i), ((tails - 1 - i) / kTails) & 1);
    if (rank == 0)
      for (uint32_t i = 0; i < kUnits && i < units; ++i) mbar_wait(BARI(v_full, i), ((units - 1 - i) / kUnits) & 1);
    mbar_wait(BAR(drain), 0);                            // no product outlives the pair's memory: the last few tiles'
  } else if (warp == kSoft + 2) {
    // ---- products (of the first CTA, for both) -------------------------------------
    if (rank == 0) {
      constexpr uint32_t id_s = idesc_bf16(128, 128, false, false), id_o = idesc_bf16(128, 256, false, true),
                         id_o1 = idesc_bf16(128, 128, false, true);
      const uint32_t el = elect_one();
      uint32_t ku = 0, vu = 0, gt = 0;                   // units used, tiles so far
      int seg = 0, pend_seg = 0;
      bool pend = false, pend_first = false, live = true;

      auto values = [&]() -> bool {                      // O += P C of tile gt - 1 (of gt, after the last)
        const uint32_t u = gt - 1;
        const bool after = pend_first && pend_seg > 0;   // the last segment's O has been read
        // lane j < nu: unit j; nu: the weights; nu + 1: O
        const uint32_t un = vu + lane;
        const bool wants = lane <= nu || (lane == nu + 1 && after);
        const uint32_t bar = lane < nu ? BARI(v_full, un % kUnits) : lane == nu ? BARI(p_full, u & 1) : BAR(o_free);
        const uint32_t parity = lane < nu ? (un / kUnits) & 1 : lane == nu ? (u >> 1) & 1 : (pend_seg - 1) & 1;
        if (!lanes_wait<true>(wants, bar, parity, abort)) return false;
        fence_after();
        const uint32_t more = __shfl_sync(0xffffffffu, pend_first ? 0 : 1, 0);
        for (int j = 0; j < nu; ++j, ++vu) {             // product j / 2, tokens 64 (j % 2) ..
          const uint32_t base = __shfl_sync(0xffffffffu, v_ring + (vu % kUnits) * kUnitBytes, 0);
          const uint32_t d = tm_o + 128 * (j >> 1), p = p_smem + (j & 1) * kSlabBytes;
          if (ODD && j == nu - 1) {                      // the last 128 channels, all tokens
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
              mma2_e(el, d, desc_k(p_smem, kRows, ks), desc_mn(base + (ks >> 2) * kSlabBytes, 64, ks & 3), id_o1, ks == 0 ? more : 1);
          } else {
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              mma2_e(el, d, desc_k(p, kRows, ks), desc_mn(base, 64, ks), id_o, ks == 0 && (j & 1) == 0 ? more : 1);
          }
          commit2_e(el, BARI(v_empty, vu % kUnits));
        }
        commit2_e(el, BARI(pv_done, u & 1));
        pend = false;
        return true;
      };

      while (live && walk.next(a, w, s)) {
        for (int tile = s.tile0; tile < s.tile1; ++tile) {
          const bool first = tile == s.tile0;
          // lane j < nu: unit j; nu: the position slab; nu + 1: the segment's queries
          const uint32_t un = ku + lane;
          const bool wants = lane < nu || (lane == nu && rope) || (lane == nu + 1 && first);
          const uint32_t bar = lane < nu ? BARI(k_full, un % kUnits) : lane == nu ? BAR(rope_full) : BAR(q_full);
          const uint32_t parity = lane < nu ? (un / kUnits) & 1 : lane == nu ? gt & 1 : seg & 1;
          if (!lanes_wait<true>(wants, bar, parity, abort)) { live = false; break; }
          fence_after();
          const uint32_t sd = __shfl_sync(0xffffffffu, tm_s + (gt & 1) * 64, 0);
          for (int j = 0; j < nu; ++j) {
            const uint32_t base = __shfl_sync(0xffffffffu, k_ring + (ku % kUnits) * kUnitBytes, 0);
            const uint32_t qb = q_smem + 2 * j * kSlabBytes;
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
              mma2_e(el, sd, desc_k(qb, kRows, ks), desc_k(base, 64, ks), id_s, ks > 0 || j > 0);
            commit2_e(el, BARI(k_empty, ku % kUnits));
            ++ku;
          }
          if (rope) {
            const uint32_t qb = q_smem + 2 * nu * kSlabBytes;
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) mma2_e(el, sd, desc_k(qb, kRows, ks), desc_k(rope_smem, 64, ks), id_s, 1);
            commit2_e(el, BAR(rope_empty));
          }
          commit2_e(el, BARI(s_full, gt & 1));
          if (tile + 1 == s.tile1) commit2_e(el, BAR(q_empty));
          if (pend && !values()) { live = false; break; }
          pend = true;
          pend_first = first;
          pend_seg = seg;
          ++gt;
        }
        ++seg;
      }
      if (live && pend) values();
      commit2_e(el, BAR(drain));
    }
    __syncwarp();
  } else {
    // ---- softmax and results ---------------------------------------------------
    uint32_t gt = 0, tails = 0;
    bool dead = false;
    const int quarter = warp & 3, half = warp >> 2;
    const uint32_t quad = (uint32_t)quarter << 21;       // TMEM lanes 32 quarter ..
    const int row = 32 * (quarter & 1) + lane;           // this thread's row of the CTA
    const int part = quarter >> 1;                       // tokens 64 part + 32 half .. of a tile
    const uint32_t p_at = p_smem + part * kSlabBytes + row * 128;
    while (!dead && walk.next(a, w, s)) {
      const int own_lim = mla_row_limit(a, s, kRows * rank + row), pre_lim = kRows * rank + row < s.nrows ? a.prefix_len : 0;
      float m = kNone, l = 0.f;
      for (int tile = s.tile0; tile < s.tile1; ++tile, ++gt) {
        const uint32_t buf = gt & 1;
        const MlaTile tl = mla_tile(a, w, s, tile);
        const int lim = tile < s.pre ? pre_lim : own_lim, c0 = tl.t0 + 64 * part + 32 * half;
        dead |= !wait_phase(BARI(s_full, buf), (gt >> 1) & 1, abort);
        fence_after();
        float v[32];
        tmem_ld32(tm_s + buf * 64 + 32 * half + quad, v);
        if (c0 + 32 > lim) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (c0 + i >= lim) v[i] = -INFINITY;
        }
        float sum = 0.f;
        // weights against the reference as it is; the vote after them says whether a score
        // has outgrown one
        uint32_t pk[16];
        auto weights = [&]() {
          float top = -INFINITY;
          sum = 0.f;
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const float y0 = fmaf(v[i], a.scale_log2, -m), y1 = fmaf(v[i + 1], a.scale_log2, -m);
            top = fmaxf(top, fmaxf(y0, y1));
            const float p0 = ex2(y0), p1 = ex2(y1);
            sum += p0 + p1;                              // fp32 weights; the product takes them as bf16
            const __nv_bfloat162 u = __floats2bfloat162_rn(p0, p1);
            pk[i / 2] = *reinterpret_cast<const uint32_t*>(&u);
          }
          return top;
        };
        auto put = [&]() {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                         :: "r"(p_at + (uint32_t)(((4 * half + i) ^ (row & 7)) << 4)), "r"(pk[4 * i]), "r"(pk[4 * i + 1]),
                            "r"(pk[4 * i + 2]), "r"(pk[4 * i + 3]) : "memory");
        };
        const bool fresh = tile == s.tile0;              // no reference yet: to the maximum at once
        const float top = fresh ? 0.f : weights();
        if (gt >= 1) dead |= !wait_phase(BARI(pv_done, buf ^ 1), ((gt - 1) >> 1) & 1, abort);   // P's last reader
        if (!fresh) put();
        // rows of the page past the tokens' end: whatever they hold must not meet the zero
        // weights as NaN or infinity
        const int past = tl.tokens - tl.t0;
        if (past < kTile) {
          dead |= !wait_phase(BARI(tail, tails % kTails), (tails / kTails) & 1, abort);
          ++tails;
          for (int k = 0; k < 2 * nu; ++k) {             // slabs of tokens 64 h ..
            const int j = k >> 1, h = ODD && j == nu - 1 ? k & 1 : j & 1;
            const int from = max(0, past - 64 * h), clear = (64 - from) * 8;
            const uint32_t slab = v_ring + ((gt * nu + j) % kUnits) * kUnitBytes + (k & 1) * kSlabBytes + from * 128;
            for (int i = threadIdx.x; i < clear; i += 32 * kSoft)
              asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" :: "r"(slab + i * 16), "r"(0) : "memory");
          }
        }
        if (!fresh) fence_async_smem();
        fence_before();
        if (fresh || vote(top > kLazy || dead)) {
          if (!fresh && vote(dead)) { dead = true; break; }
          // some row's reference moves to the tile's maximum, and its sums with it
          float x = v[0];
#pragma unroll
          for (int i = 1; i < 32; ++i) x = fmaxf(x, v[i]);
          row_x[2 * part + half][row] = x;
          if (vote(dead)) { dead = true; break; }
          x = a.scale_log2 * fmaxf(fmaxf(row_x[0][row], row_x[1][row]), fmaxf(row_x[2][row], row_x[3][row]));
          float f = 1.f;
          bool again = false;                            // the row already has sums
          if (x > m + kLazy) { again = m != kNone; f = ex2(m - x); m = x; l *= f; }
          if (vote(again)) {
            // O holds every earlier tile of the segment: the last of them is done (waited for above,
            // after the last fence)
            fence_after();
            for (int c = 0; c < 32 * nu; c += 16) {
              float o[16];
              const uint32_t at = tm_o + half * 32 * nu + c + quad;
              tmem_ld16(at, o);
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] *= f;
              tmem_st16(at, o);
            }
          }
          weights();
          put();
          fence_async_smem();
          fence_before();
          if (vote(dead)) { dead = true; break; }
        }
        if (threadIdx.x == 0) arrive_first(BARI(p_full, buf));
        l += sum;
      }
      if (dead) break;
      // results of the segment
      dead |= !wait_phase(BARI(pv_done, (gt - 1) & 1), ((gt - 1) >> 1) & 1, abort);
      const bool whole = mla_whole(a, w, s);
      row_x[2 * part + half][row] = l;
      if (vote(dead)) { dead = true; break; }
      fence_after();
      l = (row_x[0][row] + row_x[1][row]) + (row_x[2][row] + row_x[3][row]);
      const int r = kRows * rank + row;                  // row of the item
      const int64_t slot = (s.item + pair) * w.nr + r;
      if (threadIdx.x == 0 && rank == 0) mla_note_item(w, s, pair);
      if (r < s.nrows && part == 0 && half == 0) {
        const float mr = l > 0.f ? m : -INFINITY;
        if (!whole) w.part_ml[slot] = make_float2(mr, l);
        else if (a.lse) a.lse[s.row0 + r] = 0.6931471805599453f * (mr + log2f(l));
      }
      // the channel that a column of O holds in this thread's lanes
      const auto channel = [&](int col) {
        const int g = col >> 7;
        return 256 * g + (ODD && 2 * g + 1 == nu ? 64 : 128) * part + (col & 127);
      };
      if (whole) {
        const float inv = l > 0.f ? 1.f / l : 0.f;
        for (int c = 0; c < 32 * nu; c += 16) {
          float o[16];
          const int col = half * 32 * nu + c;
          tmem_ld16(tm_o + col + quad, o);
          if (r < s.nrows) {
            __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(a.o) + (s.row0 + r) * a.d_c + channel(col);
#pragma unroll
            for (int i = 0; i < 16; i += 8) {
              const float x[8] = {o[i] * inv, o[i + 1] * inv, o[i + 2] * inv, o[i + 3] * inv,
                                  o[i + 4] * inv, o[i + 5] * inv, o[i + 6] * inv, o[i + 7] * inv};
              store8(out + i, x);
            }
          }
        }
      } else {
        // 16 lanes x 32 columns at a time: four lanes hold 32 consecutive bytes of a row, so every
        // store fills whole sectors (a thread per row writes half sectors: 7.5 us for 128 rows)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r0 = kRows * rank + 32 * (quarter & 1) + 16 * h + (lane >> 2);
          float* out = w.part_o + ((s.item + pair) * w.nr + r0) * a.d_c + 2 * (lane & 3);
          for (int c = 0; c < 32 * nu; c += 32) {
            float o[16];
            const int col = half * 32 * nu + c;
            tmem_ld_16x32(tm_o + col + quad + ((uint32_t)h << 20), o);
            float* at = out + channel(col);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (r0 < s.nrows) store2(at + 8 * i, make_float2(o[4 * i], o[4 * i + 1]));
              if (r0 + 8 < s.nrows) store2(at + 8 * a.d_c + 8 * i, make_float2(o[4 * i + 2], o[4 * i + 3]));
            }
          }
        }
      }
      fence_before();
      vote(false);                                       // all have read O, and row_x
      if (threadIdx.x == 0) arrive_first(BAR(o_free));
    }
  }
  fence_before();
  __syncthreads();                                     // which also brings each warp together
  // After a wait that gave up, the second CTA's copies may be on their way still: they count on the
  // first one's barriers, where nobody may have waited for them. They get a millisecond to land.
  if (*abort)
    for (const long long t0 = clock64(); clock64() - t0 < (1LL << 21);) {}
  cluster_sync();
  fence_after();
  if (warp == kSoft + 2) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" :: "r"(tm), "r"(kCols));
  mla_grid_leave(w);
#undef BAR
#undef BARI
}

template <bool ODD>
cudaError_t run(const MlaArgs& a, const MlaPart& w, int sms, cudaStream_t s) {
  const int64_t rows = (int64_t)a.B * a.seq_rows;
  const int box_rows = std::gcd(a.page_tokens, 64);
  CUtensorMap mq, mqr{}, mc, mr;
  if (!make_map_row_slabs(&mq, a.q, rows, a.d_c, kRows) ||
      (a.d_r > 0 && !make_map_2d(&mqr, a.q_pe, rows, a.d_r, 2, 64, kRows, true)) ||
      !make_map_slabs(&mc, a.pages, a.n_pages, a.page_bytes, a.page_tokens, a.d_c + a.d_r, a.d_c / 64, box_rows,
                      box_rows == 64 ? 2 : 1) ||
      !make_map_pages(&mr, a.pages, a.n_pages, a.page_bytes, a.page_tokens, a.d_c + a.d_r, 64, box_rows))
    return cudaErrorInvalidValue;
  const int smem = smem_bytes(2 * (a.d_c / 128) + (a.d_r > 0));
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = mla_allow_smem(kda_mla_pair_kernel<ODD>, smem_bytes(9), allowed);
  if (e != cudaSuccess) return e;
  return mla_launch(kda_mla_pair_kernel<ODD>, sms / 2 * 2, kThreads, smem, s, a, w, mq, mqr, mc, mr, box_rows);
}

}  // namespace

cudaError_t launch_mla_pair(const MlaArgs& a, const MlaPart& w, int sms, cudaStream_t s) {
  return a.d_c % 256 ? run<true>(a, w, sms, s) : run<false>(a, w, sms, s);
}

int read_and_clear_mla_pair_errors(int* flags) {
  int word = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&word, g_kda_device_error, sizeof(int));
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_kda_device_error, &zero, sizeof(int));
  *flags |= word;
  return (int)e;
}

}  // namespace kda
