// bf16 attention over the latent page cache on the tensor cores (kda_mla.cuh has the
// division of work, kda_mla_decode.cu the formulas and the merge).
//
// One CTA per SM walks its piece of the line of tiles.  An item is NR query rows (the
// heads and draft positions that read the same tokens); a tile is 64 tokens, staged
// once by TMA as column slabs [64 tokens][64 values] and used twice, since c is both
// key and value:
//   S^T = K Q^T      M = 64 tokens, N = NR rows, K = d_c + d_r;
//   O^T += C^T P^T   M = 128 channels, N = NR rows, K = 64 tokens: the slabs, read MN-major.
// Rows are columns of both accumulators, so the products cost what the live rows need (the
// other orientation pads them to 64 or 128, and O would take all 512 TMEM columns at
// 64 rows); O^T takes NR d_c / 128 columns.
// Warps 0-7 do the softmax and write results: warps w and w + 4 share 16 tokens of S^T (a
// quarter of the TMEM lanes) and take half of the rows each; a thread of a 16x256b TMEM
// load holds 2 tokens of NR / 8 rows, and stmatrix writes the weights transposed, as P.
// Warp 8 issues the copies, warp 9 the products.  S^T is double-buffered: that of the next
// tile runs during the softmax of this one when its slabs have arrived in time; when they
// have not, O^T of this tile goes first so that its slabs are free for the copies.
//
// The running reference m of a row moves only when the maximum rises more than 2^8
// above it (weights then stay below 2^8, far inside bf16's and fp32's range), so O in
// TMEM is rescaled rarely.
//
// Both operands of O's products are bf16, so the weights are rounded to it (their sum, and so lse, is
// of the fp32 weights): against fp64, o is off by 1.7e-3 to 2.1e-3 of its size instead of the 1.66e-3 of
// its own rounding.  tf32 products of fp32 weights would need the values as fp32 in shared memory, twice the
// bytes of what bounds the kernels.
//
// Bound by HBM up to 32 rows (256 sequences of 512-8192 tokens, 32 heads, d_c = 512,
// d_r = 64: 148 us, 5.7 TB/s, 84% of the measured copy rate); at 64 rows by shared-memory bandwidth
// (operands and copies: 2500 clocks per tile, the products' own rate 1088).
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

constexpr int kSoft = kMlaSoft;        // softmax warps, two per quarter of the TMEM lanes
constexpr int kThreads = 32 * (kSoft + 2);
constexpr int kTile = 64;
constexpr int kPairBytes = 16384;      // two column slabs: [64 tokens][64 values] each
constexpr int kSlabBytes = 8192;

template <int NR> struct Cfg {
  static constexpr int kPBytes = NR * 128;
  static constexpr int kPBufs = NR == 64 ? 1 : 2;    // P tiles: at 64 rows the second's room goes to a position slab
  static constexpr int kPairs = NR == 64 ? 8 : NR == 32 ? 10 : 11;   // ring of slab pairs
  static constexpr int kRopes = 2;                   // ring of position slabs
  static constexpr int smem(int slabs) {             // Q slabs, P tiles, the rings
    return 1024 + slabs * NR * 128 + kPBufs * kPBytes + kPairs * kPairBytes + kRopes * kSlabBytes;
  }
  static_assert(smem(9) + 2048 <= 232448, "2 KB are left for the static shared memory");
  static constexpr uint32_t kCols = NR == 64 ? 512 : NR == 32 ? 256 : 128;   // TMEM: 4 NR of O^T, 2 NR of S^T
};

struct Bars {
  uint64_t pair_full[11], pair_empty[11];
  uint64_t rope_full[2], rope_empty[2];
  uint64_t q_full, q_empty;
  uint64_t s_full[2], p_full[2], pv_done[2];
  uint64_t o_free, drain;
};

// 16 lanes x 8 n columns: v[4 i + c] of a thread is lane / 4 + 8 (c / 2) and column
// 8 i + 2 (lane % 4) + c % 2
__device__ __forceinline__ void tmem_ld_16x8n(uint32_t taddr, float (&v)[4]) {
  uint32_t r[4];
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0,%1,%2,%3}, [%4];\n\ttcgen05.wait::ld.sync.aligned;"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(taddr) : "memory");
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_ld_16x8n(uint32_t taddr, float (&v)[8]) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\ttcgen05.wait::ld.sync.aligned;"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr) : "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_ld_16x8n(uint32_t taddr, float (&v)[16]) { tmem_ld_16x32(taddr, v); }
// 32 lanes x 8 or 16 columns, and back
__device__ __forceinline__ void tmem_ldn(uint32_t taddr, float (&v)[8]) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\ttcgen05.wait::ld.sync.aligned;"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr) : "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_ldn(uint32_t taddr, float (&v)[16]) { tmem_ld16(taddr, v); }
__device__ __forceinline__ void tmem_stn(uint32_t taddr, const float (&v)[8]) {
  uint32_t r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = __float_as_uint(v[i]);
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n\ttcgen05.wait::st.sync.aligned;"
               :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_stn(uint32_t taddr, const float (&v)[16]) { tmem_st16(taddr, v); }
// two 8 x 8 blocks of bf16, each stored transposed: lane i < 16 gives the address of row
// i % 8 of block i / 8
__device__ __forceinline__ void stmatrix2_t(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("stmatrix.sync.aligned.m8n8.x2.trans.shared.b16 [%0], {%1, %2};" :: "r"(addr), "r"(a), "r"(b) : "memory");
}

template <int NR>
__global__ void __launch_bounds__(kThreads, 1)
kda_mla_tc_kernel(const MlaArgs a, const MlaPart w, const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_qr,
                  const __grid_constant__ CUtensorMap map_c, const __grid_constant__ CUtensorMap map_r, const int box_rows) {
  using C = Cfg<NR>;
  extern __shared__ unsigned char dyn[];
  __shared__ Bars bars;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  // per row: the tile's maximum, or the sum, of each quarter; the rescale factor, or 1 / l
  __shared__ float row_x[4][NR], row_f[NR];
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
      mbar_init(BARI(s_full, i), 1); mbar_init(BARI(p_full, i), 1); mbar_init(BARI(pv_done, i), 1);
    }
    mbar_init(BAR(q_full), 1); mbar_init(BAR(q_empty), 1); mbar_init(BAR(o_free), 1); mbar_init(BAR(drain), 1);
    mbar_init_fence();
  }
  if (warp == kSoft + 1) tmem_alloc(smem_u32(&tmem_slot), C::kCols);
  fence_before();
  mla_grid_enter(w);
  MlaWalk walk = mla_plan<kThreads>(a, w, blockIdx.x, gridDim.x);   // ends in a block barrier
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
    // lane (slab, box); with boxes of 64 rows one copy brings both slabs
    const int nbox = kTile / box_rows, sl = lane / nbox, box = lane % nbox;
    const bool copies = lane < (nbox == 1 ? 1 : 2 * nbox);
    while (live && walk.next(a, w, s)) {
      if (seg > 0 && !wait_phase_w(BAR(q_empty), (seg - 1) & 1, abort)) break;
      if (lane == 0) {
        mbar_expect_tx(BAR(q_full), (uint32_t)slabs * NR * 128);
        tma_load_3d(q_smem, &map_q, 0, (int)s.row0, 0, BAR(q_full));
        if (rope) tma_load_2d(q_smem + 2 * np * NR * 128, &map_qr, 0, (int)s.row0, BAR(q_full));
      }
      ++seg;
      for (int tile = s.tile0; tile < s.tile1; ++tile) {
        // boxes past the item's tokens come from beyond the last page, that is as zeros
        const int t = tile * kTile + box * box_rows;
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
          if (copies)
            tma_load_4d(pair_smem + pr.slot * kPairBytes + sl * kSlabBytes + box * box_rows * 128, &map_c, y, 2 * j + sl, z, bar);
          pr.step(C::kPairs);
          ++pairs_sent;
        }
        if (!live) break;
        if (rope) {
          if (ropes_sent >= C::kRopes && !wait_phase_w(BARI(rope_empty, rr.slot), rr.phase ^ 1, abort)) { live = false; break; }
          const uint32_t bar = BARI(rope_full, rr.slot);
          if (lane == 0) mbar_expect_tx(bar, kSlabBytes);
          __syncwarp();
          if (sl == 0) tma_load_3d(rope_smem + rr.slot * kSlabBytes + box * box_rows * 128, &map_r, a.d_c, y, z, bar);
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
    // The whole warp runs this, one elected lane issues, and the lanes test the barriers of a
    // tile's slabs side by side: operand descriptors then stay in uniform registers and the
    // products follow one another without a wait (36 of them with a wait and an election
    // each took 1960 clocks to issue and ~1150 to run).
    constexpr uint32_t id_s = idesc_bf16(64, NR, false, false), id_o = idesc_bf16(128, NR, true, false);
    const uint32_t el = elect_one();
    int kslot = 0, vslot = 0;                            // first pair of the next tile as keys, as values
    uint32_t kphase = 0, gt = 0;                         // tiles so far
    int seg = 0, pend_seg = 0;
    bool pend = false, pend_first = false, live = true;

    auto values = [&]() -> bool {                        // O^T += C^T P^T of tile gt - 1
      const uint32_t u = gt - 1;
      const bool after = pend_first && pend_seg > 0;     // the last segment's O has been read
      if (!lanes_wait(lane == 0 || (lane == 1 && after), lane == 0 ? BARI(p_full, u & 1) : BAR(o_free),
                      lane == 0 ? (u >> 1) & 1 : (pend_seg - 1) & 1, abort))
        return false;
      fence_after();
      const uint32_t pb = p_smem + (u % C::kPBufs) * C::kPBytes;
      const uint32_t more = pend_first ? 0 : 1;
      for (int j = 0; j < np; ++j) {
        const uint32_t vd = desc_lo_mn(pair_smem + vslot * kPairBytes), pd = desc_lo_k(pb);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)                   // 16 tokens on: 2 KB of values, 32 bytes of weights
          mma_e(el, tm_o + j * NR, vd + ks * 128, pd + ks * 2, id_o, ks == 0 ? more : 1);
        commit_e(el, BARI(pair_empty, vslot));
        if (++vslot == C::kPairs) vslot = 0;
      }
      commit_e(el, BARI(pv_done, u & 1));
      pend = false;
      return true;
    };

    while (live && __shfl_sync(0xffffffffu, walk.next(a, w, s), 0)) {
      const int tile0 = __shfl_sync(0xffffffffu, s.tile0, 0), tile1 = __shfl_sync(0xffffffffu, s.tile1, 0);
      for (int tile = tile0; tile < tile1; ++tile) {
        const bool first = tile == tile0;
        // lane j < np: pair j; np: the position slab; np + 1: the segment's queries
        const int slot = kslot + lane, wrap = slot >= C::kPairs;
        const bool wants = lane < np || (lane == np && rope) || (lane == np + 1 && first);
        const uint32_t bar = lane < np ? BARI(pair_full, wrap ? slot - C::kPairs : slot)
                             : lane == np ? BARI(rope_full, gt % C::kRopes) : BAR(q_full);
        const uint32_t parity = lane < np ? kphase ^ wrap : lane == np ? (gt / C::kRopes) & 1 : seg & 1;
        if (pend) {
          // Whichever is ready first: the keys of this tile, or the weights of the last one (the
          // values go first when the keys are late, which also frees their slabs)
          const bool after = pend_first && pend_seg > 0;
          const uint32_t v = gt - 1;
          const uint32_t pbar = lane == 16 ? BARI(p_full, v & 1) : lane == 17 && after ? BAR(o_free) : bar;
          const uint32_t ppar = lane == 16 ? (v >> 1) & 1 : lane == 17 && after ? (pend_seg - 1) & 1 : parity;
          const uint32_t keys = __ballot_sync(0xffffffffu, wants), weights = 0x10000u | (after ? 0x20000u : 0u);
          const long long t0 = clock64();
          for (int i = 1;; ++i) {
            const uint32_t done = lanes_poll(wants || lane >= 16 ? pbar : BARI(p_full, v & 1), ppar);
            if ((done & keys) == keys) break;
            if ((done & weights) == weights) {
              if (!values()) live = false;
              break;
            }
            if (i % 256 == 0 && __any_sync(0xffffffffu, *abort || clock64() - t0 > (1LL << 31))) {
              if (*abort == 0) atomicOr(&g_kda_device_error, kDevErrWait);
              *abort = 1;
              live = false;
              break;
            }
          }
          if (!live) break;
        }
        if (!lanes_wait(wants, bar, parity, abort)) { live = false; break; }
        fence_after();
        const uint32_t sd = tm_s + (gt & 1) * NR;
        for (int j = 0; j < np; ++j) {
          const uint32_t kd = desc_lo_k(pair_smem + kslot * kPairBytes), qd = desc_lo_k(q_smem + 2 * j * NR * 128);
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)                 // 16 values on: 32 bytes in a slab, or the next slab
            mma_e(el, sd, kd + (ks & 3) * 2 + (ks >> 2) * (kSlabBytes >> 4), qd + (ks & 3) * 2 + (ks >> 2) * (NR * 128 >> 4), id_s,
                  ks > 0 || j > 0);
          if (++kslot == C::kPairs) { kslot = 0; kphase ^= 1; }
        }
        if (rope) {
          const uint32_t kd = desc_lo_k(rope_smem + (gt % C::kRopes) * kSlabBytes), qd = desc_lo_k(q_smem + 2 * np * NR * 128);
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) mma_e(el, sd, kd + ks * 2, qd + ks * 2, id_s, 1);
        }
        commit_e(el, BARI(s_full, gt & 1));
        if (rope) commit_e(el, BARI(rope_empty, gt % C::kRopes));
        if (tile + 1 == tile1) commit_e(el, BAR(q_empty));
        if (pend && !values()) { live = false; break; }
        pend = true;
        pend_first = first;
        pend_seg = seg;
        ++gt;
      }
      ++seg;
    }
    if (live && pend) values();
    commit_e(el, BAR(drain));                            // no product outlives the CTA's memory
    mbar_wait(BAR(drain), 0);
    __syncwarp();
  } else {
    // ---- softmax and results ---------------------------------------------------
    constexpr int NI = NR / 16;                          // blocks of 8 rows per warp
    constexpr int NC = NR / 2 < 16 ? NR / 2 : 16;        // columns of O^T per TMEM access
    uint32_t gt = 0;
    bool dead = false;
    int vslot = 0;                                       // first pair of the tile
    const int quarter = warp & 3, half = warp >> 2;
    const uint32_t quad = (uint32_t)quarter << 21;       // TMEM lanes 32 quarter ..
    const int tok = 16 * quarter + (lane >> 2);          // this thread's tokens of a tile: tok and tok + 8
    const int col0 = half * (NR / 2) + 2 * (lane & 3);   // its rows: col0 + 8 i + e, i < NI, e < 2
    // stmatrix: P is [NR rows][64 tokens], 128-byte swizzle
    const int srow = half * (NR / 2) + (lane & 7), schunk = 2 * quarter + ((lane >> 3) & 1);
    const uint32_t p_at = p_smem + srow * 128 + (uint32_t)((schunk ^ (lane & 7)) << 4);
    while (!dead && walk.next(a, w, s)) {
      int lim[NI][2], lim_min = s.tokens;
      float m[NI][2], l[NI][2];
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          lim[i][e] = mla_row_limit(a, s, col0 + 8 * i + e);
          lim_min = min(lim_min, lim[i][e]);
          m[i][e] = kNone;
          l[i][e] = 0.f;
        }
      for (int tile = s.tile0; tile < s.tile1; ++tile, ++gt) {
        const uint32_t buf = gt & 1;
        const int t0 = tile * kTile;
        dead |= !wait_phase(BARI(s_full, buf), (gt >> 1) & 1, abort);
        fence_after();
        float v[4 * NI], p[4 * NI];                      // [i][token][e]
        const uint32_t pb = p_at + (gt % C::kPBufs) * C::kPBytes;
        tmem_ld_16x8n(tm_s + buf * NR + half * (NR / 2) + quad, v);
        if (t0 + kTile > lim_min) {
#pragma unroll
          for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (t0 + tok + 8 * (c >> 1) >= lim[i][c & 1]) v[4 * i + c] = -INFINITY;
        }
        // weights against the references as they are, written at once; the vote after it says
        // whether a score has outgrown one
        auto weights = [&]() {
          float top = -INFINITY;
#pragma unroll
          for (int i = 0; i < NI; ++i) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const float y = fmaf(v[4 * i + c], a.scale_log2, -m[i][c & 1]);
              top = fmaxf(top, y);
              p[4 * i + c] = ex2(y);
            }
            const __nv_bfloat162 u = __floats2bfloat162_rn(p[4 * i], p[4 * i + 1]);
            const __nv_bfloat162 x = __floats2bfloat162_rn(p[4 * i + 2], p[4 * i + 3]);
            stmatrix2_t(pb + i * 1024, *reinterpret_cast<const uint32_t*>(&u), *reinterpret_cast<const uint32_t*>(&x));
          }
          return top;
        };
        if (gt >= C::kPBufs) {                           // the P tile's last reader
          const uint32_t u = gt - C::kPBufs;
          dead |= !wait_phase(BARI(pv_done, u & 1), (u >> 1) & 1, abort);
        }
        const bool fresh = tile == s.tile0;              // no references yet: to the maxima at once
        const float top = fresh ? 0.f : weights();
        // the tile's tokens past the item's end: whatever the page holds there must not
        // meet the zero weights as NaN or infinity
        const int past = s.tokens - t0;
        if (past < kTile) {
          for (int j = 0; j < np; ++j) {
            const int slot = vslot + j >= C::kPairs ? vslot + j - C::kPairs : vslot + j;
            const uint32_t slab = pair_smem + slot * kPairBytes + half * kSlabBytes;   // a slab per four warps
            for (int i = past * 128 + (threadIdx.x & 127) * 16; i < kSlabBytes; i += 128 * 16)
              asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" :: "r"(slab + i), "r"(0) : "memory");
          }
        }
        vslot += np;
        if (vslot >= C::kPairs) vslot -= C::kPairs;
        if (!fresh) fence_async_smem();
        fence_before();
        if (fresh || vote(top > kLazy || dead)) {
          if (!fresh && vote(dead)) { dead = true; break; }
          // some row's reference moves to the tile's maximum, and its sums with it
#pragma unroll
          for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float x = fmaxf(v[4 * i + e], v[4 * i + 2 + e]);
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
              if (lane < 4) row_x[quarter][col0 + 8 * i + e] = x;
            }
          if (vote(dead)) { dead = true; break; }
          bool again = false;                            // a row that already has sums
#pragma unroll
          for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int r = col0 + 8 * i + e;
              const float x = a.scale_log2 * fmaxf(fmaxf(row_x[0][r], row_x[1][r]), fmaxf(row_x[2][r], row_x[3][r]));
              float f = 1.f;
              if (x > m[i][e] + kLazy) { again |= m[i][e] != kNone; f = ex2(m[i][e] - x); m[i][e] = x; }
              l[i][e] *= f;
              if (quarter == 0 && lane < 4) row_f[r] = f;
            }
          if (vote(again)) {
            // O^T holds every earlier tile of the segment once the last of them is done
            dead |= !wait_phase(BARI(pv_done, buf ^ 1), ((gt - 1) >> 1) & 1, abort);
            fence_after();
            for (int j = 0; j < np; ++j)
#pragma unroll
              for (int c = 0; c < NR / 2; c += NC) {
                float o[NC];
                const int col = half * (NR / 2) + c;
                const uint32_t at = tm_o + j * NR + col + quad;
                tmem_ldn(at, o);
#pragma unroll
                for (int i = 0; i < NC; ++i) o[i] *= row_f[col + i];
                tmem_stn(at, o);
              }
          }
          weights();
          fence_async_smem();
          fence_before();
          if (vote(dead)) { dead = true; break; }
        }
        if (threadIdx.x == 0) mbar_arrive(BARI(p_full, buf));
#pragma unroll
        for (int i = 0; i < NI; ++i) {                   // sums of the fp32 weights
          l[i][0] += p[4 * i] + p[4 * i + 2];
          l[i][1] += p[4 * i + 1] + p[4 * i + 3];
        }
      }
      if (dead) break;
      // results of the segment
      const bool whole = mla_whole(a, w, s);
      const int64_t slot = (s.item + blockIdx.x) * w.nr;
      if (threadIdx.x == 0) mla_note_item(w, s, blockIdx.x);
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) l[i][e] += __shfl_xor_sync(0xffffffffu, l[i][e], o);
          if (lane < 4) row_x[quarter][col0 + 8 * i + e] = l[i][e];
        }
      vote(false);                                       // all sums are there; every use of row_f is over
      if (quarter == 0 && lane < 4) {
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = col0 + 8 * i + e;
            const float lr = (row_x[0][r] + row_x[1][r]) + (row_x[2][r] + row_x[3][r]);
            const float mr = lr > 0.f ? m[i][e] : -INFINITY;
            row_f[r] = lr > 0.f ? 1.f / lr : 0.f;
            if (r < s.nrows) {
              if (!whole) w.part_ml[slot + r] = make_float2(mr, lr);
              else if (a.lse) a.lse[s.row0 + r] = 0.6931471805599453f * (mr + log2f(lr));
            }
          }
      }
      dead |= !wait_phase(BARI(pv_done, (gt - 1) & 1), ((gt - 1) >> 1) & 1, abort);
      if (vote(dead)) { dead = true; break; }
      fence_after();
      for (int j = 0; j < np; ++j)
#pragma unroll
        for (int c = 0; c < NR / 2; c += NC) {
          float o[NC];
          const int col = half * (NR / 2) + c, e = 128 * j + 32 * quarter + lane;
          tmem_ldn(tm_o + j * NR + col + quad, o);
          if (whole) {
            __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(a.o) + (s.row0 + col) * a.d_c + e;
#pragma unroll
            for (int i = 0; i < NC; ++i, out += a.d_c)
              if (col + i < s.nrows) *out = __float2bfloat16_rn(o[i] * row_f[col + i]);
          } else {
            float* out = w.part_o + (slot + col) * a.d_c + e;
#pragma unroll
            for (int i = 0; i < NC; ++i, out += a.d_c)
              if (col + i < s.nrows) *out = o[i];
          }
        }
      fence_before();
      vote(false);                                       // all have read O^T, row_x and row_f
      if (threadIdx.x == 0) mbar_arrive(BAR(o_free));
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == kSoft + 1) tmem_dealloc(tm, C::kCols);
  mla_grid_leave(w);
#undef BAR
#undef BARI
}

template <int NR>
cudaError_t run(const MlaArgs& a, const MlaPart& w, int ctas, cudaStream_t s) {
  const int64_t rows = (int64_t)a.B * a.seq_rows;
  const int box_rows = std::gcd(a.page_tokens, kTile);
  CUtensorMap mq, mqr{}, mc, mr;
  if (!make_map_row_slabs(&mq, a.q, rows, a.d_c, NR) ||
      (a.d_r > 0 && !make_map_2d(&mqr, a.q_pe, rows, a.d_r, 2, 64, NR, true)) ||
      !make_map_slabs(&mc, a.pages, a.n_pages, a.page_bytes, a.page_tokens, a.d_c + a.d_r, a.d_c / 64, box_rows,
                      box_rows == 64 ? 2 : 1) ||
      !make_map_pages(&mr, a.pages, a.n_pages, a.page_bytes, a.page_tokens, a.d_c + a.d_r, 64, box_rows))
    return cudaErrorInvalidValue;
  const int smem = Cfg<NR>::smem(2 * (a.d_c / 128) + (a.d_r > 0));
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = mla_allow_smem(kda_mla_tc_kernel<NR>, Cfg<NR>::smem(9), allowed);
  if (e != cudaSuccess) return e;
  return mla_launch(kda_mla_tc_kernel<NR>, ctas, kThreads, smem, s, a, w, mq, mqr, mc, mr, box_rows);
}

}  // namespace

cudaError_t launch_mla_tc(const MlaArgs& a, const MlaPart& w, int sms, cudaStream_t s) {
  return w.nr == 16 ? run<16>(a, w, sms, s) : w.nr == 32 ? run<32>(a, w, sms, s) : run<64>(a, w, sms, s);
}

int read_and_clear_mla_tc_errors(int* flags) {
  int word = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&word, g_kda_device_error, sizeof(int));
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_kda_device_error, &zero, sizeof(int));
  *flags |= word;
  return (int)e;
}

}  // namespace kda
