// The latent page cache (MLA_KV pages): arguments of its kernels, the division of
// attention work among CTAs, and the form of partial results.
//
// The work of a call is one or two parts (MlaPart), each one launch: the prefix and the
// sequences' own tokens go to the kernel that suits their rows.  In a part, work is
// counted in tiles of tokens.  An item is a tile of at most `nr` query rows with the
// tokens they attend to: first the rows of the whole batch, nr at a time, against the
// shared prefix; then, sequence by sequence, the sequence's rows against its own tokens.
// The tiles of all items in order, and before each item's tiles a few units for what an item
// costs besides them (its queries' load, its results), form one line that is cut into
// equal pieces, one per worker (a CTA, or a pair of them), so ragged lengths and few long
// sequences fill the GPU alike.  Where a sequence's rows fill items of their own, the prefix
// needs no items: a joint part's items hold a sequence's rows with the prefix's tiles and
// then its own, which leaves one result per row instead of two.  A piece may end inside an item: every (worker, item) pair that meets leaves
// a partial result in slot worker + item (both only ever grow along the line, so slots
// are distinct), and the merge kernel joins the slots of each row.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

namespace kda {

constexpr int kSms = 152;             // of a GB300: grids of the norms and divisions of linear attention's work go by it
constexpr int kMlaMaxTokens = 0x7fffff00;   // positions and a tile past them fit an int
constexpr int kMlaMaxCtas = 192;      // bound on the workers of a part (workspace size)

struct MlaAppendArgs {
  unsigned char* pages;               // [n_pages][page_bytes]
  int64_t page_bytes, n_pages;
  int page_tokens;
  const int32_t *slots, *positions;   // [T]
  const float* rope;                  // [n_pos][d_r]: cos | sin
  int n_pos;
  const void *c, *k_pe, *norm_weight; // rows c_stride, k_pe_stride elements apart; [d_c] or nullptr
  int64_t c_stride, k_pe_stride;
  const void* q_pe;                   // or nullptr
  int64_t q_stride_t, q_stride_h;
  void* q_pe_out;                     // [T][H][d_r]
  float eps;
  int T, H, d_c, d_r, dtype, style;
};
cudaError_t launch_mla_append(const MlaAppendArgs& a, cudaStream_t s);
int read_and_clear_mla_append_errors(int* flags);

struct MlaArgs {
  const void *q, *q_pe;               // [B][n_q][H][d_c], [B][n_q][H][d_r]
  const unsigned char* pages;
  int64_t page_bytes, n_pages;
  int page_tokens;
  const int32_t* prefix_pages;
  int prefix_len;
  const int32_t* page_table;          // [B][max_pages]
  int64_t max_pages;
  const int32_t* lens;                // [B]
  float scale_log2;                   // scale * log2(e): scores and statistics are in log2 units
  void* o;                            // [B][n_q][H][d_c]
  float* lse;                         // [B][n_q][H] or nullptr
  int B, n_q, H, d_c, d_r, dtype;
  int seq_rows;                       // n_q * H
};
struct MlaPart {
  int kernel;                         // kMlaSimt, kMlaTc, kMlaPair
  int nr, tile;                       // rows per item, tokens per tile
  int prefix_cost, own_cost;          // units of an item besides its tiles
  int row_tiles;                      // items per sequence (0: own tokens are not this part's)
  int prefix_items, prefix_tiles;     // items and tiles per item of the prefix (0: not this part's)
  int joint;                          // 1: no prefix items; every own item begins with the prefix's tiles
  float* part_o;                      // [slots][nr][d_c], not yet divided by l
  float2* part_ml;                    // [slots][nr]: reference m (log2 units), sum l
  int2* item_ctas;                    // [items]: first and last worker that met the item
  int64_t own_items;
  int second;                         // 1: follows another part of the call, whose results it does not read
  int64_t items() const { return prefix_items + own_items; }
};
enum { kMlaSimt, kMlaTc, kMlaPair };
// The parts of a call (one or two; sizes only, no pointers).
int mla_parts(int B, int seq_rows, int64_t prefix_len, int dtype, MlaPart (&parts)[2]);
cudaError_t launch_mla_decode(const MlaArgs& a, const MlaPart* parts, int n, cudaStream_t s);
int read_and_clear_mla_errors(int* flags);
// The bf16 kernels: one CTA per item (kda_mla_tc.cu), a pair of CTAs (kda_mla_pair.cu).
cudaError_t launch_mla_tc(const MlaArgs& a, const MlaPart& w, int sms, cudaStream_t s);
int read_and_clear_mla_tc_errors(int* flags);
cudaError_t launch_mla_pair(const MlaArgs& a, const MlaPart& w, int sms, cudaStream_t s);
int read_and_clear_mla_pair_errors(int* flags);

#ifdef __CUDACC__

// Launch as a programmatic dependent of the preceding kernel on an eager stream, so that its
// launch and set-up overlap that kernel's end; inside a stream capture the plain launch is kept
// (replayed graphs pipeline their kernel nodes better without it).
template <typename Kern, typename... Args>
inline cudaError_t mla_launch(Kern kern, dim3 grid, dim3 block, size_t smem, cudaStream_t s, const Args&... args) {
  cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(s, &cap) != cudaSuccess) {
    cudaGetLastError();
    cap = cudaStreamCaptureStatusActive;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cap == cudaStreamCaptureStatusNone ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
  return e != cudaSuccess ? e : cudaGetLastError();
}
// Allow a kernel its largest dynamic shared memory, once per device.
template <typename Kern>
inline cudaError_t mla_allow_smem(Kern kern, int bytes, std::atomic<uint64_t>& devices) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  const uint64_t bit = 1ull << (dev & 63);
  if (e != cudaSuccess || (dev < 64 && (devices.load(std::memory_order_relaxed) & bit))) return e;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) devices.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// The kernels' side of it.  A first part waits for the preceding kernel before it touches
// memory; a second part need not wait for the first, but ends only after it, since the merge
// waits for the second alone.  The first lets the second in only once its own wait is over, so
// what came before the call is complete for both.
__device__ __forceinline__ void mla_grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void mla_grid_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void mla_grid_enter(const MlaPart& w) {
  if (!w.second) mla_grid_wait();
  mla_grid_next();
}
__device__ __forceinline__ void mla_grid_leave(const MlaPart& w) {
  if (w.second) mla_grid_wait();
}

// tokens of sequence b's own pages (0 for a padded row)
__device__ __forceinline__ int mla_own_tokens(const MlaArgs& a, int b) {
  const int64_t room = min(a.max_pages * a.page_tokens, (int64_t)kMlaMaxTokens);
  const int n = max(0, a.lens[b]);
  return (int)min((int64_t)n, room);
}
__device__ __forceinline__ int mla_tiles(const MlaPart& w, int tokens) { return tokens / w.tile + (tokens % w.tile != 0); }
// tiles of sequence b's items, and their units on the line (0: nothing to attend to)
__device__ __forceinline__ int mla_seq_tiles(const MlaArgs& a, const MlaPart& w, int b) {
  const int pre = w.joint && a.lens[b] >= 0 ? w.prefix_tiles : 0;
  return pre + mla_tiles(w, mla_own_tokens(a, b));
}
__device__ __forceinline__ int mla_seq_units(const MlaArgs& a, const MlaPart& w, int b) {
  const int n = mla_seq_tiles(a, w, b);
  return n ? n + w.own_cost : 0;
}

// One (worker, item) meeting: tiles [tile0, tile1) of an item of `tokens` tokens.
struct MlaSeg {
  int64_t item;
  int64_t row0;          // first row of the item among all B * n_q * H rows
  int nrows;             // live rows of the item (<= nr)
  int b;                 // sequence, or -1: the prefix
  int j0;                // row0's index within its sequence (own items)
  int pre;               // leading tiles that are the prefix's (joint items)
  int tokens, tile0, tile1, tiles;   // tokens: of the tiles after those
};

// Where a tile's tokens are: those of sequence b (-1: the prefix) from t0, of `tokens` in all.
struct MlaTile {
  int b, t0, tokens;
};

// Where a worker's piece of the line starts, and the walk along it.
struct MlaWalk {
  int64_t left;          // units of the piece not yet handed out
  int prefix_item;       // next prefix item; own items follow prefix_items
  int b, r, unit;        // next own item; units of the next item that lie before the piece

  __device__ __forceinline__ bool next(const MlaArgs& a, const MlaPart& w, MlaSeg& s) {
    do {
      if (left <= 0) return false;
      if (prefix_item < w.prefix_items) {
        s.item = prefix_item;
        s.row0 = (int64_t)prefix_item * w.nr;
        s.nrows = (int)min((int64_t)w.nr, (int64_t)a.B * a.seq_rows - s.row0);
        s.b = -1;
        s.j0 = 0;
        s.pre = 0;
        s.tokens = a.prefix_len;
        s.tiles = w.prefix_tiles;
      } else {
        int n = mla_seq_tiles(a, w, b);
        while (n == 0) {
          if (++b >= a.B) return false;
          n = mla_seq_tiles(a, w, b);
        }
        s.item = w.prefix_items + (int64_t)b * w.row_tiles + r;
        s.j0 = r * w.nr;
        s.row0 = (int64_t)b * a.seq_rows + s.j0;
        s.nrows = min(w.nr, a.seq_rows - s.j0);
        s.b = b;
        s.pre = w.joint ? w.prefix_tiles : 0;
        s.tokens = mla_own_tokens(a, b);
        s.tiles = n;
      }
      const int cost = s.b < 0 ? w.prefix_cost : w.own_cost;
      const int units = s.tiles + cost, end = (int)min((int64_t)units, unit + left);
      s.tile0 = max(0, unit - cost);
      s.tile1 = max(0, end - cost);
      left -= end - unit;
      unit = end;
      if (unit == units) {
        unit = 0;
        if (s.b < 0) {
          ++prefix_item;
        } else if (++r == w.row_tiles) {
          r = 0;
          if (++b >= a.B) left = 0;
        }
      }
    } while (s.tile0 == s.tile1);      // the piece ends before the item's first tile
    return true;
  }
};

// The piece of worker `cta` of `n_ctas`: all NT threads of the block call it.  Each
// thread adds up the units of a run of sequences, a block scan places the runs, and
// the thread whose run holds the piece's first unit walks to it.
template <int NT>
__device__ __forceinline__ MlaWalk mla_plan(const MlaArgs& a, const MlaPart& w, int cta, int n_ctas) {
  static_assert(NT % 32 == 0 && NT <= 1024, "whole warps");
  __shared__ int64_t warp_sum[NT / 32];
  __shared__ MlaWalk found;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n_seqs = w.row_tiles > 0 ? a.B : 0;
  const int per = (n_seqs + NT - 1) / NT;
  const int lo = min(n_seqs, tid * per), hi = min(n_seqs, lo + per);
  int64_t mine = 0;
  for (int b = lo; b < hi; ++b) mine += (int64_t)mla_seq_units(a, w, b) * w.row_tiles;
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t up = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += up;
  }
  if (lane == 31) warp_sum[warp] = incl;
  if (tid == 0) found.left = 0;
  __syncthreads();
  const int prefix_units = w.prefix_tiles + w.prefix_cost;
  const int64_t prefix_total = (int64_t)w.prefix_items * prefix_units;
  int64_t total = prefix_total, before = prefix_total + incl - mine;
#pragma unroll
  for (int i = 0; i < NT / 32; ++i) {
    total += warp_sum[i];
    if (i < warp) before += warp_sum[i];
  }
  // a 64-bit division costs some hundred clocks at the start of every call
  const int64_t piece = total < (1LL << 31) ? ((uint32_t)total + n_ctas - 1) / (uint32_t)n_ctas : (total + n_ctas - 1) / n_ctas;
  const int64_t start = cta * piece, left = min(piece, total - start);
  if (left > 0) {
    if (start < prefix_total) {
      if (tid == 0) {
        found.left = left;
        found.prefix_item = start < (1LL << 31) ? (uint32_t)start / (uint32_t)prefix_units : (int)(start / prefix_units);
        found.unit = (int)(start - (int64_t)found.prefix_item * prefix_units);
        found.b = found.r = 0;
      }
    } else if (start >= before && start < before + mine) {
      int64_t at = before;
      int b = lo, n = mla_seq_units(a, w, b);
      while (start >= at + (int64_t)n * w.row_tiles) {
        at += (int64_t)n * w.row_tiles;
        n = mla_seq_units(a, w, ++b);
      }
      found.left = left;
      found.prefix_item = w.prefix_items;
      found.b = b;
      found.r = 0;
      for (; start >= at + n; at += n) ++found.r;
      found.unit = (int)(start - at);
    }
  }
  __syncthreads();
  return found;
}

// A segment whose item no other segment and no prefix item shares: its rows are final.
__device__ __forceinline__ bool mla_whole(const MlaArgs& a, const MlaPart& w, const MlaSeg& s) {
  return (a.prefix_len == 0 || w.joint) && s.tile0 == 0 && s.tile1 == s.tiles;
}
__device__ __forceinline__ MlaTile mla_tile(const MlaArgs& a, const MlaPart& w, const MlaSeg& s, int tile) {
  if (tile < s.pre) return {-1, tile * w.tile, a.prefix_len};
  return {s.b, (tile - s.pre) * w.tile, s.tokens};
}
// Tokens that row `i` of the segment's item attends to (0 past the live rows).
__device__ __forceinline__ int mla_row_limit(const MlaArgs& a, const MlaSeg& s, int i) {
  if (i >= s.nrows) return 0;
  if (s.b < 0) return s.tokens;
  return max(0, s.tokens - (a.n_q - 1 - (s.j0 + i) / a.H));
}
// Page of token t of the segment's item, -1 if the id names no page (raises *bad).
__device__ __forceinline__ int64_t mla_page(const MlaArgs& a, int b, int t, bool* bad) {
  const int p = t / a.page_tokens;
  const int id = b < 0 ? a.prefix_pages[p] : a.page_table[b * a.max_pages + p];
  if (id >= 0 && id < a.n_pages) return id;
  *bad = true;
  return -1;
}
// Note the workers that meet an item, for the merge.
__device__ __forceinline__ void mla_note_item(const MlaPart& w, const MlaSeg& s, int cta) {
  if (s.tile0 == 0) w.item_ctas[s.item].x = cta;
  if (s.tile1 == s.tiles) w.item_ctas[s.item].y = cta;
}
#endif

}  // namespace kda
