// Attention of decode queries over the latent page cache: a prefix that the whole
// batch shares, computed once for all rows, and each sequence's own pages.
//
// Row r = (b, i, h) attends to tokens t with keys [c_t | k_t] and values c_t:
//   x_t = scale log2(e) (q_r . c_t + qpe_r . k_t),  p_t = 2^(x_t - m),
//   o_r = sum p_t c_t / l,  l = sum p_t,  lse_r = ln 2 (m + log2 l),
// in one pass over the tokens with the running reference m and sum l.  The line of
// tiles is cut over the CTAs (kda_mla.cuh); pieces (m_j, l_j, o_j) of a row join as
//   m = max m_j,  l = sum 2^(m_j - m) l_j,  o = sum 2^(m_j - m) o_j / l.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "../../include/kda.h"
#include "kda_common.cuh"
#include "kda_mla.cuh"
#include "kda_tc.cuh"

namespace kda {
namespace {

// 2^(m_j - m) of two references, either of which may be -inf (no token seen yet).
__device__ __forceinline__ float rescale(float from, float to) { return from == -INFINITY ? 0.f : exp2f(from - to); }

// ---------------------------------------------------------------------------
// fp32 kernel, on CUDA cores (the bf16 ones: kda_mla_tc.cu, kda_mla_pair.cu).  32 rows per
// item, tiles of 32 tokens, 8 warps.  The next tile is copied (cp.async) while this one is
// computed.  Shared memory hands a warp one float per lane and clock, so a thread that
// multiplies R by C values reads R + C floats for R C FMAs, four warps' worth of which run at
// once: R and C decide.
//   Scores: a warp takes 4 tokens by 32 rows, a thread 8 rows by 4 tokens of every eighth group
//   of 16 bytes along a row (12 floats for 32 FMAs; the eight partial sums meet by
//   shuffles).  4 by 4 with fewer slices took 6000 clocks a tile of 288 values a row.
//   Softmax: a warp per four rows, a lane per token.
//   Sums over c: a thread 8 rows by d_c / 32 channels, half of the tile's tokens in four warps
//   each; the halves meet at the segment's end.  NB = d_c / 128 is a template argument
//   so that the loads of several tokens are under way together (5800 clocks a tile without).
// 64 sequences of 2000 tokens, 32 heads, d_c = 512, d_r = 64: 268 us, 33 TFLOP/s, bound by the
// reads of shared memory, which take as long as the FMAs and overlap them in part.  16 sequences of up
// to 421 tokens behind 1024, 16 heads, d_c = 256, d_r = 32: 26.5 us with the merge, latency
// of three tiles per CTA.
constexpr int kSimtRows = 32;
constexpr int kSimtTile = 32;
constexpr int kSimtThreads = 256;
constexpr int kSimtLdS = kSimtTile + 4;

size_t simt_smem(int d) {
  const int ld = d + 4;                           // rows 16 bytes apart in the banks
  return ((size_t)(kSimtRows + 2 * kSimtTile) * ld + kSimtRows * kSimtLdS) * sizeof(float);
}

// 16 bytes global -> shared, zeros if not `live`
__device__ __forceinline__ void copy16(float* dst, const float* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
               :: "r"(tc::smem_u32(dst)), "l"(src), "r"(live ? 16 : 0) : "memory");
}

template <int NB>
__global__ void __launch_bounds__(kSimtThreads) kda_mla_simt_kernel(const MlaArgs a, const MlaPart w) {
  extern __shared__ __align__(16) float sm[];
  __shared__ float row_f[kSimtRows];              // factor of a row's sums so far; at the end 1 / l
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int d = a.d_c + a.d_r, ld = d + 4;
  float* Q = sm;                                  // [rows][ld]
  float* Ks = Q + kSimtRows * ld;                 // [2][tokens][ld]
  float* S = Ks + 2 * kSimtTile * ld;             // [rows][ldS]: scores, then weights
  const int orow = 8 * (warp & 3), half = warp >> 2;   // rows of this warp's sums, its half of a tile
  constexpr int ldS = kSimtLdS;
  const float* qc = static_cast<const float*>(a.q);
  const float* qr = static_cast<const float*>(a.q_pe);
  const float* pages = reinterpret_cast<const float*>(a.pages);
  bool bad = false;
  mla_grid_enter(w);
  MlaWalk walk = mla_plan<kSimtThreads>(a, w, blockIdx.x, gridDim.x);
  MlaSeg s;
  while (walk.next(a, w, s)) {
    __syncthreads();                              // the last segment's reads of Q, K and S are done
    const int t_end = min(s.tokens, s.tile1 * kSimtTile);
    // lane l < 4 looks up the page of the warp's token l of a tile; -1: no row
    const auto offset = [&](int t0) -> int64_t {
      const int t = t0 + 4 * warp + (lane & 3);
      if (t >= t_end) return -1;
      const int64_t page = mla_page(a, s.b, t, &bad);
      return page < 0 ? -1 : page * (a.page_bytes / 4) + (int64_t)(t % a.page_tokens) * d;
    };
    const auto copy_tile = [&](float* K, int64_t off) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int64_t o = __shfl_sync(0xffffffffu, off, k);
        for (int e = 4 * lane; e < d; e += 128) copy16(K + (4 * warp + k) * ld + e, pages + (o < 0 ? 0 : o + e), o >= 0);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    for (int r = warp; r < kSimtRows; r += kSimtThreads / 32)
      for (int e = 4 * lane; e < d; e += 128) {
        const bool c = e < a.d_c, live = r < s.nrows;
        const float* src = c ? qc + (s.row0 + r) * a.d_c + e : qr + (s.row0 + r) * a.d_r + e - a.d_c;
        copy16(Q + r * ld + e, live ? src : qc, live);
      }
    float m[4], l[4];                             // rows 4 warp + k
    float o[8][NB][4];                            // rows orow + k; [block][channel]
    int lim[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      m[k] = -INFINITY;
      l[k] = 0.f;
      lim[k] = min(t_end, mla_row_limit(a, s, 4 * warp + k));
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[k][j][i] = 0.f;
    int t0 = s.tile0 * kSimtTile;
    copy_tile(Ks, offset(t0));
    int64_t next = offset(t0 + kSimtTile);
    for (int buf = 0; t0 < t_end; t0 += kSimtTile, buf ^= 1) {
      float* K = Ks + buf * kSimtTile * ld;
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncthreads();                            // this tile is here, and nobody reads the other buffer or S
      if (t0 + kSimtTile < t_end) {
        copy_tile(Ks + (buf ^ 1) * kSimtTile * ld, next);
        next = offset(t0 + 2 * kSimtTile);
      }
      {
        const int slice = lane & 7, rg = lane >> 3;                // rows rg + 4 i, tokens 4 warp + j
        const float* x0 = Q + rg * ld;
        const float* y0 = K + 4 * warp * ld;
        float acc[8][4] = {};
        for (int e = 4 * slice; e < d; e += 32) {
          float4 x[8], y[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4*>(y0 + j * ld + e);
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = *reinterpret_cast<const float4*>(x0 + 4 * i * ld + e);
#pragma unroll
          for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              acc[i][j] = fmaf(x[i].x, y[j].x, acc[i][j]);
              acc[i][j] = fmaf(x[i].y, y[j].y, acc[i][j]);
              acc[i][j] = fmaf(x[i].z, y[j].z, acc[i][j]);
              acc[i][j] = fmaf(x[i].w, y[j].w, acc[i][j]);
            }
        }
        __syncwarp();
        // each exchange joins two slices and halves a lane's rows; slice i is left with rows i
#pragma unroll
        for (int n = 4; n > 0; n >>= 1) {
          const bool up = slice & n;
#pragma unroll
          for (int i = 0; i < n; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float other = __shfl_xor_sync(0xffffffffu, up ? acc[i][j] : acc[i + n][j], n);
              acc[i][j] = (up ? acc[i + n][j] : acc[i][j]) + other;
            }
        }
        *reinterpret_cast<float4*>(S + (rg + 4 * slice) * ldS + 4 * warp) = make_float4(acc[0][0], acc[0][1], acc[0][2], acc[0][3]);
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float* row = S + (4 * warp + k) * ldS;
        const float x = t0 + lane < lim[k] ? a.scale_log2 * row[lane] : -INFINITY;
        float top = x;
#pragma unroll
        for (int f = 16; f > 0; f >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, f));
        const float mn = fmaxf(m[k], top), base = mn == -INFINITY ? 0.f : mn;
        const float p = exp2f(x - base), f = rescale(m[k], base);
        m[k] = mn;
        l[k] = l[k] * f + p;                      // per lane; joined at the segment's end
        row[lane] = p;
        if (lane == 0) row_f[4 * warp + k] = f;
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float f = row_f[orow + k];
        if (f != 1.f) {
#pragma unroll
          for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[k][j][i] *= f;
        }
      }
#pragma unroll 1
      for (int t = 16 * half; t < 16 * half + 16; t += 4) {
        float4 c[4][NB];
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int j = 0; j < NB; ++j) c[u][j] = *reinterpret_cast<const float4*>(K + (t + u) * ld + 128 * j + 4 * lane);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float4 p4 = *reinterpret_cast<const float4*>(S + (orow + k) * ldS + t);
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const float p = u == 0 ? p4.x : u == 1 ? p4.y : u == 2 ? p4.z : p4.w;
#pragma unroll
            for (int j = 0; j < NB; ++j) {
              o[k][j][0] = fmaf(p, c[u][j].x, o[k][j][0]);
              o[k][j][1] = fmaf(p, c[u][j].y, o[k][j][1]);
              o[k][j][2] = fmaf(p, c[u][j].z, o[k][j][2]);
              o[k][j][3] = fmaf(p, c[u][j].w, o[k][j][3]);
            }
          }
        }
      }
    }
    const bool whole = mla_whole(a, w, s);
    if (tid == 0) mla_note_item(w, s, blockIdx.x);
    const int64_t slot = (s.item + blockIdx.x) * w.nr;
    __syncthreads();                              // reads of K and row_f are done
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int r = 4 * warp + k;
#pragma unroll
      for (int f = 16; f > 0; f >>= 1) l[k] += __shfl_xor_sync(0xffffffffu, l[k], f);
      if (lane == 0) {
        row_f[r] = !whole ? 1.f : l[k] > 0.f ? 1.f / l[k] : 0.f;
        if (r < s.nrows) {
          if (!whole) w.part_ml[slot + r] = make_float2(m[k], l[k]);
          else if (a.lse) a.lse[s.row0 + r] = 0.6931471805599453f * (m[k] + log2f(l[k]));
        }
      }
    }
    // each of two warps gives the other its sums of four of their eight rows
    float* give = Ks + 4 * lane;                  // [rows][d_c]
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const float* x = half ? o[k][j] : o[4 + k][j];
        *reinterpret_cast<float4*>(give + (orow + 4 * (half ^ 1) + k) * a.d_c + 128 * j) = make_float4(x[0], x[1], x[2], x[3]);
      }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int r = orow + 4 * half + k;
      if (r >= s.nrows) break;
      const float f = row_f[r];
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const float* x = half ? o[4 + k][j] : o[k][j];
        const float4 y = *reinterpret_cast<const float4*>(give + r * a.d_c + 128 * j);
        const float4 z = make_float4((x[0] + y.x) * f, (x[1] + y.y) * f, (x[2] + y.z) * f, (x[3] + y.w) * f);
        if (whole) store4(static_cast<float*>(a.o) + (s.row0 + r) * a.d_c + 128 * j + 4 * lane, z);
        else store4(w.part_o + (slot + r) * a.d_c + 128 * j + 4 * lane, z);
      }
    }
  }
  if (bad) atomicOr(&tc::g_kda_device_error, KDA_DEVERR_INDEX);
}

// ---------------------------------------------------------------------------
// Join the partial results of each row.  Rows that no token reaches get o = 0 and
// lse = -inf.  `pre` is the part that holds the prefix, `own` the one that holds the
// sequences' own tokens.  A lane reads the statistics of one slot and four groups of four
// channels of each; WARPS warps share a row's slots.
template <typename T, int WARPS>
__global__ void __launch_bounds__(128) kda_mla_merge_kernel(const MlaArgs a, const MlaPart pre, const MlaPart own) {
  __shared__ float4 sum[WARPS > 1 ? WARPS : 1][128];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, share = warp % WARPS;
  const unsigned row = blockIdx.x * (4 / WARPS) + warp / WARPS;
  const bool here = row < (unsigned)a.B * a.seq_rows;
  const int b = here ? row / a.seq_rows : 0, j = here ? row % a.seq_rows : 0;
  mla_grid_wait();
  mla_grid_next();
  int64_t at[2] = {0, 0};                         // row of the first slot, prefix and own tokens
  int n0 = 0, n1 = 0;                             // slots
  if (here && a.lens[b] >= 0) {
    if (pre.prefix_items > 0) {
      const unsigned item = row / pre.nr;
      const int2 c = pre.item_ctas[item];
      at[0] = ((int64_t)item + c.x) * pre.nr + row % pre.nr;
      n0 = c.y - c.x + 1;
    }
    if (mla_seq_tiles(a, own, b) > 0) {
      const int64_t item = own.prefix_items + (int64_t)b * own.row_tiles + j / own.nr;
      const int2 c = own.item_ctas[item];
      at[1] = (item + c.x) * own.nr + j % own.nr;
      n1 = c.y - c.x + 1;
    }
  }
  // one slot and no prefix item: written whole by the attention kernel
  const bool done = !here || (pre.prefix_items == 0 && n1 == 1);
  if (WARPS == 1 && done) return;
  const int n = done ? 0 : n0 + n1;
  const auto slot = [&](int k) { return k < n0 ? at[0] + (int64_t)k * pre.nr : at[1] + (int64_t)(k - n0) * own.nr; };
  float m = -INFINITY;
  for (int k = lane; k < n; k += 32) m = fmaxf(m, (k < n0 ? pre.part_ml : own.part_ml)[slot(k)].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float base = m == -INFINITY ? 0.f : m;
  float l = 0.f;
  float4 acc[4];
#pragma unroll
  for (int g = 0; g < 4; ++g) acc[g] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k0 = 0; k0 < n; k0 += 32) {
    float f = 0.f;
    if (k0 + lane < n) {
      const float2 x = (k0 + lane < n0 ? pre.part_ml : own.part_ml)[slot(k0 + lane)];
      f = rescale(x.x, base);
      l = fmaf(f, x.y, l);
    }
    const int end = min(32, n - k0);
#pragma unroll 4
    for (int i = share; i < end; i += WARPS) {
      const float fi = __shfl_sync(0xffffffffu, f, i);
      const float* o = (k0 + i < n0 ? pre.part_o : own.part_o) + slot(k0 + i) * a.d_c + 4 * lane;
#pragma unroll
      for (int g = 0; g < 4; ++g)
        if (128 * g < a.d_c) acc[g] = f4_fma(fi, *reinterpret_cast<const float4*>(o + 128 * g), acc[g]);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  const float inv = l > 0.f ? 1.f / l : 0.f;
  T* out = reinterpret_cast<T*>(a.o) + (int64_t)row * a.d_c + 4 * lane;
  if constexpr (WARPS > 1) {
#pragma unroll
    for (int g = 0; g < 4; ++g) sum[warp][32 * g + lane] = acc[g];
    __syncthreads();
    // this warp's share of the row's channels
#pragma unroll
    for (int g = share; g < 4; g += WARPS) {
      float4 x = sum[warp - share][32 * g + lane];
#pragma unroll
      for (int v = 1; v < WARPS; ++v) x = f4_fma(1.f, sum[warp - share + v][32 * g + lane], x);
      if (!done && 128 * g < a.d_c) store4(out + 128 * g, make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv));
    }
  } else {
#pragma unroll
    for (int g = 0; g < 4; ++g)
      if (128 * g < a.d_c) store4(out + 128 * g, make_float4(acc[g].x * inv, acc[g].y * inv, acc[g].z * inv, acc[g].w * inv));
  }
  if (!done && share == 0 && lane == 0 && a.lse) a.lse[row] = 0.6931471805599453f * (m + log2f(l));
}

template <int NB>
cudaError_t run_simt(const MlaArgs& a, const MlaPart& w, int sms, cudaStream_t s) {
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = mla_allow_smem(kda_mla_simt_kernel<NB>, (int)simt_smem(128 * NB + 64), allowed);
  if (e != cudaSuccess) return e;
  return mla_launch(kda_mla_simt_kernel<NB>, sms, kSimtThreads, simt_smem(a.d_c + a.d_r), s, a, w);
}
cudaError_t launch_mla_simt(const MlaArgs& a, const MlaPart& w, int sms, cudaStream_t s) {
  switch (a.d_c / 128) {
    case 1: return run_simt<1>(a, w, sms, s);
    case 2: return run_simt<2>(a, w, sms, s);
    case 3: return run_simt<3>(a, w, sms, s);
    default: return run_simt<4>(a, w, sms, s);
  }
}

template <typename T>
cudaError_t run_merge(const MlaArgs& a, const MlaPart& pre, const MlaPart& own, cudaStream_t s) {
  // Few rows have many slots each: four warps per row.  One / four, us per call of 32 heads: 8 sequences of 100-1000
  // tokens behind 2000 29 / 20, 16 31 / 22, 32 32 / 28, 63 39 / 40, 64 of 600 alone 22 / 23, 128 33 / 38.
  const unsigned rows = (unsigned)a.B * a.seq_rows;
  return rows < 2048 ? mla_launch(kda_mla_merge_kernel<T, 4>, rows, 128, 0, s, a, pre, own)
                     : mla_launch(kda_mla_merge_kernel<T, 1>, (rows + 3) / 4, 128, 0, s, a, pre, own);
}

// SM count of the current device, looked up once per device.
cudaError_t device_sms(int* sms) {
  static std::atomic<int> known[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && (*sms = known[dev].load(std::memory_order_relaxed)) > 0) return cudaSuccess;
  e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess && dev < 64) known[dev].store(*sms, std::memory_order_relaxed);
  return e;
}

}  // namespace

// Which kernel takes what.  fp32: the CUDA-core kernel.  bf16: the pair kernel wherever
// more than 64 rows read the same tokens (its products are full at 128 rows, and its cost
// per tile is shared by them), else the one-CTA kernel.
// Own tokens at 65 rows and more, one CTA / pair, us per call at 66, 96 and 128 rows a sequence:
// one sequence of 1000 tokens 16.9 / 16.4, 16.8 / 16.1, 16.9 / 16.4; 16 of 100-1000 20.2 / 19.6,
// 21.3 / 20.8, 23.1 / 21.0; 64 of 100-2000 43 / 31, 44 / 32, 46 / 33; 128 of 500-4000 122 / 90,
// 126 / 93, 129 / 96; 32 of 10-300 behind 4000 46 / 37, 51 / 44, 57 / 45.
// A prefix whose owners go to the
// one-CTA kernel is worth a launch of its own above 2^22 rows x tokens: prefix apart / all in
// one launch, us per call: 16 sequences of 32 heads over 1000 tokens (0.5e6) 21 / 19, 37 of
// 3x20 (2.2e6) 38 / 29, 64 of 32 over 2048 (4.2e6) 40 / 38, 100 of 16 over 3000 (4.8e6) 41 / 43,
// 64 of 32 over 4096 (8.4e6) 46 / 52, 128 of 32 over 8192 (34e6) 87 / 142.  Near the bound it
// can be wrong by a tenth where an owner has few rows (256 of 4 over 2048, 2.1e6: 34 / 38).
int mla_parts(int B, int seq_rows, int64_t prefix_len, int dtype, MlaPart (&parts)[2]) {
  const int64_t rows = (int64_t)B * seq_rows;
  const bool bf16 = dtype == KDA_BF16;
  const auto make = [&](bool pair, bool prefix, bool own) {
    MlaPart w{};
    w.kernel = !bf16 ? kMlaSimt : pair ? kMlaPair : kMlaTc;
    w.tile = !bf16 ? kSimtTile : pair ? 128 : 64;
    // Measured, us per call.  One CTA, at 1 / 2 / 3 / 4 units: batch of 256 151.2 / 151.4 / 152.5 /
    // 154.7, 37 sequences of 3x20 33.2 / 28.3 / 28.5 / 28.0.  Pair (its items' ends and starts do not
    // overlap), at 3 / 4 / 5 / 6 / 8 units: 8-token drafts 114.7 / 114.5 / 115.7 / 117.1 / 119.3 (without any, 2.8
    // times as long), 128 behind a prefix 133.0 / 130.6 / 131.8 / 131.6 / 133.2: 3 to 6 differ by less than
    // one GPU from another, what counts is that there are some.  fp32, at 0 / 1 / 2: 32.1 / 26.5 / 26.6.
    w.prefix_cost = w.own_cost = !bf16 ? 1 : pair ? 4 : 2;
    // no more rows than an item can have: smaller products, and shared memory for more tiles
    const int64_t most = prefix ? rows : seq_rows;
    w.nr = !bf16 ? kSimtRows : pair ? 128 : most <= 16 ? 16 : most <= 32 ? 32 : 64;
    if (prefix) w.prefix_tiles = (int)((prefix_len + w.tile - 1) / w.tile);
    if (own) w.row_tiles = (seq_rows + w.nr - 1) / w.nr;
    // Joint where a sequence's rows leave few of its items' rows empty (the prefix's tiles cost
    // the same for an empty row).  Prefix apart / joint, us per call, at 80, 96, 112, 128, 192 and 256 rows:
    // 8 sequences behind 16000 tokens 34 / 40, 36 / 40, 38 / 40, 42 / 40, 55 / 64, 66 / 64; 32 of 10-300 behind
    // 4000 38 / 44, 41 / 44, 44 / 44, 47 / 45, 66 / 71, 76 / 73; 64 of 500-3000 behind 1000 61 / 62,
    // 66 / 64, 68 / 66, 71 / 68, 117 / 98, 128 / 102.  The lengths decide it between three quarters and whole
    // items, and the host does not know them.
    w.joint = pair && prefix && own && 4 * seq_rows >= 3 * w.row_tiles * w.nr;
    if (prefix && !w.joint) w.prefix_items = (int)((rows + w.nr - 1) / w.nr);
    w.own_items = (int64_t)B * w.row_tiles;
    return w;
  };
  const bool own_pair = bf16 && seq_rows > 64;
  const bool pre_pair = own_pair || (bf16 && rows > 64 && rows * prefix_len > ((int64_t)1 << 22));
  if (prefix_len == 0) {
    parts[0] = make(own_pair, false, true);
    return 1;
  }
  if (pre_pair == own_pair) {
    parts[0] = make(pre_pair, true, true);
    return 1;
  }
  parts[0] = make(pre_pair, true, false);
  parts[1] = make(own_pair, false, true);
  parts[1].second = 1;
  return 2;
}

cudaError_t launch_mla_decode(const MlaArgs& a, const MlaPart* parts, int n, cudaStream_t s) {
  int sms = 0;
  cudaError_t e = device_sms(&sms);
  sms = std::min(sms, kMlaMaxCtas);
  for (int i = 0; i < n && e == cudaSuccess; ++i) {
    const MlaPart& w = parts[i];
    e = w.kernel == kMlaPair ? launch_mla_pair(a, w, sms, s) : w.kernel == kMlaTc ? launch_mla_tc(a, w, sms, s) : launch_mla_simt(a, w, sms, s);
  }
  if (e != cudaSuccess) return e;
  return a.dtype == KDA_BF16 ? run_merge<__nv_bfloat16>(a, parts[0], parts[n - 1], s) : run_merge<float>(a, parts[0], parts[n - 1], s);
}

int read_and_clear_mla_errors(int* flags) {
  int word = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&word, tc::g_kda_device_error, sizeof(int));
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(tc::g_kda_device_error, &zero, sizeof(int));
  *flags |= word;
  if (e == cudaSuccess) e = (cudaError_t)read_and_clear_mla_tc_errors(flags);
  if (e == cudaSuccess) e = (cudaError_t)read_and_clear_mla_pair_errors(flags);
  return (int)e;
}

}  // namespace kda
