// Appending tokens to the latent page cache, with the position rotation applied on
// the way.  Per token: the row [c | k_pe] of d_c + d_r values, c normalised
// (c / sqrt(mean c^2 + eps) * w, when a weight is given) and the pairs of k_pe
// rotated by the token's angles, goes to its slot's page; every query head's d_r
// position values are rotated by the same angles.
//
// One pass: each value is read once and written once, so the work is bound by HBM
// for prompts and by latency for decode batches.  A warp takes one token's row, or
// for one token a group of query heads: a lane owns 8 pairs (16-byte loads of both
// halves, or of 16 adjacent values), whose cosines and sines stay in registers over
// the warp's heads.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/kda.h"
#include "kda_common.cuh"
#include "kda_mla.cuh"
#include "kda_tc.cuh"

namespace kda {
namespace {

constexpr int kWarps = 8;             // warps (tasks) per CTA
constexpr int kHeadIters = 4;         // query-head groups per warp

// Rotate 8 pairs: (x1, x2) -> (x1 cos - x2 sin, x2 cos + x1 sin).
template <typename T, bool INTERLEAVED>
__device__ __forceinline__ void rotate8(const T* src, T* dst, int half, int e, const float (&cs)[8],
                                        const float (&sn)[8]) {
  float a[8], b[8];
  if constexpr (INTERLEAVED) {
    float u[8], v[8];
    load8(src + 2 * e, u);
    load8(src + 2 * e + 8, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[i] = u[2 * i]; b[i] = u[2 * i + 1];
      a[4 + i] = v[2 * i]; b[4 + i] = v[2 * i + 1];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      u[2 * i] = a[i] * cs[i] - b[i] * sn[i];
      u[2 * i + 1] = b[i] * cs[i] + a[i] * sn[i];
      v[2 * i] = a[4 + i] * cs[4 + i] - b[4 + i] * sn[4 + i];
      v[2 * i + 1] = b[4 + i] * cs[4 + i] + a[4 + i] * sn[4 + i];
    }
    store8(dst + 2 * e, u);
    store8(dst + 2 * e + 8, v);
  } else {
    load8(src + e, a);
    load8(src + half + e, b);
    float u[8], v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      u[i] = a[i] * cs[i] - b[i] * sn[i];
      v[i] = b[i] * cs[i] + a[i] * sn[i];
    }
    store8(dst + e, u);
    store8(dst + half + e, v);
  }
}

template <typename T, bool INTERLEAVED>
__global__ void __launch_bounds__(32 * kWarps) kda_mla_append_kernel(const MlaAppendArgs a, int parts) {
  mla_grid_wait();
  mla_grid_next();
  const int lane = threadIdx.x & 31;
  const int64_t task = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int64_t t = task / parts;
  const int part = (int)(task - t * parts);
  if (t >= a.T) return;
  const int half = a.d_r / 2, groups = half / 8;       // groups of 8 pairs per head
  const int pos = a.d_r ? a.positions[t] : 0;
  const bool pos_ok = a.d_r == 0 || (pos >= 0 && pos < a.n_pos);
  if (!pos_ok && part == 0 && lane == 0) atomicOr(&tc::g_kda_device_error, KDA_DEVERR_INDEX);
  float cs[8], sn[8];
  const int grp = groups ? lane % groups : 0;
  if (a.d_r && pos_ok) {
    load8(a.rope + (int64_t)pos * a.d_r + 8 * grp, cs);
    load8(a.rope + (int64_t)pos * a.d_r + half + 8 * grp, sn);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) cs[i] = sn[i] = 0.f;   // no angle: zero rows
  }
  if (part == 0) {                                      // the token's cache row
    const int slot = a.slots[t];
    if (slot < 0 || slot >= a.n_pages * a.page_tokens || !pos_ok) return;
    T* row = reinterpret_cast<T*>(a.pages + (int64_t)(slot / a.page_tokens) * a.page_bytes) +
             (int64_t)(slot % a.page_tokens) * (a.d_c + a.d_r);
    const T* c = reinterpret_cast<const T*>(a.c) + t * a.c_stride;
    float x[2][8];
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int d = 8 * (lane + 32 * k);
      if (d < a.d_c) {
        load8(c + d, x[k]);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(x[k][i], x[k][i], ss);
      }
    }
    const T* w = reinterpret_cast<const T*>(a.norm_weight);
    float r = 1.f;
    if (w) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      r = 1.f / sqrtf(ss / (float)a.d_c + a.eps);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int d = 8 * (lane + 32 * k);
      if (d < a.d_c) {
        if (w) {
          float g[8];
          load8(w + d, g);
#pragma unroll
          for (int i = 0; i < 8; ++i) x[k][i] = x[k][i] * r * g[i];
        }
        store8(row + d, x[k]);
      }
    }
    if (lane < groups)
      rotate8<T, INTERLEAVED>(reinterpret_cast<const T*>(a.k_pe) + t * a.k_pe_stride, row + a.d_c, half, 8 * grp, cs, sn);
    return;
  }
  const int per_iter = 32 / groups;                     // heads per warp pass
  const int h0 = (part - 1) * per_iter * kHeadIters + lane / groups;
  if (lane >= per_iter * groups) return;
  const T* q = reinterpret_cast<const T*>(a.q_pe) + t * a.q_stride_t;
  T* out = reinterpret_cast<T*>(a.q_pe_out) + t * (int64_t)a.H * a.d_r;
#pragma unroll
  for (int k = 0; k < kHeadIters; ++k) {
    const int h = h0 + k * per_iter;
    if (h >= a.H) break;
    if (pos_ok) {
      rotate8<T, INTERLEAVED>(q + h * a.q_stride_h, out + (int64_t)h * a.d_r, half, 8 * grp, cs, sn);
    } else {
      store8(out + (int64_t)h * a.d_r + 16 * grp, cs);
      store8(out + (int64_t)h * a.d_r + 16 * grp + 8, cs);
    }
  }
}

template <typename T>
cudaError_t run_append(const MlaAppendArgs& a, int parts, unsigned grid, cudaStream_t s) {
  return a.style == KDA_ROPE_INTERLEAVED ? mla_launch(kda_mla_append_kernel<T, true>, grid, 32 * kWarps, 0, s, a, parts)
                                         : mla_launch(kda_mla_append_kernel<T, false>, grid, 32 * kWarps, 0, s, a, parts);
}

}  // namespace

cudaError_t launch_mla_append(const MlaAppendArgs& a, cudaStream_t s) {
  int parts = 1;
  if (a.q_pe) {
    const int heads = 32 / (a.d_r / 16) * kHeadIters;
    parts += (a.H + heads - 1) / heads;
  }
  const int64_t grid = ((int64_t)a.T * parts + kWarps - 1) / kWarps;
  return a.dtype == KDA_BF16 ? run_append<__nv_bfloat16>(a, parts, (unsigned)grid, s) : run_append<float>(a, parts, (unsigned)grid, s);
}

int read_and_clear_mla_append_errors(int* flags) {
  int word = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&word, tc::g_kda_device_error, sizeof(int));
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(tc::g_kda_device_error, &zero, sizeof(int));
  *flags |= word;
  return (int)e;
}

}  // namespace kda
