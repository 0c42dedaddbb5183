// Appending tokens to the latent page cache, with the position rotation applied on
// the way.  Per token: the row [c | k_pe] of d_c + d_r values, c normalised
// (c / sqrt(mean c^2 + eps) * w, when a weight is given) and the pairs of k_pe
// rotated by the token's angles, goes to its slot's page; every query head's d_r
// position values are rotated by the same angles.
//
// One pass: each value is read once and written once, so the work is bound by HBM
// for prompts and by latency for decode batches (2.8 us for 256 tokens, most of it the
// launch and the chain position -> angles).  A warp takes one token's row, or for one token
// groups of query heads: a lane owns 8 pairs (16-byte loads of both halves, or of 16
// adjacent values), whose cosines and sines stay in registers over the warp's heads.
// 32768 tokens, 32 heads, bf16: 63 us, 5.6 TB/s (83% of the measured copy rate; the
// queries' position parts are 128-byte pieces of longer rows).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/kda.h"
#include "kda_common.cuh"
#include "kda_mla.cuh"
#include "kda_tc.cuh"

namespace kda {
namespace {

constexpr int kWarps = 8;             // warps (tasks) per CTA

// Eight values as they lie in memory: kept like this between load and use, a bf16 warp needs
// half the registers, and more warps fit (as floats, 99 registers a thread: 125 us for a
// 32768-token prompt).
template <typename T> struct Raw8;
template <> struct Raw8<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
};
template <> struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
};

// 8 pairs of a head: values e .. of both halves, or 16 neighbours from 2 e; and as x1 = a, x2 = b.
template <bool INTERLEAVED, typename T>
__device__ __forceinline__ void load_pairs(const T* src, int half, int e, Raw8<T>& x, Raw8<T>& y) {
  x.load(INTERLEAVED ? src + 2 * e : src + e);
  y.load(INTERLEAVED ? src + 2 * e + 8 : src + half + e);
}
template <bool INTERLEAVED, typename T>
__device__ __forceinline__ void get_pairs(const Raw8<T>& x, const Raw8<T>& y, float (&a)[8], float (&b)[8]) {
  if constexpr (INTERLEAVED) {
    float u[8], v[8];
    x.get(u);
    y.get(v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[i] = u[2 * i]; b[i] = u[2 * i + 1];
      a[4 + i] = v[2 * i]; b[4 + i] = v[2 * i + 1];
    }
  } else {
    x.get(a);
    y.get(b);
  }
}
// The pairs rotated, (x1, x2) -> (x1 cos - x2 sin, x2 cos + x1 sin), and stored.
template <bool INTERLEAVED, typename T>
__device__ __forceinline__ void store_rotated(T* dst, int half, int e, const float (&a)[8], const float (&b)[8],
                                              const float (&cs)[8], const float (&sn)[8]) {
  float u[8], v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    u[i] = a[i] * cs[i] - b[i] * sn[i];
    v[i] = b[i] * cs[i] + a[i] * sn[i];
  }
  if constexpr (INTERLEAVED) {
    float x[8], y[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = u[i]; x[2 * i + 1] = v[i];
      y[2 * i] = u[4 + i]; y[2 * i + 1] = v[4 + i];
    }
    store8(dst + 2 * e, x);
    store8(dst + 2 * e + 8, y);
  } else {
    store8(dst + e, u);
    store8(dst + half + e, v);
  }
}

// ITERS: query-head groups per warp.  A warp's loads are all issued before its first store (the
// outputs may be the inputs' own memory, so the compiler keeps their order).  Measured for
// bf16 at 32768 tokens, 32 heads, d_c 512, d_r 64 (353 MB): 1 / 2 / 4 groups per warp 94 / 71
// / 68 us at four CTAs per SM, 4 groups at three CTAs 70 us; loads and stores in turn, 77 us.
template <typename T, bool INTERLEAVED, int ITERS>
__global__ void __launch_bounds__(32 * kWarps, sizeof(T) == 2 ? 4 : 2) kda_mla_append_kernel(const MlaAppendArgs a, int parts) {
  mla_grid_wait();
  mla_grid_next();
  const int lane = threadIdx.x & 31;
  const unsigned task = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int t = (int)(task / (unsigned)parts), part = (int)(task - (unsigned)t * parts);
  if (t >= a.T) return;
  const int half = a.d_r / 2, groups = half / 8;       // groups of 8 pairs per head
  const int pos = a.d_r ? a.positions[t] : 0;
  const bool pos_ok = a.d_r == 0 || (pos >= 0 && pos < a.n_pos);
  const int grp = groups ? lane % groups : 0;
  const auto angles = [&](float (&cs)[8], float (&sn)[8]) {
    if (a.d_r && pos_ok) {
      load8(a.rope + (int64_t)pos * a.d_r + 8 * grp, cs);
      load8(a.rope + (int64_t)pos * a.d_r + half + 8 * grp, sn);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) cs[i] = sn[i] = 0.f;
    }
  };
  float cs[8], sn[8];
  if (part == 0) {                                      // the token's cache row
    const int slot = a.slots[t];
    const T* c = reinterpret_cast<const T*>(a.c) + t * a.c_stride;
    const T* w = reinterpret_cast<const T*>(a.norm_weight);
    Raw8<T> x[2], g[2], ka, kb;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int d = 8 * (lane + 32 * k);
      if (d < a.d_c) {
        x[k].load(c + d);
        if (w) g[k].load(w + d);
      }
    }
    if (lane < groups) load_pairs<INTERLEAVED>(reinterpret_cast<const T*>(a.k_pe) + t * a.k_pe_stride, half, 8 * grp, ka, kb);
    angles(cs, sn);
    if (!pos_ok && lane == 0) atomicOr(&tc::g_kda_device_error, KDA_DEVERR_INDEX);
    if (slot < 0 || slot >= a.n_pages * a.page_tokens || !pos_ok) return;
    T* row = reinterpret_cast<T*>(a.pages + (int64_t)(slot / a.page_tokens) * a.page_bytes) +
             (int64_t)(slot % a.page_tokens) * (a.d_c + a.d_r);
    float r = 1.f;
    if (w) {
      float ss = 0.f;
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (8 * (lane + 32 * k) < a.d_c) {
          float v[8];
          x[k].get(v);
#pragma unroll
          for (int i = 0; i < 8; ++i) ss = fmaf(v[i], v[i], ss);
        }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      r = 1.f / sqrtf(ss / (float)a.d_c + a.eps);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int d = 8 * (lane + 32 * k);
      if (d < a.d_c) {
        float v[8];
        x[k].get(v);
        if (w) {
          float f[8];
          g[k].get(f);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = v[i] * r * f[i];
        }
        store8(row + d, v);
      }
    }
    if (lane < groups) {
      float u[8], v[8];
      get_pairs<INTERLEAVED>(ka, kb, u, v);
      store_rotated<INTERLEAVED>(row + a.d_c, half, 8 * grp, u, v, cs, sn);
    }
    return;
  }
  const int per_iter = 32 / groups;                     // heads per group of heads
  const int h0 = (part - 1) * per_iter * ITERS + lane / groups;
  if (lane >= per_iter * groups) return;
  const T* q = reinterpret_cast<const T*>(a.q_pe) + t * a.q_stride_t;
  T* out = reinterpret_cast<T*>(a.q_pe_out) + t * (int64_t)a.H * a.d_r;
  Raw8<T> qa[ITERS], qb[ITERS];
#pragma unroll
  for (int k = 0; k < ITERS; ++k)
    if (h0 + k * per_iter < a.H) load_pairs<INTERLEAVED>(q + (h0 + k * per_iter) * a.q_stride_h, half, 8 * grp, qa[k], qb[k]);
  angles(cs, sn);
#pragma unroll
  for (int k = 0; k < ITERS; ++k) {
    if (h0 + k * per_iter >= a.H) break;
    float u[8], v[8];
    get_pairs<INTERLEAVED>(qa[k], qb[k], u, v);
    if (!pos_ok) {                                      // no angle: zeros, whatever the query holds
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] = v[i] = 0.f;
    }
    store_rotated<INTERLEAVED>(out + (int64_t)(h0 + k * per_iter) * a.d_r, half, 8 * grp, u, v, cs, sn);
  }
}

template <typename T, int ITERS>
cudaError_t run_append(const MlaAppendArgs& a, cudaStream_t s) {
  int parts = 1;
  if (a.q_pe) {
    const int heads = 32 / (a.d_r / 16) * ITERS;
    parts += (a.H + heads - 1) / heads;
  }
  const unsigned grid = (unsigned)(((int64_t)a.T * parts + kWarps - 1) / kWarps);
  return a.style == KDA_ROPE_INTERLEAVED ? mla_launch(kda_mla_append_kernel<T, true, ITERS>, grid, 32 * kWarps, 0, s, a, parts)
                                         : mla_launch(kda_mla_append_kernel<T, false, ITERS>, grid, 32 * kWarps, 0, s, a, parts);
}

}  // namespace

cudaError_t launch_mla_append(const MlaAppendArgs& a, cudaStream_t s) {
  return a.dtype == KDA_BF16 ? run_append<__nv_bfloat16, 4>(a, s) : run_append<float, 1>(a, s);
}

int read_and_clear_mla_append_errors(int* flags) {
  int word = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&word, tc::g_kda_device_error, sizeof(int));
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(tc::g_kda_device_error, &zero, sizeof(int));
  *flags |= word;
  return (int)e;
}

}  // namespace kda
