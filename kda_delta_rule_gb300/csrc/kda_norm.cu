// The norms around a block of a hybrid stack, each one pass over HBM.
//
// gated:     y = rms(x) w act(gate), or rms(x act(gate)) w, for every head of every token; rms(x) = x / sqrt(mean x^2 + eps).
//            A row of d values lies in 4 to 32 lanes of one warp, 8 values a lane (16-byte accesses for bf16), so its
//            sum is a few shuffles.  Three accesses per value: bound by HBM for prompts, by the launch for decode batches.
// residual:  h' = h + a s act(gate) [rms(y) w_post]; x = rms(h') w_pre, for every token.  A row lies in the registers of one
//            warp or of a few; the sums of squares of y and of h' follow one another, everything else is read once and
//            written once.  x is computed from h' before its rounding.
//
// Values are fp32 from load to store, and each output is rounded once.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/kda.h"
#include "kda_common.cuh"
#include "kda_mla.cuh"
#include "kda_norm.h"

namespace kda {
namespace {

// Eight values as they lie in memory, until they are used.
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

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// v times act(g): two channels at a time where an instruction takes them, and one test of `act` for all.  With u = e^(-|g| / 2), which does not
// underflow where a sigmoid of g can still matter, sigmoid(g) is 1 / (1 + u^2), times u^2 below zero, and u multiplies v twice.  FINE, where an
// output is fp32: the exponent with what its product with log2(e) / 2 rounded off, so that a far gate keeps its bits (without, -80 is off by
// 3e-6, which bf16 does not show).  32768 tokens of 32 heads of 128 in bf16 take 142 us, with expf 174.
template <bool FINE, bool SILU>
__device__ __forceinline__ void sigmoid8(float (&v)[8], const float (&g)[8]) {
  constexpr float C = 0.72134752f, REST = 9.6298149e-9f, LN2 = 0.69314718f;   // log2(e) / 2 = C + REST
  const float2 one = make_float2(1.f, 1.f);
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    float2 u;
    if constexpr (FINE) {
      float x[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float a = fabsf(g[j + i]), y = a * C, e = fminf(fmaf(a, REST, fmaf(a, C, -y)), 1.f);   // 1: of an infinite gate, whose w is 0
        const float w = ex2(-y);
        x[i] = fmaf(w, -LN2 * e, w);
      }
      u = make_float2(x[0], x[1]);
    } else {
      const float2 y = __fmul2_rn(make_float2(g[j], g[j + 1]), make_float2(C, C));
      u = make_float2(ex2(-fabsf(y.x)), ex2(-fabsf(y.y)));
    }
    const float2 d = __ffma2_rn(u, u, one), m = make_float2(g[j] < 0.f ? u.x : 1.f, g[j + 1] < 0.f ? u.y : 1.f);
    float2 p = __fmul2_rn(__fmul2_rn(make_float2(v[j], v[j + 1]), make_float2(rcp(d.x), rcp(d.y))), m);
    if (SILU) p = __fmul2_rn(p, make_float2(g[j], g[j + 1]));
    p = __fmul2_rn(p, m);
    v[j] = p.x;
    v[j + 1] = p.y;
  }
}
template <bool FINE>
__device__ __forceinline__ void gate8(float (&v)[8], const float (&g)[8], int act) {
  if (act == KDA_ACT_NONE) {
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const float2 p = __fmul2_rn(make_float2(v[j], v[j + 1]), make_float2(g[j], g[j + 1]));
      v[j] = p.x;
      v[j + 1] = p.y;
    }
  } else if (act == KDA_ACT_SILU) {
    sigmoid8<FINE, true>(v, g);
  } else {
    sigmoid8<FINE, false>(v, g);
  }
}
// v times f, and times w
__device__ __forceinline__ void scale8(float (&v)[8], float f, const float (&w)[8]) {
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const float2 p = __fmul2_rn(__fmul2_rn(make_float2(v[j], v[j + 1]), make_float2(f, f)), make_float2(w[j], w[j + 1]));
    v[j] = p.x;
    v[j + 1] = p.y;
  }
}

constexpr int kWarps = 4;

// LPR lanes a row, V vectors of 8 values a lane, R rows under way for each lane: 32768 tokens of 32 heads of 128 take 159 us with one
// row a lane, 142 with two (85% of the measured copy rate), 191 with three, which leave too few warps; with CTAs of eight warps 153.
template <typename T, int LPR, int V, int R>
__global__ void __launch_bounds__(32 * kWarps) kda_gated_norm_kernel(const GatedNormArgs a) {
  mla_grid_wait();
  mla_grid_next();
  constexpr int RPW = 32 / LPR;
  const int lane = threadIdx.x & 31, sub = lane % LPR;
  const unsigned rows = (unsigned)(a.T * a.H), H = (unsigned)a.H;
  const unsigned row0 = (blockIdx.x * kWarps + (threadIdx.x >> 5)) * (RPW * R) + lane / LPR;
  Raw8<T> rx[R][V], rz[R][V], rw[R][V];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const unsigned row = row0 + r * RPW;
    if (row >= rows) continue;
    const unsigned t = row / H, h = row - t * H;
    const T* x = reinterpret_cast<const T*>(a.x) + t * a.x_stride + (int64_t)h * a.d;
    const T* z = reinterpret_cast<const T*>(a.gate) + t * a.gate_stride + (int64_t)h * a.d;
    const T* w = reinterpret_cast<const T*>(a.weight) + (int64_t)h * a.weight_stride;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = 8 * (sub + i * LPR);
      if (e < a.d) {
        rx[r][i].load(x + e);
        if (a.gate) rz[r][i].load(z + e);
        if (r == 0 || a.weight_stride != 0) rw[r][i].load(w + e);
        else rw[r][i] = rw[0][i];
      }
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const unsigned row = row0 + r * RPW;
    const bool in = row < rows;
    float v[V][8], ss = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const bool has = in && 8 * (sub + i * LPR) < a.d;
      rx[r][i].get(v[i]);
      if (a.gate && a.gate_first) {
        float g[8];
        rz[r][i].get(g);
        gate8<sizeof(T) == 4>(v[i], g, a.act);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (!has) v[i][j] = 0.f;
        ss = fmaf(v[i][j], v[i][j], ss);
      }
    }
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float f = 1.f / sqrtf(ss / (float)a.d + a.eps);
    T* y = reinterpret_cast<T*>(a.y) + (int64_t)row * a.d;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = 8 * (sub + i * LPR);
      if (!in || e >= a.d) continue;
      float w[8];
      rw[r][i].get(w);
      scale8(v[i], f, w);
      if (a.gate && !a.gate_first) {
        rz[r][i].get(w);
        gate8<sizeof(T) == 4>(v[i], w, a.act);
      }
      store8(y + e, v[i]);
    }
  }
}

template <typename T, int LPR, int V, int R>
cudaError_t run_gated_rows(const GatedNormArgs& a, cudaStream_t s) {
  const int64_t per = kWarps * (32 / LPR) * R;
  return mla_launch(kda_gated_norm_kernel<T, LPR, V, R>, (unsigned)((a.T * a.H + per - 1) / per), 32 * kWarps, 0, s, a);
}
template <typename T, int LPR, int V>
cudaError_t run_gated(const GatedNormArgs& a, cudaStream_t s) {
  // Two rows a lane where a row has little under way, one bf16 vector a lane, and 64 warps of rows for every SM are there (one row / two, us,
  // d = 128: 9728 rows 3.30 / 3.65, 19456 5.19 / 4.94, 524288 80.6 / 72.4; d = 64: 19456 rows 3.29 / 3.60, 38912 5.17 / 4.81).  Two vectors
  // a lane, and fp32, are better by themselves (524288 rows, bf16 of 512 values 262 / 360; 155648, fp32 of 256 67.6 / 68.3, 9728 6.4 / 7.0).
  if constexpr (V * sizeof(T) <= 2)
    if (a.T * a.H >= kSms * 64 * (32 / LPR)) return run_gated_rows<T, LPR, V, 2>(a, s);
  return run_gated_rows<T, LPR, V, 1>(a, s);
}
template <typename T>
cudaError_t run_gated_d(const GatedNormArgs& a, cudaStream_t s) {
  const int vecs = a.d / 8;
  if (vecs <= 4) return run_gated<T, 4, 1>(a, s);
  if (vecs <= 8) return run_gated<T, 8, 1>(a, s);
  if (vecs <= 16) return run_gated<T, 16, 1>(a, s);
  if (vecs <= 32) return run_gated<T, 32, 1>(a, s);
  if (vecs <= 64) return run_gated<T, 32, 2>(a, s);
  return run_gated<T, 32, 4>(a, s);
}

// The sum of x over a row's threads, tx of them (a whole number of warps): by shuffles, and across warps through `red`.
__device__ __forceinline__ float row_sum(float x, int tx, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  if (tx == 32) return x;
  const int warp = threadIdx.x >> 5, n = tx >> 5;
  if ((threadIdx.x & 31) == 0) red[warp] = x;
  __syncthreads();
  x = 0.f;
  for (int i = 0; i < n; ++i) x += red[i];
  return x;
}

// V vectors of 8 values a thread; blockDim.x threads a row, blockDim.y rows at a time (of one warp each, if more than one).  A CTA walks
// over rows, and asks for the next one's values as soon as this one's are in h, before the sum over h; where only one fits an SM (V = 4), it
// has one row, and the next CTA's loads begin when it ends.  Two on an SM for rows of up to 6144 values.  16384 rows, bf16, every part (a CTA a
// row / walking, us): h in bf16, 2048 values 84.0 / 73.2, 6144 217 / 211, 8192 270 / 333; h in fp32, 2048 values 92.9 / 82.2, 6144 256 / 262 (80% of
// the measured copy rate), 8192 330 / 404.
template <typename T, typename TH, int V>
__global__ void __launch_bounds__(V == 2 ? 384 : 512, V == 4 ? 1 : 2) kda_residual_norm_kernel(const ResidualNormArgs a) {
  __shared__ float red[4][16];
  mla_grid_wait();
  mla_grid_next();
  const int tx = blockDim.x;
  const T *post = reinterpret_cast<const T*>(a.post_weight), *pre = reinterpret_cast<const T*>(a.pre_weight);
  const T* cs = reinterpret_cast<const T*>(a.channel_scale);
  Raw8<T> ry[V], rz[V];
  Raw8<TH> rh[V];
  const auto fetch = [&](int64_t t) {
    const T* y = reinterpret_cast<const T*>(a.y) + t * a.y_stride;
    const T* z = reinterpret_cast<const T*>(a.gate) + t * a.gate_stride;
    const TH* hi = reinterpret_cast<const TH*>(a.h_in) + t * a.h_stride;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = 8 * (threadIdx.x + i * tx);
      if (e < a.D) {
        ry[i].load(y + e);
        if (a.gate) rz[i].load(z + e);
        rh[i].load(hi + e);
      }
    }
  };
  const int64_t step = (int64_t)gridDim.x * blockDim.y;
  int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (t < a.T) fetch(t);
  for (int turn = 0; t < a.T; t += step, turn ^= 2) {   // rows of one warp end their loops apart; others have the block to themselves
    float r = 1.f;
    if (a.post_weight) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (8 * (threadIdx.x + i * tx) >= a.D) continue;
        float v[8];
        ry[i].get(v);
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(v[j], v[j], ss);
      }
      r = 1.f / sqrtf(row_sum(ss, tx, red[turn]) / (float)a.D + a.eps);
    }
    TH* ho = reinterpret_cast<TH*>(a.h_out) + t * a.h_stride;
    float h[V][8], ss = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = 8 * (threadIdx.x + i * tx);
      if (e >= a.D) continue;
      float u[8], f[8];
      ry[i].get(u);
      if (a.post_weight) {
        load8(post + e, f);
        scale8(u, r, f);
      }
      if (a.gate) {
        rz[i].get(f);
        gate8<sizeof(TH) == 4>(u, f, a.act);
      }
      if (cs) {
        load8(cs + e, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) u[j] *= f[j];
      }
      rh[i].get(h[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        h[i][j] = fmaf(a.res_scale, u[j], h[i][j]);
        ss = fmaf(h[i][j], h[i][j], ss);
      }
      store8(ho + e, h[i]);
    }
    if (t + step < a.T) fetch(t + step);
    r = 1.f / sqrtf(row_sum(ss, tx, red[turn + 1]) / (float)a.D + a.eps);
    T* x = reinterpret_cast<T*>(a.x) + t * a.D;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = 8 * (threadIdx.x + i * tx);
      if (e >= a.D) continue;
      float f[8];
      load8(pre + e, f);
      scale8(h[i], r, f);
      store8(x + e, h[i]);
    }
  }
}

template <typename T, typename TH, int V>
cudaError_t run_residual(const ResidualNormArgs& a, int tx, cudaStream_t s) {
  const auto kern = kda_residual_norm_kernel<T, TH, V>;
  if constexpr (V == 4) return mla_launch(kern, (unsigned)a.T, dim3((unsigned)tx), 0, s, a);
  static std::atomic<int> fits[17];                     // CTAs of this many warps that an SM holds
  const int ty = tx == 32 ? 4 : 1, warps = tx * ty / 32;
  int per = fits[warps].load(std::memory_order_relaxed);
  if (per == 0) {
    const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kern, tx * ty, 0);
    if (e != cudaSuccess) return e;
    fits[warps].store(per = per > 0 ? per : 1, std::memory_order_relaxed);
  }
  const int64_t need = (a.T + ty - 1) / ty, most = kSms * (int64_t)per;
  return mla_launch(kern, (unsigned)(need < most ? need : most), dim3((unsigned)tx, (unsigned)ty), 0, s, a);
}
template <typename T, typename TH>
cudaError_t run_residual_d(const ResidualNormArgs& a, cudaStream_t s) {
  const int vecs = a.D / 8;
  const auto threads = [&](int v) { return ((vecs + v - 1) / v + 31) / 32 * 32; };
  // One vector a thread for up to 256 of them, and 512 for few rows; else two, for up to 768 threads' worth, so that two CTAs share an SM; else
  // four.  One / two / four, us, h in fp32 and every part: 2048 values, 304 rows 4.5 / 4.9 / 6.5, 8192 rows 42.3 / 43.3 / 53.4; 4096 values, 304
  // rows 6.5 / 6.6 / 7.9, 456 9.2 / 7.6 / 8.7, 1024 14.7 / 15.5 / 17.8, 8192 91.6 / 86.4 / 103; two / four, 6144 values, 64 rows 5.3 / 7.0 (four walking over
  // rows as two do).
  if (vecs <= 256 || (vecs <= 512 && a.T <= 304)) return run_residual<T, TH, 1>(a, threads(1), s);
  if (vecs <= 768) return run_residual<T, TH, 2>(a, threads(2), s);
  return run_residual<T, TH, 4>(a, threads(4), s);
}

}  // namespace

cudaError_t launch_gated_norm(const GatedNormArgs& a, cudaStream_t s) {
  return a.dtype == KDA_BF16 ? run_gated_d<__nv_bfloat16>(a, s) : run_gated_d<float>(a, s);
}
cudaError_t launch_residual_norm(const ResidualNormArgs& a, cudaStream_t s) {
  if (a.dtype == KDA_F32) return run_residual_d<float, float>(a, s);
  return a.h_dtype == KDA_F32 ? run_residual_d<__nv_bfloat16, float>(a, s) : run_residual_d<__nv_bfloat16, __nv_bfloat16>(a, s);
}

}  // namespace kda
