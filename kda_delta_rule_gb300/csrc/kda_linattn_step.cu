// Linear attention with one decay for each head, one or a few tokens per sequence:
//
//   S_t = e^(g_t) S_(t-1) + k_t v_t^T,   o_t = scale S_t^T q_t
//
// One CTA per (sequence, head, slice of the state's columns): the columns of S are independent given q, k
// and g, and a CTA keeps its slice in registers over all tokens of the call, so a state is read once and written
// once whatever the number of tokens.  Bound by HBM, 2 dk dv 4 bytes per head: 256 sequences of 32 heads of 128 x 128 in 161 us, 99% of the
// measured copy rate.  A thread owns four consecutive
// columns of four consecutive rows, and so on (their keys and queries are then read at once); the state's loads are issued first, the tokens'
// rows and decays are staged while they are under way.  Each token's outputs are sums over the row groups, which meet in
// shared memory after the last token.  Where a state decays little, it is taken by e^g - 1, which fp32 holds better than e^g, and added to itself: a
// factor rounded the same way for every token of a fixed decay was off by 7e-4 of the state after 16384 tokens.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/kda.h"
#include "kda_common.cuh"
#include "kda_linattn.h"
#include "kda_mla.cuh"
#include "kda_tc.cuh"

namespace kda {
namespace {

template <int DK, int DVS>
struct LinStepCfg {
  static constexpr int NT = DK * DVS / 16 < 64 ? 64 : (DK * DVS / 16 > 256 ? 256 : DK * DVS / 16);
  static constexpr int TPR = DVS / 4;                  // threads per row
  static constexpr int RG = NT / TPR;                  // row groups
  static constexpr int RPT = DK / RG;                  // rows per thread
  static_assert(RPT % 4 == 0, "runs of four rows");
};
template <int DK, int DVS>
constexpr size_t lin_step_smem(int steps) {
  return (size_t)steps * (2 * DK + DVS + 4 + LinStepCfg<DK, DVS>::RG * DVS) * sizeof(float);
}

template <int DK, int DVS, typename T>
__global__ void __launch_bounds__((LinStepCfg<DK, DVS>::NT), (512 / LinStepCfg<DK, DVS>::NT)) kda_linattn_step_kernel(const LinStepArgs a) {
  using C = LinStepCfg<DK, DVS>;
  constexpr int NT = C::NT, TPR = C::TPR, RG = C::RG, RPT = C::RPT;
  extern __shared__ float4 smem4[];
  float* sk = reinterpret_cast<float*>(smem4);         // [steps][DK]
  float* sq = sk + a.steps * DK;                       // [steps][DK]
  float* sv = sq + a.steps * DK;                       // [steps][DVS]
  float2* sd = reinterpret_cast<float2*>(sv + a.steps * DVS);   // [steps], and as much again: e^g - 1 and 1, or e^g and 0
  float* part = sv + a.steps * (DVS + 4);              // [steps][RG][DVS]
  mla_grid_wait();
  mla_grid_next();
  const int tid = threadIdx.x, col = 4 * (tid % TPR), rg = tid / TPR;
  const int dv = a.dv, slices = dv / DVS;
  const unsigned head = blockIdx.x / (unsigned)slices, c0 = (blockIdx.x - head * slices) * DVS;
  const int b = head / (unsigned)a.H, h = head - (unsigned)b * a.H;
  const int64_t from = a.slot_in ? a.slot_in[b] : b, to = a.slot_out ? a.slot_out[b] : from;
  const bool live = from >= 0 && from < a.n_slots && (!a.S_out || (to >= 0 && to < a.n_slots));
  float4 S[RPT];
  if (live) {
    const float* src = a.S_in + ((from * a.H + h) * DK) * dv + c0 + col;
#pragma unroll
    for (int i = 0; i < RPT; ++i) S[i] = ld_stream(src + (int64_t)(4 * rg + i % 4 + i / 4 * (4 * RG)) * dv);
  }
  const int n = live ? (a.n_accepted ? max(0, min(a.n_accepted[b], a.steps)) : a.steps) : 0;
  const int hk = h / a.share;
  for (int e = tid; e < n * (DK / 4); e += NT) {
    const int s = e / (DK / 4), i = 4 * (e - s * (DK / 4));
    const int64_t row = (int64_t)s * a.B + b;
    const float4 kk = load4(reinterpret_cast<const T*>(a.k) + row * a.k_stride + hk * DK + i);
    const float4 qq = load4(reinterpret_cast<const T*>(a.q) + row * a.q_stride + hk * DK + i);
    *reinterpret_cast<float4*>(sk + s * DK + i) = kk;
    *reinterpret_cast<float4*>(sq + s * DK + i) = qq;
  }
  for (int e = tid; e < n * (DVS / 4); e += NT) {
    const int s = e / (DVS / 4), i = 4 * (e - s * (DVS / 4));
    const float4 x = load4(reinterpret_cast<const T*>(a.v) + ((int64_t)s * a.B + b) * a.v_stride + (int64_t)h * dv + c0 + i);
    *reinterpret_cast<float4*>(sv + s * DVS + i) = x;
  }
  for (int s = tid; s < n; s += NT) {
    const float g = a.g[((int64_t)s * a.B + b) * a.g_stride + h];
    if (!(g <= 0.f)) atomicOr(&tc::g_kda_device_error, KDA_DEVERR_GATE);
    sd[s] = g >= -0.17f && g <= 0.f ? make_float2(lin_near_one(g), 1.f) : make_float2(expf(g), 0.f);
  }
  __syncthreads();
  for (int s = 0; s < n; ++s) {
    const float2 f = sd[s];
    const float d = f.x;
    const float4 x = *reinterpret_cast<const float4*>(sv + s * DVS + col);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    const auto token = [&](auto decayed) {
#pragma unroll
      for (int i = 0; i < RPT; i += 4) {
        const int row = s * DK + 4 * rg + i * RG;
        const float4 k4 = *reinterpret_cast<const float4*>(sk + row), q4 = *reinterpret_cast<const float4*>(sq + row);
        const float kk[4] = {k4.x, k4.y, k4.z, k4.w}, qq[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          S[i + r] = f4_fma(kk[r], x, decayed(S[i + r]));
          acc = f4_fma(qq[r], S[i + r], acc);
        }
      }
    };
    if (f.y != 0.f) token([d](float4 y) { return f4_fma(d, y, y); });
    else token([d](float4 y) { return make_float4(d * y.x, d * y.y, d * y.z, d * y.w); });
    *reinterpret_cast<float4*>(part + (s * RG + rg) * DVS + col) = acc;
  }
  if (live && a.S_out) {
    float* dst = a.S_out + ((to * a.H + h) * DK) * dv + c0 + col;
#pragma unroll
    for (int i = 0; i < RPT; ++i) st_stream(dst + (int64_t)(4 * rg + i % 4 + i / 4 * (4 * RG)) * dv, S[i]);
  }
  __syncthreads();
  T* o = reinterpret_cast<T*>(a.o) + ((int64_t)b * a.H + h) * dv + c0;
  for (int e = tid; e < a.steps * TPR; e += NT) {
    const int s = e / TPR, c = 4 * (e - s * TPR);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (s < n) {
#pragma unroll
      for (int r = 0; r < RG; ++r) acc = f4_fma(1.f, *reinterpret_cast<const float4*>(part + (s * RG + r) * DVS + c), acc);
      acc = make_float4(a.scale * acc.x, a.scale * acc.y, a.scale * acc.z, a.scale * acc.w);
    }
    store4(o + (int64_t)s * a.B * a.H * dv + c, acc);
  }
}

template <int DK, int DVS, typename T>
cudaError_t run(const LinStepArgs& a, cudaStream_t s) {
  static std::atomic<uint64_t> allowed{0};
  const size_t smem = lin_step_smem<DK, DVS>(a.steps);
  const auto kern = kda_linattn_step_kernel<DK, DVS, T>;
  if (smem > 48 * 1024) {
    const cudaError_t e = mla_allow_smem(kern, (int)lin_step_smem<DK, DVS>(KDA_MAX_DRAFT), allowed);
    if (e != cudaSuccess) return e;
  }
  const unsigned grid = (unsigned)((int64_t)a.B * a.H * (a.dv / DVS));
  return mla_launch(kern, grid, LinStepCfg<DK, DVS>::NT, smem, s, a);
}

template <int DK, typename T>
cudaError_t run_dk(const LinStepArgs& a, cudaStream_t s) {
  // Few heads: slices of 32 columns, so that a state's latency is spread over several SMs; many: whole rows, whose tokens are staged once.
  // Slices / whole rows, us, one token, 128 x 128: 32 heads 3.3 / 4.2, 96 (384 slices) 4.8 / 5.2, 128 6.4 / 5.6, 1024 27.6 / 23.6; 128 x 64: 192 heads
  // (384 slices) 4.8 / 5.1, 256 6.4 / 5.6.  Smaller states: within a tenth of one another from there on.
  const bool narrow = (int64_t)a.B * a.H * (a.dv / 32) < 512;
  if (a.dv == 32 || narrow) return run<DK, 32, T>(a, s);
  return a.dv == 64 ? run<DK, 64, T>(a, s) : run<DK, 128, T>(a, s);
}
template <typename T>
cudaError_t run_t(const LinStepArgs& a, cudaStream_t s) {
  return a.dk == 32 ? run_dk<32, T>(a, s) : a.dk == 64 ? run_dk<64, T>(a, s) : run_dk<128, T>(a, s);
}

}  // namespace

cudaError_t launch_linattn_step(const LinStepArgs& a, cudaStream_t s) {
  return a.dtype == KDA_BF16 ? run_t<__nv_bfloat16>(a, s) : run_t<float>(a, s);
}

int read_and_clear_linattn_step_errors(int* flags) {
  int word = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&word, tc::g_kda_device_error, sizeof(int));
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(tc::g_kda_device_error, &zero, sizeof(int));
  *flags |= word;
  return (int)e;
}

}  // namespace kda
