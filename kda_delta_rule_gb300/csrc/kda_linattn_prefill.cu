// Linear attention with one decay for each head over packed sequences: the CUDA-core kernel, the scan of
// the segments' states, and the choice of kernels.
//
//   S_t = e^(g_t) S_(t-1) + k_t v_t^T,   o_t = scale S_t^T q_t
//
// CUDA-core kernel (fp32): one CTA per (segment, head, 32 columns of the state), which stays in registers; a
// thread owns four columns of every 16th row.  Tokens come in batches of 16.  With b_t the log decay summed from the
// batch's start, S_t = e^(b_t) (S_0 + sum_(j <= t) e^(-b_j) k_j v_j^T): the bracket grows by one fused multiply-add per element and
// token, and one rounded factor e^(b_16) per batch meets the state, so that a state that hardly decays keeps fp32's
// precision over tens of thousands of tokens (a factor per token, all rounded the same way for a fixed
// decay, would not).  A batch that decays by more than 2^40 takes the plain form, one factor per token, instead
// of weights that leave fp32's range.  Bound by the FMA pipe: 2 dk dv per token and head.
#include <cuda_runtime.h>

#include "../../include/kda.h"
#include "kda_common.cuh"
#include "kda_linattn.h"
#include "kda_mla.cuh"
#include "kda_tc.cuh"

namespace kda {
namespace {

constexpr int kNT = 128, kNB = 16;          // threads; tokens per batch
constexpr int kDVS = 32;                    // state columns per CTA
constexpr int kTPR = kDVS / 4, kRG = kNT / kTPR;

// The states of a segment and the pages they go to: element (i, j) of head h's state, dv columns in all.
template <int DK>
__device__ __forceinline__ void lin_store_state(float* dst, const float4 (&S)[DK / kRG], int dv, int rg) {
#pragma unroll
  for (int i = 0; i < DK / kRG; ++i) *reinterpret_cast<float4*>(dst + (int64_t)(rg + i * kRG) * dv) = S[i];
}

template <int DK, bool LOCAL>
__global__ void __launch_bounds__(kNT) kda_linattn_simt_kernel(const LinPrefillArgs a, const __grid_constant__ LinSched sched) {
  constexpr int RPT = DK / kRG;
  constexpr int NQ = kNB * DK / 4 / kNT;    // float4 of q (and of k) per thread and batch
  __shared__ __align__(16) float sk[kNB][DK], sq[kNB][DK], sv[kNB][kDVS], part[kNB][kRG][kDVS];
  __shared__ float s_in[kNB], s_out[kNB], s_end;   // weights of a token's k v^T and of its output; factor of the batch
  __shared__ int s_plain;
  mla_grid_wait();
  mla_grid_next();
  const int tid = threadIdx.x, col = 4 * (tid % kTPR), rg = tid / kTPR;
  const int slices = a.dv / kDVS;
  const int h = blockIdx.y / slices, c0 = (blockIdx.y - h * slices) * kDVS, hk = h / a.share;
  int which = blockIdx.x;
  if (LOCAL) {                              // every segment but each sequence's last: slot -> segment
    int lo = 0, hi = sched.n_seqs - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (sched.item_base[mid] - mid <= which) lo = mid; else hi = mid - 1;
    }
    which += lo;
  }
  const LinItem it = lin_item(sched, which);
  const int64_t hstate = (int64_t)DK * a.dv;
  const int64_t tile = (int64_t)rg * a.dv + c0 + col;
  float4 S[RPT];
  const float* src = nullptr;
  if (!LOCAL) {
    if (it.nth > 0) src = a.seg_state + ((int64_t)lin_slot(sched, it.place, it.nth - 1) * a.H + h) * hstate;
    else if (a.S0) src = a.S0 + ((int64_t)it.seq * a.H + h) * hstate;
  }
#pragma unroll
  for (int i = 0; i < RPT; ++i)
    S[i] = src ? *reinterpret_cast<const float4*>(src + tile + (int64_t)i * kRG * a.dv) : make_float4(0.f, 0.f, 0.f, 0.f);
  const float* q = static_cast<const float*>(a.q) + hk * DK;
  const float* k = static_cast<const float*>(a.k) + hk * DK;
  const float* v = static_cast<const float*>(a.v) + h * a.dv + c0;
  float* o = static_cast<float*>(a.o) + (int64_t)h * a.dv + c0;
  float4 nq[NQ], nk[NQ], nv;
  float ng = 0.f;
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  const auto fetch = [&](int t) {           // the batch of tokens from t of the segment
#pragma unroll
    for (int e = 0; e < NQ; ++e) {
      const int f = tid + e * kNT, s = f / (DK / 4), i = 4 * (f % (DK / 4));
      const bool in = t + s < it.n;
      if (!LOCAL) nq[e] = in ? load4(q + (it.t0 + t + s) * a.q_stride + i) : zero;
      nk[e] = in ? load4(k + (it.t0 + t + s) * a.k_stride + i) : zero;
    }
    const int s = tid / kTPR;
    nv = t + s < it.n ? load4(v + (it.t0 + t + s) * a.v_stride + col) : zero;
    if (tid < kNB) ng = t + tid < it.n ? a.g[(it.t0 + t + tid) * a.g_stride + h] : 0.f;
  };
  int64_t decay = 0;
  fetch(0);
  for (int t = 0; t < it.n; t += kNB) {
    const int n = min(kNB, it.n - t);
#pragma unroll
    for (int e = 0; e < NQ; ++e) {
      const int f = tid + e * kNT, s = f / (DK / 4), i = 4 * (f % (DK / 4));
      if (!LOCAL) *reinterpret_cast<float4*>(&sq[s][i]) = nq[e];
      *reinterpret_cast<float4*>(&sk[s][i]) = nk[e];
    }
    *reinterpret_cast<float4*>(&sv[tid / kTPR][col]) = nv;
    if (tid < 32) {                         // the batch's decays
      bool bad = false;
      const int64_t one = lin_fixed(tid < n ? ng : 0.f, &bad);
      if (bad) atomicOr(&tc::g_kda_device_error, KDA_DEVERR_GATE);
      int64_t sum = one;
#pragma unroll
      for (int w = 1; w < kNB; w <<= 1) {
        const int64_t up = __shfl_up_sync(0xffffffffu, sum, w);
        if (tid >= w) sum += up;
      }
      const int64_t all = __shfl_sync(0xffffffffu, sum, kNB - 1);
      if (decay > kLinLeast) decay += all;
      const bool plain = all < -(40ll << 32);
      if (tid < kNB) {
        s_in[tid] = plain ? exp2f(lin_float(one)) : exp2f(-lin_float(sum));
        s_out[tid] = plain ? a.scale : a.scale * exp2f(lin_float(sum));
      }
      if (tid == 0) {
        s_plain = plain;
        s_end = exp2f(lin_float(all));
      }
    }
    __syncthreads();
    if (t + kNB < it.n) fetch(t + kNB);
    if (!s_plain) {
      for (int s = 0; s < n; ++s) {
        const float f = s_in[s];
        float4 x = *reinterpret_cast<const float4*>(&sv[s][col]), acc = zero;
        x = make_float4(f * x.x, f * x.y, f * x.z, f * x.w);
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
          S[i] = f4_fma(sk[s][rg + i * kRG], x, S[i]);
          if (!LOCAL) acc = f4_fma(sq[s][rg + i * kRG], S[i], acc);
        }
        if (!LOCAL) *reinterpret_cast<float4*>(&part[s][rg][col]) = acc;
      }
      const float f = s_end;
#pragma unroll
      for (int i = 0; i < RPT; ++i) S[i] = make_float4(f * S[i].x, f * S[i].y, f * S[i].z, f * S[i].w);
    } else {
      for (int s = 0; s < n; ++s) {
        const float d = s_in[s];
        const float4 x = *reinterpret_cast<const float4*>(&sv[s][col]);
        float4 acc = zero;
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
          S[i] = f4_fma(sk[s][rg + i * kRG], x, make_float4(d * S[i].x, d * S[i].y, d * S[i].z, d * S[i].w));
          if (!LOCAL) acc = f4_fma(sq[s][rg + i * kRG], S[i], acc);
        }
        if (!LOCAL) *reinterpret_cast<float4*>(&part[s][rg][col]) = acc;
      }
    }
    __syncthreads();
    if (!LOCAL) {
      const int s = tid / kTPR;
      if (s < n) {
        float4 acc = zero;
        const float f = s_out[s];
#pragma unroll
        for (int r = 0; r < kRG; ++r) acc = f4_fma(f, *reinterpret_cast<const float4*>(&part[s][r][col]), acc);
        store4(o + (it.t0 + t + s) * (int64_t)a.H * a.dv + col, acc);
      }
      const int pos = it.nth * sched.seg_len + t + n;
      if (a.ckpt_stride > 0 && pos % a.ckpt_stride == 0) {   // a boundary is a batch's end: strides are whole chunks
        const int64_t c = (int64_t)sched.ckpt_base[it.place] + pos / a.ckpt_stride - 1;
        if (c < a.num_ckpt) {
          float* page = reinterpret_cast<float*>(a.pages + (int64_t)a.ckpt_page_ids[c] * a.page_bytes);
          lin_store_state<DK>(page + h * hstate + tile, S, a.dv, 0);
          if (blockIdx.y == 0) {
            for (int64_t e = a.H * hstate + tid; e < a.page_bytes / 4; e += kNT) page[e] = 0.f;
            if (tid == 0 && a.ckpt_pos) a.ckpt_pos[c] = pos;
          }
        }
      }
      __syncthreads();                      // s_out and part are read before the next batch's
    }
  }
  if (LOCAL) {
    const int64_t at = (int64_t)lin_slot(sched, it.place, it.nth) * a.H + h;
    lin_store_state<DK>(a.seg_state + at * hstate + tile, S, a.dv, 0);
    if (c0 == 0 && tid == 0) a.seg_decay[at] = decay;
  } else if (it.last) {
    lin_store_state<DK>(a.S_final + ((int64_t)it.seq * a.H + h) * hstate + tile, S, a.dv, 0);
  }
}

// The segments' start states from their own states: X_(p+1) = e^(G_p) X_p + L_p, X_0 = S0.  X_(p+1) takes L_p's place.  Each
// thread walks one float4 of a state along its sequence's segments.
__global__ void __launch_bounds__(128) kda_linattn_scan_kernel(const LinPrefillArgs a, const __grid_constant__ LinSched sched) {
  mla_grid_wait();
  mla_grid_next();
  const int place = blockIdx.z, h = blockIdx.y;
  const int n = sched.item_base[place + 1] - sched.item_base[place] - 1;
  const int64_t hstate = (int64_t)a.dk * a.dv;
  const int64_t e = 4 * ((int64_t)blockIdx.x * blockDim.x + threadIdx.x);
  if (e >= hstate) return;
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  if (a.S0) x = *reinterpret_cast<const float4*>(a.S0 + ((int64_t)sched.seq[place] * a.H + h) * hstate + e);
  const int64_t first = (int64_t)lin_slot(sched, place, 0) * a.H + h;
#pragma unroll 4
  for (int p = 0; p < n; ++p) {
    const int64_t at = first + (int64_t)p * a.H;
    float4* s = reinterpret_cast<float4*>(a.seg_state + at * hstate + e);
    const float f = exp2f(lin_float(a.seg_decay[at]));
    const float4 l = *s;
    x = make_float4(fmaf(f, x.x, l.x), fmaf(f, x.y, l.y), fmaf(f, x.z, l.z), fmaf(f, x.w, l.w));
    *s = x;
  }
}

template <int DK>
cudaError_t run_simt(const LinPrefillArgs& a, const LinSched& sched, cudaStream_t s) {
  const dim3 grid((unsigned)sched.n_items, (unsigned)(a.H * (a.dv / kDVS)));
  const int local = sched.n_items - sched.n_seqs;
  if (local > 0) {
    if (const cudaError_t e = mla_launch(kda_linattn_simt_kernel<DK, true>, dim3((unsigned)local, grid.y), kNT, 0, s, a, sched)) return e;
    if (const cudaError_t e = launch_linattn_scan(a, sched, s)) return e;
  }
  return mla_launch(kda_linattn_simt_kernel<DK, false>, grid, kNT, 0, s, a, sched);
}

}  // namespace

cudaError_t launch_linattn_scan(const LinPrefillArgs& a, const LinSched& sched, cudaStream_t s) {
  int split = 0;                            // sequences of several segments come first
  while (split < sched.n_seqs && sched.item_base[split + 1] - sched.item_base[split] > 1) ++split;
  return mla_launch(kda_linattn_scan_kernel, dim3((unsigned)((a.dk * a.dv / 4 + 127) / 128), (unsigned)a.H, (unsigned)split), 128, 0, s, a, sched);
}

cudaError_t launch_linattn_prefill(const LinPrefillArgs& a, const LinSched& sched, cudaStream_t s) {
  if (a.dtype == KDA_BF16 && a.T > 0)       // without a token, states are copied: either kernel
    return a.dk == 32 ? launch_linattn_tc_32(a, sched, s) : a.dk == 64 ? launch_linattn_tc_64(a, sched, s) : launch_linattn_tc_128(a, sched, s);
  return a.dk == 32 ? run_simt<32>(a, sched, s) : a.dk == 64 ? run_simt<64>(a, sched, s) : run_simt<128>(a, sched, s);
}

int read_and_clear_linattn_errors(int* flags) {
  int word = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&word, tc::g_kda_device_error, sizeof(int));
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(tc::g_kda_device_error, &zero, sizeof(int));
  *flags |= word;
  int st = (int)e;
  if (st == 0) st = read_and_clear_linattn_step_errors(flags);
  if (st == 0) st = read_and_clear_linattn_tc_32_errors(flags);
  if (st == 0) st = read_and_clear_linattn_tc_64_errors(flags);
  if (st == 0) st = read_and_clear_linattn_tc_128_errors(flags);
  return st;
}

}  // namespace kda
