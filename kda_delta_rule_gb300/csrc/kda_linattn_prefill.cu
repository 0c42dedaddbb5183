// Linear attention with one decay for each head over packed sequences: the CUDA-core kernel, the scan of
// the segments' states, and the choice of kernels.
//
//   S_t = e^(g_t) S_(t-1) + k_t v_t^T,   o_t = scale S_t^T q_t
//
// CUDA-core kernel (fp32, and bf16 sequences of a few tokens): one CTA per (segment, head, 32 columns of the state), which stays in registers; a
// thread owns four columns of runs of four rows.  Tokens come in batches of 16.  With b_t the log decay summed from some earlier token,
// S_t = e^(b_t) (S_0 + sum_(j <= t) e^(-b_j) k_j v_j^T): the bracket grows by one fused multiply-add per element and token, and is
// multiplied out only before a batch that would take b past -40 (in log2 units).  So a state that hardly decays meets few rounded factors
// and keeps fp32's precision over tens of thousands of tokens; a factor per token or batch, rounded the same way every time for a fixed
// decay, would not.  The bracket is up to 2^40 of the state: what it holds may be 2^85 in size, with some room for sums.  A batch that decays
// by more than 2^40 takes the plain form, one factor per token, which is slower (8192 tokens of 32 heads of 128 x 128: 1140 us, the
// bracket 850 to 880; with room for 2^24 alone, heads that decay by 1 to 1.7 a token would take it too).  Bound by the FMA pipe: 2 dk dv
// per token and head; with few CTAs by the latency of a token's steps.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/kda.h"
#include "kda_common.cuh"
#include "kda_linattn.h"
#include "kda_mla.cuh"
#include "kda_tc.cuh"

namespace kda {
namespace {

constexpr int kNT = 128, kNB = kLinBatch;   // threads with a part of the state; tokens per batch
constexpr int kDVS = 32;                    // state columns per CTA
constexpr int kTPR = kDVS / 4, kRG = kNT / kTPR;
constexpr int64_t kRoom = 40ll << kLinBits; // log2 units that the bracket may stand above the state

// Rows of a thread's part of the state: runs of four (two for 32 rows), so that their keys and queries are read at once.
template <int DK>
__device__ __forceinline__ int lin_row(int rg, int i) {
  constexpr int RUN = DK / kRG < 4 ? DK / kRG : 4;
  return RUN * rg + i % RUN + i / RUN * (RUN * kRG);
}
template <int N>
__device__ __forceinline__ void lds_run(const float* p, float (&v)[N]) {
  if constexpr (N == 2) {
    const float2 x = *reinterpret_cast<const float2*>(p);
    v[0] = x.x; v[1] = x.y;
  } else {
    const float4 x = *reinterpret_cast<const float4*>(p);
    v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
  }
}

// LOCAL: the segments' states from zero, without outputs.  A fifth warp works out the decays of the next batch.
// `second`: follows another kernel of the call, which has waited for what came before it, and need not wait for that kernel but to end.
template <int DK, typename T, bool LOCAL>
__global__ void __launch_bounds__(kNT + 32) kda_linattn_simt_kernel(const LinPrefillArgs a, const __grid_constant__ LinSched sched, int second) {
  constexpr int RPT = DK / kRG, RUN = RPT < 4 ? RPT : 4;
  constexpr int NQ = kNB * DK / 4 / kNT;    // float4 of q (and of k) per thread and batch
  __shared__ __align__(16) float sk[kNB][DK], sq[kNB][DK], sv[kNB][kDVS], part[kNB][kRG][kDVS];
  // per batch: weights of a token's k v^T and of its output; a factor of the bracket before the batch (0: none), and the one that
  // makes it the state after the batch
  __shared__ float s_in[2][kNB], s_out[2][kNB], s_pre[2], s_now[2];
  __shared__ int s_plain[2];
  if (!second) mla_grid_wait();
  mla_grid_next();
  const int tid = threadIdx.x, col = 4 * (tid % kTPR), rg = tid / kTPR;
  const int slices = a.dv / kDVS, ctas = a.H * slices;
  int which = blockIdx.x / (unsigned)ctas;
  const int part_of = blockIdx.x - which * ctas, h = part_of / slices, c0 = (part_of - h * slices) * kDVS, hk = h / a.share;
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
  const bool decays = tid >= kNT;
  float4 S[RPT];
  const float* src = nullptr;
  if (!LOCAL && !decays) {
    if (it.nth > 0) src = a.seg_state + ((int64_t)lin_slot(sched, it.place, it.nth - 1) * a.H + h) * hstate;
    else if (a.S0) src = a.S0 + ((int64_t)it.seq * a.H + h) * hstate;
  }
#pragma unroll
  for (int i = 0; i < RPT; ++i)
    S[i] = src ? *reinterpret_cast<const float4*>(src + (int64_t)lin_row<DK>(rg, i) * a.dv + c0 + col) : make_float4(0.f, 0.f, 0.f, 0.f);
  float now = 1.f;
  const auto store = [&](float* dst) {      // the state, element (i, j) of the head's
#pragma unroll
    for (int i = 0; i < RPT; ++i)
      *reinterpret_cast<float4*>(dst + (int64_t)lin_row<DK>(rg, i) * a.dv + c0 + col) = make_float4(now * S[i].x, now * S[i].y, now * S[i].z, now * S[i].w);
  };
  const T* q = reinterpret_cast<const T*>(a.q) + hk * DK;
  const T* k = reinterpret_cast<const T*>(a.k) + hk * DK;
  const T* v = reinterpret_cast<const T*>(a.v) + h * a.dv + c0;
  T* o = reinterpret_cast<T*>(a.o) + (int64_t)h * a.dv + c0;
  float4 nq[NQ], nk[NQ], nv;
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
  };
  int64_t decay = 0, since = 0;             // log decays of the segment; since the bracket was last multiplied out
  const auto work_out = [&](int t, float g) {   // the decays of the batch from t, one token a lane
    const int lane = tid - kNT, p = (t / kNB) & 1;
    bool bad = false;
    const int64_t one = lin_fixed(g, &bad);
    if (bad) atomicOr(&tc::g_kda_device_error, KDA_DEVERR_GATE);
    int64_t sum = one;
#pragma unroll
    for (int w = 1; w < kNB; w <<= 1) {
      const int64_t up = __shfl_up_sync(0xffffffffu, sum, w);
      if (lane >= w) sum += up;
    }
    const int64_t all = __shfl_sync(0xffffffffu, sum, kNB - 1);
    if (decay > kLinLeast) decay += all;
    const bool plain = all < -kRoom, pre = since != 0 && since + all < -kRoom;
    const float before = exp2f(lin_float(since));
    if (pre) since = 0;
    if (lane < kNB) {
      s_in[p][lane] = plain ? exp2f(lin_float(one)) : exp2f(-lin_float(since + sum));
      s_out[p][lane] = plain ? 1.f : exp2f(lin_float(since + sum));
    }
    if (!plain) since += all;
    if (lane == 0) {
      s_plain[p] = plain;
      s_pre[p] = pre ? before : 0.f;
      s_now[p] = exp2f(lin_float(since));
    }
  };
  const auto log_decay = [&](int t) {       // of this lane's token in the batch from t
    const int s = tid - kNT;
    return s < kNB && t + s < it.n ? a.g[(it.t0 + t + s) * a.g_stride + h] : 0.f;
  };
  float ng = 0.f;
  if (decays) {
    work_out(0, log_decay(0));
    ng = log_decay(kNB);
  } else {
    fetch(0);
  }
  for (int t = 0; t < it.n; t += kNB) {
    const int n = min(kNB, it.n - t), p = (t / kNB) & 1;
    if (!decays) {
#pragma unroll
      for (int e = 0; e < NQ; ++e) {
        const int f = tid + e * kNT, s = f / (DK / 4), i = 4 * (f % (DK / 4));
        if (!LOCAL) *reinterpret_cast<float4*>(&sq[s][i]) = nq[e];
        *reinterpret_cast<float4*>(&sk[s][i]) = nk[e];
      }
      *reinterpret_cast<float4*>(&sv[tid / kTPR][col]) = nv;
    }
    __syncthreads();
    if (decays) {
      if (t + kNB < it.n) work_out(t + kNB, ng);
      ng = log_decay(t + 2 * kNB);
    } else {
      if (t + kNB < it.n) fetch(t + kNB);
      const bool plain = s_plain[p];
      const float pre = s_pre[p];
      now = s_now[p];
      if (pre != 0.f) {
#pragma unroll
        for (int i = 0; i < RPT; ++i) S[i] = make_float4(pre * S[i].x, pre * S[i].y, pre * S[i].z, pre * S[i].w);
      }
      const auto token = [&](int s) {
        const float f = s_in[p][s], d = plain ? f : 1.f;
        float4 x = *reinterpret_cast<const float4*>(&sv[s][col]), acc = zero;
        if (!plain) x = make_float4(f * x.x, f * x.y, f * x.z, f * x.w);
#pragma unroll
        for (int i = 0; i < RPT; i += RUN) {
          float kk[RUN], qq[RUN];
          lds_run<RUN>(&sk[s][lin_row<DK>(rg, i)], kk);
          if (!LOCAL) lds_run<RUN>(&sq[s][lin_row<DK>(rg, i)], qq);
#pragma unroll
          for (int r = 0; r < RUN; ++r) {
            if (plain) S[i + r] = make_float4(d * S[i + r].x, d * S[i + r].y, d * S[i + r].z, d * S[i + r].w);
            S[i + r] = f4_fma(kk[r], x, S[i + r]);
            if (!LOCAL) acc = f4_fma(qq[r], S[i + r], acc);
          }
        }
        if (!LOCAL) *reinterpret_cast<float4*>(&part[s][rg][col]) = acc;
      };
      if (n == kNB && !plain) {
#pragma unroll 4
        for (int s = 0; s < kNB; ++s) token(s);
      } else {
        for (int s = 0; s < n; ++s) token(s);
      }
    }
    __syncthreads();
    if (!LOCAL && !decays) {
      const int s = tid / kTPR;
      if (s < n) {
        float4 acc = zero;
        const float f = s_out[p][s];
#pragma unroll
        for (int r = 0; r < kRG; ++r) acc = f4_fma(f, *reinterpret_cast<const float4*>(&part[s][r][col]), acc);
        const float c = a.scale;                // last: its product with the weight could leave fp32's range
        store4(o + (it.t0 + t + s) * (int64_t)a.H * a.dv + col, make_float4(c * acc.x, c * acc.y, c * acc.z, c * acc.w));
      }
      const int pos = it.nth * sched.seg_len + t + n;
      if (a.ckpt_stride > 0 && pos % a.ckpt_stride == 0) {   // a boundary is a batch's end: strides are whole chunks
        const int64_t c = (int64_t)sched.ckpt_base[it.place] + pos / a.ckpt_stride - 1;
        if (c < a.num_ckpt) {
          float* page = reinterpret_cast<float*>(a.pages + (int64_t)a.ckpt_page_ids[c] * a.page_bytes);
          store(page + h * hstate);
          if (part_of == 0) {
            for (int64_t e = a.H * hstate + tid; e < a.page_bytes / 4; e += kNT) page[e] = 0.f;
            if (tid == 0 && a.ckpt_pos) a.ckpt_pos[c] = pos;
          }
        }
      }
    }
  }
  if (LOCAL) {
    const int64_t at = (int64_t)lin_slot(sched, it.place, it.nth) * a.H + h;
    if (!decays) store(a.seg_state + at * hstate);
    if (c0 == 0 && tid == kNT) a.seg_decay[at] = lin_factor(decay);
  } else if (it.last && !decays) {
    store(a.S_final + ((int64_t)it.seq * a.H + h) * hstate);
  }
  if (second) mla_grid_wait();
}

// The segments' start states from their own states: X_(p+1) = e^(G_p) X_p + L_p, X_0 = S0.  X_(p+1) takes L_p's place.  Each
// thread walks two values of a state along its sequence's segments, eight segments' loads under way together (31 segments of four heads:
// one after another 19 us).
__global__ void __launch_bounds__(128) kda_linattn_scan_kernel(const LinPrefillArgs a, const __grid_constant__ LinSched sched) {
  mla_grid_wait();
  mla_grid_next();
  constexpr int AT = 8;
  const int place = blockIdx.z, h = blockIdx.y;
  const int n = sched.item_base[place + 1] - sched.item_base[place] - 1;
  const int64_t hstate = (int64_t)a.dk * a.dv;
  const int64_t e = 2 * ((int64_t)blockIdx.x * blockDim.x + threadIdx.x);
  if (e >= hstate) return;
  float2 x = make_float2(0.f, 0.f);
  if (a.S0) x = load2(a.S0 + ((int64_t)sched.seq[place] * a.H + h) * hstate + e);
  const int64_t first = (int64_t)lin_slot(sched, place, 0) * a.H + h;
  for (int p = 0; p < n; p += AT) {
    float2 l[AT], f[AT];
#pragma unroll
    for (int i = 0; i < AT; ++i)
      if (p + i < n) {
        const int64_t at = first + (int64_t)(p + i) * a.H;
        l[i] = load2(a.seg_state + at * hstate + e);
        f[i] = a.seg_decay[at];
      }
#pragma unroll
    for (int i = 0; i < AT; ++i)
      if (p + i < n) {
        x = make_float2(fmaf(f[i].x, x.x, fmaf(f[i].y, x.x, l[i].x)), fmaf(f[i].x, x.y, fmaf(f[i].y, x.y, l[i].y)));
        store2(a.seg_state + (first + (int64_t)(p + i) * a.H) * hstate + e, x);
      }
  }
}

// The outputs times a power of two.
__global__ void __launch_bounds__(256) kda_linattn_scale_kernel(__nv_bfloat16* o, int64_t n, float f) {
  mla_grid_wait();
  mla_grid_next();
  for (int64_t e = 4 * ((int64_t)blockIdx.x * 256 + threadIdx.x); e < n; e += 4 * 256 * (int64_t)gridDim.x) {
    const float4 x = load4(o + e);
    store4(o + e, make_float4(f * x.x, f * x.y, f * x.z, f * x.w));
  }
}

template <int DK, typename T>
cudaError_t run_simt(const LinPrefillArgs& a, const LinSched& sched, int second, cudaStream_t s) {
  const int64_t ctas = (int64_t)a.H * (a.dv / kDVS), local = sched.n_items - sched.n_seqs;
  if constexpr (sizeof(T) == 4) {           // bf16: short sequences, of one segment
    if (local > 0) {
      if (const cudaError_t e = mla_launch(kda_linattn_simt_kernel<DK, T, true>, (unsigned)(local * ctas), kNT + 32, 0, s, a, sched, 0)) return e;
      if (const cudaError_t e = launch_linattn_scan(a, sched, s)) return e;
    }
  }
  return mla_launch(kda_linattn_simt_kernel<DK, T, false>, (unsigned)(sched.n_items * ctas), kNT + 32, 0, s, a, sched, second);
}
template <typename T>
cudaError_t run_simt_dk(const LinPrefillArgs& a, const LinSched& sched, int second, cudaStream_t s) {
  return a.dk == 32 ? run_simt<32, T>(a, sched, second, s) : a.dk == 64 ? run_simt<64, T>(a, sched, second, s) : run_simt<128, T>(a, sched, second, s);
}

}  // namespace

cudaError_t launch_linattn_scale(void* o, int64_t n, float f, cudaStream_t s) {
  if (n == 0) return cudaSuccess;           // a multiple of 32 otherwise
  const int64_t ctas = (n + 1023) / 1024;
  return mla_launch(kda_linattn_scale_kernel, (unsigned)(ctas < 8 * kSms ? ctas : 8 * kSms), 256, 0, s, static_cast<__nv_bfloat16*>(o), n, f);
}

cudaError_t launch_linattn_scan(const LinPrefillArgs& a, const LinSched& sched, cudaStream_t s) {
  int split = 0;                            // sequences of several segments come first
  while (split < sched.n_seqs && sched.item_base[split + 1] - sched.item_base[split] > 1) ++split;
  return mla_launch(kda_linattn_scan_kernel, dim3((unsigned)((a.dk * a.dv / 2 + 127) / 128), (unsigned)a.H, (unsigned)split), 128, 0, s, a, sched);
}

// bf16: the tensor cores take the longer sequences, a chunk of 128 tokens at a time whatever is in it; for sequences of a few tokens, or small
// heads, several CTAs of the CUDA-core kernel share an SM, and they run beside the last of the others.  768 (sequence, head)s on the
// tensor cores and the CUDA cores, us: heads of 128 x 128, 40 tokens 60 / 91; 128 x 64, 40 tokens 50 / 44, 60 tokens 50 / 61; 32 x 32, 90 tokens
// 39 / 27.
int short_tokens(int dk, int dv) {
  const int n = 400000 / (dk * dv);
  return n < kLinChunk ? n : kLinChunk;
}

cudaError_t launch_linattn_prefill(const LinPrefillArgs& a, LinSched& sched, cudaStream_t s) {
  if (a.dtype == KDA_F32) return run_simt_dk<float>(a, sched, 0, s);
  int m = sched.n_seqs;                     // sequences are in the order of their lengths
  while (m > 0 && sched.len[m - 1] <= short_tokens(a.dk, a.dv)) --m;
  const int n = sched.n_seqs, items = sched.n_items;
  if (m > 0) {
    sched.n_seqs = m;
    sched.n_items = sched.item_base[m];
    const cudaError_t e = a.dk == 32 ? launch_linattn_tc_32(a, sched, s) : a.dk == 64 ? launch_linattn_tc_64(a, sched, s) : launch_linattn_tc_128(a, sched, s);
    if (e != cudaSuccess || m == n) return e;
    const int base = sched.item_base[m];    // the others to the front
    for (int p = m; p < n; ++p) {
      sched.seq[p - m] = sched.seq[p];
      sched.start[p - m] = sched.start[p];
      sched.len[p - m] = sched.len[p];
      sched.ckpt_base[p - m] = sched.ckpt_base[p];
      sched.item_base[p - m] = sched.item_base[p] - base;
    }
    sched.item_base[n - m] = items - base;
    sched.n_seqs = n - m;
    sched.n_items = items - base;
  }
  return run_simt_dk<__nv_bfloat16>(a, sched, m > 0, s);
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
