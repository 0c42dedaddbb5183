// Linear attention with one decay for each head (kda_linattn_step, kda_linattn_prefill): arguments of
// its kernels and the division of prefill work.  Validated by kda_linattn.cpp.
//
//   S_t = e^(g_t) S_(t-1) + k_t v_t^T,   o_t = scale S_t^T q_t
//
// A packed sequence is cut into segments of whole chunks (kLinChunk tokens, fp32: kLinBatch, counted from its first one); a
// (segment, head) is one CTA's work.  Sequences of one segment need one pass.  Where the heads are too few to
// fill the GPU, longer sequences get several segments: a first pass computes each segment's state from
// zero (but the last one's), a scan turns those into the segments' start states, and the pass with the outputs then runs
// all segments at once.  The first pass reads k and v a second time, which is what the split costs.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace kda {

struct LinStepArgs {
  const float* S_in;                  // [n_slots][H][dk][dv]
  float* S_out;                       // same, or nullptr: states are not written
  const int32_t *slot_in, *slot_out;  // [B] or nullptr (row b uses slot b)
  const int32_t* n_accepted;          // [B] or nullptr (all steps)
  int64_t n_slots;
  const void *q, *k, *v;              // [steps * B] rows, *_stride elements apart
  int64_t q_stride, k_stride, v_stride;
  const float* g;                     // [steps * B] rows of H, g_stride apart (0: one row for all)
  int64_t g_stride;
  void* o;                            // [steps][B][H][dv]
  int steps, B, H, share, dk, dv, dtype;   // share: heads per q / k head
  float scale;
};
cudaError_t launch_linattn_step(const LinStepArgs& a, cudaStream_t s);
int read_and_clear_linattn_step_errors(int* flags);

constexpr int kLinChunk = 128;        // tokens per chunk
constexpr int kLinBatch = 16;         // tokens per batch of the CUDA-core kernel
constexpr int kLinMaxSeqs = 1024;     // sequences per launch

// Sequences of one launch in the order in which their segments are handed out (longest first), by value.
struct LinSched {
  int32_t n_seqs, n_items, seg_len;   // segments in all; tokens per segment (whole chunks)
  int32_t seq[kLinMaxSeqs];           // place in the order -> sequence (of this launch)
  int32_t start[kLinMaxSeqs];         // first token
  int32_t len[kLinMaxSeqs];
  int32_t ckpt_base[kLinMaxSeqs];     // first checkpoint
  int32_t item_base[kLinMaxSeqs + 1]; // first segment
};

struct LinPrefillArgs {
  const float* S0;                    // [n][H][dk][dv] or nullptr, offset to this launch's sequences
  float* S_final;
  const void *q, *k, *v;              // T rows, *_stride elements apart
  int64_t q_stride, k_stride, v_stride;
  const float* g;
  int64_t g_stride;
  void* o;                            // [T][H][dv]
  unsigned char* pages;
  int64_t page_bytes;
  const int32_t* ckpt_page_ids;
  int32_t* ckpt_pos;
  int64_t num_ckpt;
  int64_t T;
  int H, share, dk, dv, dtype, ckpt_stride;
  float scale;                        // bf16: within 2^-20 and 2^20, as a part of weights of up to 2^100
  float* seg_state;                   // workspace: [n_items - n_seqs][H][dk][dv], the segments' states, then start states
  float2* seg_decay;                  // workspace: [n_items - n_seqs][H] decays of the segments, each as the sum of two numbers
};
// Segments for these sequences (lengths of one launch, sorted longest first); n_sm CTAs run at a time.
int lin_seg_len(const int32_t* len, int n, int H, int dv, int dtype, int n_sm);
cudaError_t launch_linattn_prefill(const LinPrefillArgs& a, LinSched& sched, cudaStream_t s);   // sched is used up
cudaError_t launch_linattn_scale(void* o, int64_t n, float f, cudaStream_t s);   // n bf16 values times f, a power of two
cudaError_t launch_linattn_scan(const LinPrefillArgs& a, const LinSched& sched, cudaStream_t s);
int read_and_clear_linattn_errors(int* flags);
// bf16 on the tensor cores, one source file for each dk (kda_linattn_tc.cuh)
cudaError_t launch_linattn_tc_32(const LinPrefillArgs& a, const LinSched& sched, cudaStream_t s);
cudaError_t launch_linattn_tc_64(const LinPrefillArgs& a, const LinSched& sched, cudaStream_t s);
cudaError_t launch_linattn_tc_128(const LinPrefillArgs& a, const LinSched& sched, cudaStream_t s);
int read_and_clear_linattn_tc_32_errors(int* flags);
int read_and_clear_linattn_tc_64_errors(int* flags);
int read_and_clear_linattn_tc_128_errors(int* flags);

#ifdef __CUDACC__

// Where segment `item` lies: its sequence's place in the order, its number in the sequence, tokens [t0, t0 + n) of it.
struct LinItem {
  int place, seq, nth, n, len;
  int64_t t0, first;                  // first: the sequence's first token
  bool last;
};
__device__ __forceinline__ LinItem lin_item(const LinSched& s, int item) {
  int lo = 0, hi = s.n_seqs - 1;      // the last place whose first segment is not behind `item`
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s.item_base[mid] <= item) lo = mid; else hi = mid - 1;
  }
  LinItem r;
  r.place = lo;
  r.seq = s.seq[lo];
  r.nth = item - s.item_base[lo];
  r.len = s.len[lo];
  const int at = r.nth * s.seg_len;
  r.n = min(s.seg_len, r.len - at);
  r.first = s.start[lo];
  r.t0 = r.first + at;
  r.last = item + 1 == s.item_base[lo + 1];
  return r;
}
// Workspace slot of segment `nth` of the sequence at `place` (every segment but a sequence's last has one).
__device__ __forceinline__ int lin_slot(const LinSched& s, int place, int nth) { return s.item_base[place] - place + nth; }

// A log decay in log2 units, as a fixed-point number (2^-44): sums of them are exact, so the difference of two
// sums is good to fp32 however long the chunk has decayed, and what a token's rounding leaves is nothing over a million of them (2^-32 were
// not enough: fixed decays of 1e-10 were off by half, a state by 6e-6 after 131072 tokens).  Below -256 (also -infinity) counts as -256: such a
// token's 2^-256 is zero in fp32.  Positive or NaN decays are outside the contract (*bad).
constexpr int kLinBits = 44;
__device__ __forceinline__ int64_t lin_fixed(float g, bool* bad) {
  if (!(g <= 0.f)) *bad = true;
  return __float2ll_rn(fmaxf(g * 1.4426950408889634f, -256.f) * 0x1p44f);
}
constexpr int64_t kLinLeast = -(1ll << 60);   // sums over many tokens stop below this, 2^16 units (a step of 64 tokens adds 2^58; they are zero as factors long before)
// Its power of two as the sum of two fp32 numbers: a factor that a state meets at every chunk's or segment's end, rounded the same way
// for a fixed decay, would otherwise add up over some hundred of them (one that decays by 1e-6 a token was off by 1.1e-5 after 512 chunks).
__device__ __forceinline__ float2 lin_factor(int64_t x) {
  const double f = exp2((double)x * 0x1p-44);
  const float hi = (float)f;
  return make_float2(hi, (float)(f - (double)hi));
}
__device__ __forceinline__ float lin_float(int64_t x) { return __ll2float_rn(x) * 0x1p-44f; }
// The same of a decay in log2 units, in fp32, for the chunks' factors: where a state decays little, by the series of e^y - 1, good to some
// 2^-23 of that difference, however often it is applied; from 2^(-1/4) on the state forgets within some chunks, and one number does.
__device__ __forceinline__ float lin_near_one(float y) {   // e^y - 1
  float p = 1.f / 5040;                     // over y
  p = fmaf(p, y, 1.f / 720);
  p = fmaf(p, y, 1.f / 120);
  p = fmaf(p, y, 1.f / 24);
  p = fmaf(p, y, 1.f / 6);
  p = fmaf(p, y, 0.5f);
  return fmaf(p, y, 1.f) * y;
}
__device__ __forceinline__ float2 lin_factor_near(float x) {
  if (x < -0.25f) return make_float2(exp2f(x), 0.f);
  const float p = lin_near_one(x * 0.69314718056f), hi = 1.f + p;
  return make_float2(hi, p - (hi - 1.f));
}

#endif

}  // namespace kda
