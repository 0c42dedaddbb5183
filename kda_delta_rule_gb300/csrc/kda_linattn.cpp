// C ABI of linear attention with one decay for each head (kda_linattn_step, kda_linattn_prefill): host-side
// checks and the division of prefill work.  A call that returns an error has launched nothing.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "../../include/kda.h"
#include "kda_internal.h"
#include "kda_linattn.h"
#include "kda_mla.cuh"

namespace {

int fail(int status, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return kda::set_error(status, buf);
}

int ok() {
  kda::set_error(KDA_OK, "");
  return KDA_OK;
}

int cuda_status(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return ok();
  return fail(KDA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
size_t elem_size(int dtype) { return dtype == KDA_BF16 ? 2 : 4; }
bool head_dim_ok(int d) { return d == 32 || d == 64 || d == 128; }

struct Range {
  const void* p;
  size_t n;
};
bool overlap(const Range& a, const Range& b) {
  if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
  auto pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
  return pa < pb + b.n && pb < pa + a.n;
}
// bytes an array of rows spans
size_t span(int64_t rows, int64_t stride, int64_t last, size_t es) { return rows > 0 ? (size_t)((rows - 1) * stride + last) * es : 0; }

constexpr int kMaxHeads = 16383;            // a launch's sequences times heads times 32-column slices are an int, heads a grid's second axis
constexpr int64_t kMaxTokens = 0x7fff0000;  // positions some chunks behind a sequence's end are still ints, and it is one segment unless split

int check_heads(int H, int H_k, int dk, int dv, int dtype, float scale) {
  if (dtype != KDA_F32 && dtype != KDA_BF16) return fail(KDA_ERR_DTYPE, "dtype %d is not KDA_F32 or KDA_BF16", dtype);
  if (!head_dim_ok(dk) || !head_dim_ok(dv)) return fail(KDA_ERR_SHAPE, "dk=%d, dv=%d: must be 32, 64 or 128", dk, dv);
  if (H < 0 || H > kMaxHeads) return fail(KDA_ERR_SHAPE, "H=%d outside [0, %d]", H, kMaxHeads);
  if (H > 0 && (H_k < 1 || H % H_k != 0)) return fail(KDA_ERR_SHAPE, "H_k=%d must divide H=%d", H_k, H);
  if (!std::isfinite(scale)) return fail(KDA_ERR_ARG, "scale=%g must be finite", (double)scale);
  return KDA_OK;
}

// Rows of q, k, v, g: strides (a single row's says nothing and becomes the dense one), alignment.
int check_rows(const char* name, const void* p, int64_t rows, int64_t width, int64_t* stride, size_t es) {
  if (!p) return fail(KDA_ERR_ARG, "%s is NULL", name);
  if (!aligned16(p)) return fail(KDA_ERR_ALIGN, "%s must be 16-byte aligned", name);
  if (rows <= 1) *stride = width;
  if (*stride < width || (*stride * (int64_t)es) % 16 != 0 || *stride > (1ll << 32))
    return fail(KDA_ERR_SHAPE, "%s rows are %lld elements apart: at least %lld, a multiple of 16 bytes", name, (long long)*stride, (long long)width);
  return KDA_OK;
}
int check_decays(const float* g, int64_t rows, int H, int64_t* stride) {
  if (!g) return fail(KDA_ERR_ARG, "g is NULL");
  if (!aligned4(g)) return fail(KDA_ERR_ALIGN, "g must be 4-byte aligned");
  if (rows <= 1) *stride = 0;
  if (*stride != 0 && (*stride < H || *stride > (1ll << 32)))
    return fail(KDA_ERR_SHAPE, "g rows are %lld elements apart: 0 (one row for all tokens) or at least H=%d", (long long)*stride, H);
  return KDA_OK;
}

int check_seqlens(const int32_t* cu, int n_seqs, int64_t T) {
  if (T < 0 || T > kMaxTokens) return fail(KDA_ERR_SHAPE, "T=%lld outside [0, 2^31 - 2^16]", (long long)T);
  if (!cu) return KDA_OK;
  if (n_seqs < 1) return fail(KDA_ERR_SHAPE, "n_seqs=%d, must be >= 1", n_seqs);
  if (cu[0] != 0 || cu[n_seqs] != T) return fail(KDA_ERR_SHAPE, "cu_seqlens must run from 0 to T=%lld", (long long)T);
  for (int i = 0; i < n_seqs; ++i)
    if (cu[i + 1] < cu[i]) return fail(KDA_ERR_SHAPE, "cu_seqlens decreases at %d", i);
  return KDA_OK;
}

// The schedule of sequences [g0, g0 + n) of the call, longest first; `split`: a sequence may get several segments.
void make_sched(kda::LinSched& s, const int32_t* cu, int64_t T, int g0, int n, int ckpt_stride, int64_t ckpt_before, int H, int dv,
                int dtype, bool split) {
  const auto len = [&](int i) { return cu ? cu[g0 + i + 1] - cu[g0 + i] : (int32_t)T; };
  s.n_seqs = n;
  for (int i = 0; i < n; ++i) s.seq[i] = i;
  std::sort(s.seq, s.seq + n, [&](int a, int b) { return len(a) != len(b) ? len(a) > len(b) : a < b; });
  int32_t at[kda::kLinMaxSeqs];             // first checkpoint of each sequence
  for (int i = 0; i < n; ++i) {
    at[i] = (int32_t)ckpt_before;
    if (ckpt_stride > 0) ckpt_before += len(i) / ckpt_stride;
  }
  for (int p = 0; p < n; ++p) {
    const int i = s.seq[p];
    s.start[p] = cu ? cu[g0 + i] : 0;
    s.len[p] = len(i);
    s.ckpt_base[p] = at[i];
  }
  s.seg_len = split ? kda::lin_seg_len(s.len, n, H, dv, dtype, kda::kSms) : 0x7fffff80;
  s.item_base[0] = 0;
  for (int p = 0; p < n; ++p) s.item_base[p + 1] = s.item_base[p] + std::max(1, s.len[p] / s.seg_len + (s.len[p] % s.seg_len != 0));
  s.n_items = s.item_base[n];
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }
size_t states_bytes(const kda::LinSched& s, int H, int dk, int dv) { return round256((size_t)(s.n_items - s.n_seqs) * H * dk * dv * 4); }
size_t workspace_bytes_of(const kda::LinSched& s, int H, int dk, int dv) {
  return states_bytes(s, H, dk, dv) + round256((size_t)(s.n_items - s.n_seqs) * H * sizeof(float2));
}

}  // namespace

namespace kda {

// A split has to pay for the first pass, which reads k and v once more, and for two more launches.  Lengths are counted in steps: a
// chunk for the tensor cores (3.9 us at 128 x 128, one CTA on an SM), a batch of 16 tokens for the CUDA-core kernel (2.2 us, four CTAs on
// an SM), which is also the unit of time.  A step of the first pass takes 0.5 of one, a CTA's start and end 1.5, the
// launches and the scan 2.5 (4 of the shorter ones) and some more with the number of segments.  The numbers of segments that are tried grow by a
// quarter from eight on, so the one with the least cost may be missed (65536 tokens of 4 heads run as 32 segments of 16 chunks; 37 of 14 cost 9% less here).
int lin_seg_len(const int32_t* len, int n, int H, int dv, int dtype, int n_sm) {
  const bool tc = dtype == KDA_BF16;
  const int step = tc ? kLinChunk : kLinBatch;
  const int64_t heads = tc ? H : (int64_t)H * (dv / 32);   // the CUDA-core kernel has a CTA per 32 columns
  const double slots = tc ? n_sm : 4.0 * n_sm, start = 1.5;
  const auto steps = [&](int64_t tokens) { return (tokens + step - 1) / step; };
  const int64_t longest = n > 0 ? steps(len[0]) : 0;
  int64_t all = 0;
  for (int p = 0; p < n; ++p) all += steps(len[p]);
  const int whole = 0x7fffff80;
  if (longest < 4 || n * heads >= 4 * slots) return whole;
  const auto spread = [&](double ctas, double work, double least) {   // the time of CTAs with this much work in all
    return ctas > 0 ? std::max(least + start, std::ceil(ctas / slots) * (work / ctas + start)) : 0.;
  };
  double best = 0.95 * spread((double)n * heads, (double)all * heads, (double)longest);
  int64_t seg = 0;
  for (int64_t parts = 2; parts <= 256 && parts <= longest; parts += parts < 8 ? 1 : parts / 4) {
    const int64_t c = (longest + parts - 1) / parts;
    int64_t items = 0, first = 0;
    for (int p = 0; p < n; ++p) {
      const int64_t k = std::max<int64_t>(1, (steps(len[p]) + c - 1) / c);
      items += k;
      first += k - 1;
    }
    const double states = (double)first * heads;
    const double cost = spread((double)items * heads, (double)all * heads, (double)c) + 0.5 * spread(states, states * c, (double)c) +
                        (tc ? 2.5 : 4.) + 0.06 * parts;
    if (cost < best) {
      best = cost;
      seg = c;
    }
  }
  return seg ? (int)(seg * step) : whole;
}

}  // namespace kda

extern "C" {

int kda_linattn_step(const float* S_in, float* S_out, int64_t n_slots, const int32_t* slot_in, const int32_t* slot_out, const void* q,
                     int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride, const float* g, int64_t g_stride,
                     const int32_t* n_accepted, float scale, void* o, int steps, int B, int H, int H_k, int dk, int dv, int dtype,
                     kda_stream_t stream) {
  if (int st = check_heads(H, H_k, dk, dv, dtype, scale)) return st;
  if (B < 0) return fail(KDA_ERR_SHAPE, "negative B=%d", B);
  if (steps < 1 || steps > KDA_MAX_DRAFT) return fail(KDA_ERR_SHAPE, "steps=%d outside [1, %d]", steps, KDA_MAX_DRAFT);
  if (B == 0 || H == 0) return ok();
  const int64_t heads = (int64_t)B * H, state = (int64_t)dk * dv;
  if (heads > 0x7fffffffLL / 4 / KDA_MAX_DRAFT) return fail(KDA_ERR_SHAPE, "B*H too large");
  if (n_slots < 1 || n_slots > (1ll << 40) / (H * state)) return fail(KDA_ERR_SHAPE, "n_slots=%lld: at least 1, states within 2^40 values", (long long)n_slots);
  if (!S_in || !o) return fail(KDA_ERR_ARG, "null pointer argument");
  if (!slot_in && n_slots < B) return fail(KDA_ERR_SHAPE, "n_slots=%lld states for B=%d sequences without slot ids", (long long)n_slots, B);
  if (!slot_out && S_out && !slot_in && n_slots < B) return fail(KDA_ERR_SHAPE, "too few states");
  const size_t es = elem_size(dtype);
  const int64_t rows = (int64_t)steps * B;
  if (int st = check_rows("q", q, rows, (int64_t)H_k * dk, &q_stride, es)) return st;
  if (int st = check_rows("k", k, rows, (int64_t)H_k * dk, &k_stride, es)) return st;
  if (int st = check_rows("v", v, rows, (int64_t)H * dv, &v_stride, es)) return st;
  if (int st = check_decays(g, rows, H, &g_stride)) return st;
  if (!aligned16(S_in) || !aligned16(S_out) || !aligned16(o)) return fail(KDA_ERR_ALIGN, "states and o must be 16-byte aligned");
  if (!aligned4(slot_in) || !aligned4(slot_out) || !aligned4(n_accepted)) return fail(KDA_ERR_ALIGN, "int32 arrays must be 4-byte aligned");
  const Range states{S_in, (size_t)n_slots * H * state * 4}, to{S_out, (size_t)n_slots * H * state * 4};
  const Range out{o, (size_t)rows * H * dv * es};
  const Range in[] = {{q, span(rows, q_stride, (int64_t)H_k * dk, es)}, {k, span(rows, k_stride, (int64_t)H_k * dk, es)},
                      {v, span(rows, v_stride, (int64_t)H * dv, es)}, {g, span(g_stride ? rows : 1, g_stride, H, 4)},
                      {slot_in, (size_t)B * 4}, {slot_out, (size_t)B * 4}, {n_accepted, (size_t)B * 4}};
  for (const Range& x : in)
    if (overlap(x, out) || overlap(x, to)) return fail(KDA_ERR_ALIAS, "an output overlaps an input");
  if (overlap(out, states) || overlap(out, to)) return fail(KDA_ERR_ALIAS, "o overlaps the states");
  if (S_out && S_out != S_in && overlap(states, to)) return fail(KDA_ERR_ALIAS, "S_out overlaps a part of S_in");
  kda::LinStepArgs a{};
  a.S_in = S_in; a.S_out = S_out; a.slot_in = slot_in; a.slot_out = slot_out; a.n_accepted = n_accepted; a.n_slots = n_slots;
  a.q = q; a.k = k; a.v = v; a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride;
  a.g = g; a.g_stride = g_stride; a.o = o;
  a.steps = steps; a.B = B; a.H = H; a.share = H / H_k; a.dk = dk; a.dv = dv; a.dtype = dtype; a.scale = scale;
  return cuda_status(kda::launch_linattn_step(a, reinterpret_cast<cudaStream_t>(stream)), "kda_linattn_step launch");
}

int64_t kda_linattn_prefill_workspace_bytes(const int32_t* cu_seqlens, int n_seqs, int64_t T, int H, int dk, int dv, int dtype) {
  if (int st = check_heads(H, 1, dk, dv, dtype, 1.f)) return st;
  if (int st = check_seqlens(cu_seqlens, n_seqs, T)) return st;
  ok();
  if (H == 0) return 0;
  const int N = cu_seqlens ? n_seqs : 1;
  size_t most = 0;
  for (int g0 = 0; g0 < N; g0 += kda::kLinMaxSeqs) {
    kda::LinSched s;
    make_sched(s, cu_seqlens, T, g0, std::min(kda::kLinMaxSeqs, N - g0), 0, 0, H, dv, dtype, true);
    most = std::max(most, workspace_bytes_of(s, H, dk, dv));
  }
  return (int64_t)most;
}

int kda_linattn_prefill(const float* S0, const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                        int64_t v_stride, const float* g, int64_t g_stride, const int32_t* cu_seqlens, int n_seqs, int64_t T, int H,
                        int H_k, int dk, int dv, int dtype, float scale, int ckpt_stride, void* o, float* S_final, void* page_pool,
                        int64_t page_bytes, const int32_t* ckpt_page_ids, int32_t* ckpt_pos, int64_t num_ckpt, void* workspace,
                        int64_t workspace_bytes, kda_stream_t stream) {
  if (int st = check_heads(H, H_k, dk, dv, dtype, scale)) return st;
  if (int st = check_seqlens(cu_seqlens, n_seqs, T)) return st;
  if (ckpt_stride < 0 || ckpt_stride % kda::kLinChunk != 0)
    return fail(KDA_ERR_SHAPE, "ckpt_stride=%d must be 0 or a multiple of %d", ckpt_stride, kda::kLinChunk);
  if (H == 0) return ok();
  const int N = cu_seqlens ? n_seqs : 1;
  const int64_t state = (int64_t)dk * dv;
  const size_t es = elem_size(dtype);
  if (!S_final) return fail(KDA_ERR_ARG, "S_final is NULL");
  if (!aligned16(S0) || !aligned16(S_final)) return fail(KDA_ERR_ALIGN, "states must be 16-byte aligned");
  if (T > 0) {
    if (int st = check_rows("q", q, T, (int64_t)H_k * dk, &q_stride, es)) return st;
    if (int st = check_rows("k", k, T, (int64_t)H_k * dk, &k_stride, es)) return st;
    if (int st = check_rows("v", v, T, (int64_t)H * dv, &v_stride, es)) return st;
    if (int st = check_decays(g, T, H, &g_stride)) return st;
    if (!o) return fail(KDA_ERR_ARG, "o is NULL");
    if (!aligned16(o)) return fail(KDA_ERR_ALIGN, "o must be 16-byte aligned");
  }
  int64_t n_ck = 0;
  if (ckpt_stride > 0)
    for (int i = 0; i < N; ++i) n_ck += (cu_seqlens ? cu_seqlens[i + 1] - cu_seqlens[i] : T) / ckpt_stride;
  if (n_ck > 0) {
    if (num_ckpt < n_ck) return fail(KDA_ERR_SHAPE, "num_ckpt=%lld, the sequences have %lld checkpoints", (long long)num_ckpt, (long long)n_ck);
    if (!page_pool || !ckpt_page_ids) return fail(KDA_ERR_ARG, "checkpoints without page_pool or ckpt_page_ids");
    if (!aligned16(page_pool)) return fail(KDA_ERR_ALIGN, "page_pool must be 16-byte aligned");
    if (!aligned4(ckpt_page_ids) || !aligned4(ckpt_pos)) return fail(KDA_ERR_ALIGN, "int32 arrays must be 4-byte aligned");
    if (page_bytes % 16 != 0 || page_bytes < H * state * 4)
      return fail(KDA_ERR_SHAPE, "page_bytes=%lld: a multiple of 16 that holds H*dk*dv fp32 values", (long long)page_bytes);
  }
  const Range S{S_final, (size_t)N * H * state * 4}, out{o, (size_t)T * H * dv * es}, ws{workspace, workspace ? (size_t)std::max<int64_t>(workspace_bytes, 0) : 0};
  const Range pos{ckpt_pos, (size_t)n_ck * 4};
  const Range in[] = {{S0, (size_t)N * H * state * 4}, {q, span(T, q_stride, (int64_t)H_k * dk, es)}, {k, span(T, k_stride, (int64_t)H_k * dk, es)},
                      {v, span(T, v_stride, (int64_t)H * dv, es)}, {g, T > 0 ? span(g_stride ? T : 1, g_stride, H, 4) : 0},
                      {ckpt_page_ids, (size_t)n_ck * 4}};
  for (const Range& x : in)
    if (overlap(x, S) || overlap(x, out) || overlap(x, ws) || overlap(x, pos)) return fail(KDA_ERR_ALIAS, "an output or the workspace overlaps an input");
  if (overlap(S, out) || overlap(S, ws) || overlap(out, ws)) return fail(KDA_ERR_ALIAS, "o, S_final and the workspace overlap");
  if (overlap(pos, S) || overlap(pos, out) || overlap(pos, ws)) return fail(KDA_ERR_ALIAS, "ckpt_pos overlaps o, S_final or the workspace");
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return fail(KDA_ERR_ALIGN, "workspace must be 256-byte aligned");
  if (workspace) {
    const int64_t need = kda_linattn_prefill_workspace_bytes(cu_seqlens, n_seqs, T, H, dk, dv, dtype);
    if (need < 0) return (int)need;
    if (workspace_bytes < need) return fail(KDA_ERR_SHAPE, "workspace has %lld bytes, needs %lld", (long long)workspace_bytes, (long long)need);
  }
  kda::LinPrefillArgs a{};
  a.q = q; a.k = k; a.v = v; a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride;
  a.g = g; a.g_stride = g_stride; a.o = o;
  a.pages = static_cast<unsigned char*>(page_pool); a.page_bytes = page_bytes; a.ckpt_page_ids = ckpt_page_ids; a.ckpt_pos = ckpt_pos;
  a.num_ckpt = n_ck; a.T = T; a.H = H; a.share = H / H_k; a.dk = dk; a.dv = dv; a.dtype = dtype;
  a.ckpt_stride = n_ck > 0 ? ckpt_stride : 0;
  // On the tensor cores the factor of the outputs is a part of their weights.  Of one whose products could leave fp32's range there, the
  // weights take the significand, and the power of two multiplies the outputs afterwards, which is exact.
  a.scale = scale;
  float last = 1.f;
  if (dtype == KDA_BF16 && scale != 0.f && !(std::fabs(scale) >= 0x1p-20f && std::fabs(scale) <= 0x1p20f)) {
    int e;
    a.scale = 2.f * std::frexp(scale, &e);
    last = std::ldexp(1.f, e - 1);
  }
  int64_t ckpt_before = 0;
  for (int g0 = 0; g0 < N; g0 += kda::kLinMaxSeqs) {
    const int n = std::min(kda::kLinMaxSeqs, N - g0);
    kda::LinSched s;
    make_sched(s, cu_seqlens, T, g0, n, a.ckpt_stride, ckpt_before, H, dv, dtype, workspace != nullptr);
    a.S0 = S0 ? S0 + g0 * H * state : nullptr;
    a.S_final = S_final + g0 * H * state;
    a.seg_state = static_cast<float*>(workspace);
    a.seg_decay = reinterpret_cast<float2*>(static_cast<unsigned char*>(workspace) + states_bytes(s, H, dk, dv));
    if (int st = cuda_status(kda::launch_linattn_prefill(a, s, reinterpret_cast<cudaStream_t>(stream)), "kda_linattn_prefill launch")) return st;
    if (a.ckpt_stride > 0)
      for (int i = 0; i < n; ++i) ckpt_before += (cu_seqlens ? cu_seqlens[g0 + i + 1] - cu_seqlens[g0 + i] : T) / ckpt_stride;
  }
  if (last != 1.f)
    if (int st = cuda_status(kda::launch_linattn_scale(o, T * H * dv, last, reinterpret_cast<cudaStream_t>(stream)), "kda_linattn_prefill launch"))
      return st;
  return ok();
}

}  // extern "C"
