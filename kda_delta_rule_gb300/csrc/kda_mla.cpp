// C ABI of the latent page cache (kda_mla_append, kda_mla_decode): host-side checks
// and the workspace's layout.  A call that returns an error has launched nothing.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "../../include/kda.h"
#include "kda_internal.h"
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
size_t elem_size(int dtype) { return dtype == KDA_BF16 ? 2 : 4; }

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  if (!a || !b || na == 0 || nb == 0) return false;
  auto pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
  return pa < pb + nb && pb < pa + na;
}

int check_row(int d_c, int d_r, int dtype) {
  if (dtype != KDA_F32 && dtype != KDA_BF16) return fail(KDA_ERR_DTYPE, "dtype %d is not KDA_F32 or KDA_BF16", dtype);
  if (d_c < 128 || d_c > 512 || d_c % 128 != 0)
    return fail(KDA_ERR_SHAPE, "d_c=%d: must be 128, 256, 384 or 512", d_c);
  if (d_r < 0 || d_r > 64 || d_r % 16 != 0)
    return fail(KDA_ERR_SHAPE, "d_r=%d: must be 0, 16, 32, 48 or 64", d_r);
  return KDA_OK;
}

int check_pages(const void* pages, int64_t page_bytes, int64_t n_pages, int page_tokens, int d_c, int d_r, int dtype) {
  if (!pages) return fail(KDA_ERR_ARG, "pages is NULL");
  if (!aligned16(pages)) return fail(KDA_ERR_ALIGN, "pages must be 16-byte aligned");
  if (page_tokens < 16 || page_tokens % 16 != 0 || page_tokens > (1 << 20))
    return fail(KDA_ERR_SHAPE, "page_tokens=%d: must be a multiple of 16 up to 2^20", page_tokens);
  if (n_pages < 1 || n_pages > 0x7fffffffLL) return fail(KDA_ERR_SHAPE, "n_pages=%lld outside [1, 2^31)", (long long)n_pages);
  if (page_bytes % 16 != 0 || page_bytes < (int64_t)page_tokens * (d_c + d_r) * (int64_t)elem_size(dtype))
    return fail(KDA_ERR_SHAPE, "page_bytes=%lld: must be a multiple of 16 that holds page_tokens=%d rows",
                (long long)page_bytes, page_tokens);
  if (page_bytes > ((int64_t)1 << 38) || n_pages > ((int64_t)1 << 50) / page_bytes)
    return fail(KDA_ERR_SHAPE, "page arena too large");
  return KDA_OK;
}

// bytes an array of rows spans
size_t span(int64_t rows, int64_t stride, int64_t last, size_t es) { return rows > 0 ? ((rows - 1) * stride + last) * es : 0; }

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

// the parts of a call and where they lie in its workspace
struct Plan {
  int n;
  kda::MlaPart parts[2];
  size_t o_at[2], ml_at[2], cta_at[2], bytes;
};

Plan make_plan(int B, int n_q, int H, int d_c, int64_t prefix_len, int dtype) {
  Plan p{};
  p.n = kda::mla_parts(B, n_q * H, prefix_len, dtype, p.parts);
  for (int i = 0; i < p.n; ++i) {
    const kda::MlaPart& w = p.parts[i];
    const int64_t slots = w.items() + kda::kMlaMaxCtas;
    p.o_at[i] = p.bytes;
    p.bytes += round256((size_t)slots * w.nr * d_c * sizeof(float));
    p.ml_at[i] = p.bytes;
    p.bytes += round256((size_t)slots * w.nr * sizeof(float2));
    p.cta_at[i] = p.bytes;
    p.bytes += round256((size_t)w.items() * sizeof(int2));
  }
  return p;
}

int check_decode_sizes(int B, int n_q, int H, int d_c, int d_r, int64_t prefix_len, int dtype) {
  if (int st = check_row(d_c, d_r, dtype)) return st;
  if (B < 0 || H < 0) return fail(KDA_ERR_SHAPE, "negative B=%d or H=%d", B, H);
  if (n_q < 1 || n_q > KDA_MAX_DRAFT) return fail(KDA_ERR_SHAPE, "n_q=%d outside [1, %d]", n_q, KDA_MAX_DRAFT);
  if (H > 0 && (int64_t)n_q * H > 0x7fffffffLL / (B > 0 ? B : 1)) return fail(KDA_ERR_SHAPE, "B*n_q*H too large");
  if (prefix_len < 0 || prefix_len > kda::kMlaMaxTokens)
    return fail(KDA_ERR_SHAPE, "prefix_len=%lld outside [0, 2^31 - 256]", (long long)prefix_len);
  return KDA_OK;
}

}  // namespace

extern "C" {

int kda_mla_append(void* pages, int64_t page_bytes, int64_t n_pages, int page_tokens, const int32_t* slots,
                   const int32_t* positions, const float* rope, int n_pos, const void* c, int64_t c_stride,
                   const void* k_pe, int64_t k_pe_stride, const void* norm_weight, float eps, const void* q_pe,
                   int64_t q_stride_t, int64_t q_stride_h, void* q_pe_out, int T, int H, int d_c, int d_r, int dtype,
                   int style, kda_stream_t stream) {
  if (int st = check_row(d_c, d_r, dtype)) return st;
  if (T < 0 || H < 0) return fail(KDA_ERR_SHAPE, "negative T=%d or H=%d", T, H);
  if (style != KDA_ROPE_HALF && style != KDA_ROPE_INTERLEAVED) return fail(KDA_ERR_ARG, "style=%d is not a KDA_ROPE_*", style);
  if (T == 0) return ok();
  if (int st = check_pages(pages, page_bytes, n_pages, page_tokens, d_c, d_r, dtype)) return st;
  if (n_pages > 0x7fffffffLL / page_tokens) return fail(KDA_ERR_SHAPE, "n_pages*page_tokens exceeds the 2^31 slots");
  if (!slots || !c) return fail(KDA_ERR_ARG, "null pointer argument");
  if (norm_weight && !(eps >= 0.f && std::isfinite(eps))) return fail(KDA_ERR_ARG, "eps=%g must be finite and >= 0", (double)eps);
  const size_t es = elem_size(dtype);
  const int64_t vec = 16 / (int64_t)es;
  if (c_stride < d_c || c_stride % vec) return fail(KDA_ERR_SHAPE, "c_stride=%lld: at least d_c, a multiple of 16 bytes", (long long)c_stride);
  if (d_r > 0) {
    if (!positions || !rope || !k_pe) return fail(KDA_ERR_ARG, "null pointer argument (d_r > 0)");
    if (n_pos < 1) return fail(KDA_ERR_SHAPE, "n_pos=%d, must be >= 1", n_pos);
    if (k_pe_stride < d_r || k_pe_stride % vec)
      return fail(KDA_ERR_SHAPE, "k_pe_stride=%lld: at least d_r, a multiple of 16 bytes", (long long)k_pe_stride);
  }
  if ((int64_t)T * (H + 8) > 0x7fffffffLL) return fail(KDA_ERR_SHAPE, "T*H too large");
  const bool queries = q_pe && d_r > 0 && H > 0;
  if (q_pe && d_r == 0) return fail(KDA_ERR_ARG, "q_pe given but d_r is 0");
  if (queries) {
    if (!q_pe_out) return fail(KDA_ERR_ARG, "q_pe given without q_pe_out");
    // the stride of an axis of one entry says nothing: what a dense tensor has there
    if (H == 1) q_stride_h = d_r;
    if (T == 1) q_stride_t = (int64_t)H * d_r;
    const bool by_token = q_stride_h >= d_r && (T == 1 || q_stride_t >= (H - 1) * q_stride_h + d_r);
    const bool by_head = q_stride_t >= d_r && (H == 1 || q_stride_h >= (T - 1) * q_stride_t + d_r);
    if (q_stride_h % vec || q_stride_t % vec || !(by_token || by_head))
      return fail(KDA_ERR_SHAPE, "q_pe strides: multiples of 16 bytes, its rows apart, token by token or head by head");
  }
  const void* al[] = {c, k_pe, rope, norm_weight, q_pe, q_pe_out};
  for (const void* p : al)
    if (p && !aligned16(p)) return fail(KDA_ERR_ALIGN, "pointers must be 16-byte aligned");
  const size_t arena = (size_t)page_bytes * n_pages;
  const size_t q_out_bytes = queries ? (size_t)T * H * d_r * es : 0;
  const size_t q_bytes = queries ? span(T, q_stride_t, (H - 1) * q_stride_h + d_r, es) : 0;
  const bool in_place = queries && q_pe_out == q_pe && q_stride_h == d_r && q_stride_t == (int64_t)H * d_r;
  const struct { const void* p; size_t n; } in[] = {
      {slots, T * sizeof(int32_t)}, {positions, d_r ? T * sizeof(int32_t) : 0}, {rope, (size_t)n_pos * d_r * sizeof(float)},
      {c, span(T, c_stride, d_c, es)}, {k_pe, d_r ? span(T, k_pe_stride, d_r, es) : 0}, {norm_weight, d_c * es},
      {q_pe, in_place ? 0 : q_bytes}};
  for (const auto& x : in)
    if (overlap(pages, arena, x.p, x.n) || overlap(q_pe_out, q_out_bytes, x.p, x.n))
      return fail(KDA_ERR_ALIAS, "an output overlaps an input");
  if (overlap(pages, arena, q_pe_out, q_out_bytes)) return fail(KDA_ERR_ALIAS, "q_pe_out overlaps the pages");
  kda::MlaAppendArgs a{};
  a.pages = static_cast<unsigned char*>(pages);
  a.page_bytes = page_bytes; a.n_pages = n_pages; a.page_tokens = page_tokens;
  a.slots = slots; a.positions = positions; a.rope = rope; a.n_pos = n_pos;
  a.c = c; a.c_stride = c_stride; a.k_pe = k_pe; a.k_pe_stride = k_pe_stride;
  a.norm_weight = norm_weight; a.eps = eps;
  a.q_pe = queries ? q_pe : nullptr; a.q_stride_t = q_stride_t; a.q_stride_h = q_stride_h; a.q_pe_out = q_pe_out;
  a.T = T; a.H = H; a.d_c = d_c; a.d_r = d_r; a.dtype = dtype; a.style = style;
  return cuda_status(kda::launch_mla_append(a, reinterpret_cast<cudaStream_t>(stream)), "kda_mla_append launch");
}

int64_t kda_mla_decode_workspace_bytes(int B, int n_q, int H, int d_c, int64_t prefix_len, int dtype) {
  if (int st = check_decode_sizes(B, n_q, H, d_c, 0, prefix_len, dtype)) return st;
  ok();
  if (B == 0 || H == 0) return 0;
  return (int64_t)make_plan(B, n_q, H, d_c, prefix_len, dtype).bytes;
}

int kda_mla_decode(const void* q, const void* q_pe, const void* pages, int64_t page_bytes, int64_t n_pages,
                   int page_tokens, const int32_t* prefix_pages, int64_t prefix_len, const int32_t* page_table,
                   int64_t max_pages, const int32_t* lens, float scale, void* o, float* lse, int B, int n_q, int H,
                   int d_c, int d_r, int dtype, void* workspace, int64_t workspace_bytes, kda_stream_t stream) {
  if (int st = check_decode_sizes(B, n_q, H, d_c, d_r, prefix_len, dtype)) return st;
  if (B == 0 || H == 0) return ok();
  if (int st = check_pages(pages, page_bytes, n_pages, page_tokens, d_c, d_r, dtype)) return st;
  if (max_pages < 0 || max_pages > 0x7fffffffLL) return fail(KDA_ERR_SHAPE, "max_pages=%lld outside [0, 2^31)", (long long)max_pages);
  const float scale_log2 = scale * 1.4426950408889634f;   // log2(e): the kernels' exponentials are powers of two
  if (!(scale > 0.f && std::isfinite(scale_log2)))
    return fail(KDA_ERR_ARG, "scale=%g must be positive and, times log2(e), finite", (double)scale);
  if (!q || !lens || !o || (max_pages > 0 && !page_table) || (prefix_len > 0 && !prefix_pages) || (d_r > 0 && !q_pe))
    return fail(KDA_ERR_ARG, "null pointer argument");
  if (!aligned16(q) || !aligned16(o) || (d_r > 0 && !aligned16(q_pe)))
    return fail(KDA_ERR_ALIGN, "q, q_pe and o must be 16-byte aligned");
  Plan p = make_plan(B, n_q, H, d_c, prefix_len, dtype);
  const size_t need = p.bytes;
  if (!workspace) return fail(KDA_ERR_ARG, "workspace is NULL");
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return fail(KDA_ERR_ALIGN, "workspace must be 256-byte aligned");
  if (workspace_bytes < (int64_t)need)
    return fail(KDA_ERR_SHAPE, "workspace has %lld bytes, needs %lld", (long long)workspace_bytes, (long long)need);
  const size_t es = elem_size(dtype);
  const int64_t rows = (int64_t)B * n_q * H;
  const int64_t n_prefix = (prefix_len + page_tokens - 1) / page_tokens;
  const struct { const void* p; size_t n; } in[] = {
      {q, (size_t)rows * d_c * es}, {q_pe, (size_t)rows * d_r * es}, {pages, (size_t)page_bytes * n_pages},
      {prefix_pages, (size_t)n_prefix * 4}, {page_table, (size_t)B * max_pages * 4}, {lens, (size_t)B * 4}};
  const struct { const void* p; size_t n; } out[] = {{o, (size_t)rows * d_c * es}, {lse, (size_t)rows * 4}, {workspace, need}};
  for (int i = 0; i < 3; ++i) {
    for (const auto& x : in)
      if (overlap(out[i].p, out[i].n, x.p, x.n)) return fail(KDA_ERR_ALIAS, "an output or the workspace overlaps an input");
    for (int j = 0; j < i; ++j)
      if (overlap(out[i].p, out[i].n, out[j].p, out[j].n)) return fail(KDA_ERR_ALIAS, "o, lse and the workspace overlap");
  }
  kda::MlaArgs a{};
  a.q = q; a.q_pe = q_pe;
  a.pages = static_cast<const unsigned char*>(pages);
  a.page_bytes = page_bytes; a.n_pages = n_pages; a.page_tokens = page_tokens;
  a.prefix_pages = prefix_pages; a.prefix_len = (int)prefix_len;
  a.page_table = page_table; a.max_pages = max_pages; a.lens = lens;
  a.scale_log2 = scale_log2;
  a.o = o; a.lse = lse;
  a.B = B; a.n_q = n_q; a.H = H; a.d_c = d_c; a.d_r = d_r; a.dtype = dtype;
  a.seq_rows = n_q * H;
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  for (int i = 0; i < p.n; ++i) {
    p.parts[i].part_o = reinterpret_cast<float*>(ws + p.o_at[i]);
    p.parts[i].part_ml = reinterpret_cast<float2*>(ws + p.ml_at[i]);
    p.parts[i].item_ctas = reinterpret_cast<int2*>(ws + p.cta_at[i]);
  }
  return cuda_status(kda::launch_mla_decode(a, p.parts, p.n, reinterpret_cast<cudaStream_t>(stream)), "kda_mla_decode launch");
}

}  // extern "C"
