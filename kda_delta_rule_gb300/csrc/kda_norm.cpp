// C ABI of the norms around a block (kda_gated_norm, kda_residual_norm): host-side checks.  A call that returns an
// error has launched nothing.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "../../include/kda.h"
#include "kda_internal.h"
#include "kda_norm.h"

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
bool dtype_ok(int dtype) { return dtype == KDA_F32 || dtype == KDA_BF16; }

struct Range {
  const void* p;
  size_t n;
};
bool overlap(const Range& a, const Range& b) {
  if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
  auto pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
  return pa < pb + b.n && pb < pa + a.n;
}
size_t span(int64_t rows, int64_t stride, int64_t width, size_t es) { return rows > 0 ? (size_t)((rows - 1) * stride + width) * es : 0; }

int check_scalars(int64_t T, int act, float eps) {
  if (T < 0 || T > 0x7fffffffLL) return fail(KDA_ERR_SHAPE, "T=%lld outside [0, 2^31)", (long long)T);
  if (act != KDA_ACT_NONE && act != KDA_ACT_SILU && act != KDA_ACT_SIGMOID) return fail(KDA_ERR_ARG, "act=%d is not a KDA_ACT_*", act);
  if (!(eps >= 0.f && std::isfinite(eps))) return fail(KDA_ERR_ARG, "eps=%g must be finite and >= 0", (double)eps);
  return KDA_OK;
}
// T rows: the stride of a single one says nothing and becomes the dense one.
int check_rows(const char* name, const void* p, int64_t T, int64_t width, int64_t* stride, size_t es) {
  if (!aligned16(p)) return fail(KDA_ERR_ALIGN, "%s must be 16-byte aligned", name);
  if (T == 1) *stride = width;
  if (*stride < width || (*stride * (int64_t)es) % 16 != 0 || *stride > (1ll << 32))
    return fail(KDA_ERR_SHAPE, "%s rows are %lld elements apart: at least %lld, a multiple of 16 bytes", name, (long long)*stride, (long long)width);
  return KDA_OK;
}

}  // namespace

extern "C" {

int kda_gated_norm(const void* x, int64_t x_stride, const void* gate, int64_t gate_stride, const void* weight, int64_t weight_stride,
                   float eps, int act, int gate_first, void* y, int64_t T, int H, int d, int dtype, kda_stream_t stream) {
  if (!dtype_ok(dtype)) return fail(KDA_ERR_DTYPE, "dtype %d is not KDA_F32 or KDA_BF16", dtype);
  if (d < 8 || d > 1024 || d % 8 != 0) return fail(KDA_ERR_SHAPE, "d=%d: a multiple of 8 up to 1024", d);
  if (H < 0) return fail(KDA_ERR_SHAPE, "negative H=%d", H);
  if (int st = check_scalars(T, act, eps)) return st;
  if (T == 0 || H == 0) return ok();
  if (T * H > 0x7fffffffLL) return fail(KDA_ERR_SHAPE, "T*H too large");
  if (!x || !weight || !y) return fail(KDA_ERR_ARG, "null pointer argument");
  if (gate_first != 0 && gate_first != 1) return fail(KDA_ERR_ARG, "gate_first=%d is not 0 or 1", gate_first);
  if (weight_stride != 0 && weight_stride != d) return fail(KDA_ERR_SHAPE, "weight_stride=%lld: 0 (shared by the heads) or d=%d", (long long)weight_stride, d);
  const size_t es = elem_size(dtype);
  const int64_t width = (int64_t)H * d;
  if (int st = check_rows("x", x, T, width, &x_stride, es)) return st;
  if (gate)
    if (int st = check_rows("gate", gate, T, width, &gate_stride, es)) return st;
  if (!aligned16(weight) || !aligned16(y)) return fail(KDA_ERR_ALIGN, "weight and y must be 16-byte aligned");
  const Range out{y, (size_t)(T * width) * es};
  const bool in_place = y == x && x_stride == width, on_gate = y == gate && gate_stride == width;
  const Range in[] = {{in_place ? nullptr : x, span(T, x_stride, width, es)}, {on_gate ? nullptr : gate, span(T, gate_stride, width, es)},
                      {weight, (size_t)(weight_stride ? width : d) * es}};
  for (const Range& r : in)
    if (overlap(r, out)) return fail(KDA_ERR_ALIAS, "y overlaps an input");
  kda::GatedNormArgs a{};
  a.x = x; a.x_stride = x_stride; a.gate = gate; a.gate_stride = gate_stride; a.weight = weight; a.weight_stride = (int)weight_stride;
  a.eps = eps; a.act = act; a.gate_first = gate_first; a.y = y; a.T = T; a.H = H; a.d = d; a.dtype = dtype;
  return cuda_status(kda::launch_gated_norm(a, reinterpret_cast<cudaStream_t>(stream)), "kda_gated_norm launch");
}

int kda_residual_norm(const void* y, int64_t y_stride, const void* gate, int64_t gate_stride, const void* post_weight,
                      const void* channel_scale, float res_scale, const void* h_in, void* h_out, int64_t h_stride, int h_dtype,
                      const void* pre_weight, float eps, int act, void* x, int64_t T, int D, int dtype, kda_stream_t stream) {
  if (!dtype_ok(dtype)) return fail(KDA_ERR_DTYPE, "dtype %d is not KDA_F32 or KDA_BF16", dtype);
  if (h_dtype != KDA_F32 && h_dtype != dtype) return fail(KDA_ERR_DTYPE, "h_dtype %d is neither KDA_F32 nor dtype", h_dtype);
  if (D < 8 || D > 16384 || D % 8 != 0) return fail(KDA_ERR_SHAPE, "D=%d: a multiple of 8 up to 16384", D);
  if (int st = check_scalars(T, act, eps)) return st;
  if (!std::isfinite(res_scale)) return fail(KDA_ERR_ARG, "res_scale=%g must be finite", (double)res_scale);
  if (T == 0) return ok();
  if (!y || !h_in || !h_out || !pre_weight || !x) return fail(KDA_ERR_ARG, "null pointer argument");
  const size_t es = elem_size(dtype), hs = elem_size(h_dtype);
  if (int st = check_rows("y", y, T, D, &y_stride, es)) return st;
  if (gate)
    if (int st = check_rows("gate", gate, T, D, &gate_stride, es)) return st;
  if (int st = check_rows("h", h_in, T, D, &h_stride, hs)) return st;
  if (!aligned16(h_out) || !aligned16(x) || !aligned16(post_weight) || !aligned16(pre_weight) || !aligned16(channel_scale))
    return fail(KDA_ERR_ALIGN, "pointers must be 16-byte aligned");
  const Range ho{h_out, span(T, h_stride, D, hs)}, xo{x, (size_t)T * D * es};
  const Range in[] = {{y, span(T, y_stride, D, es)}, {gate, span(T, gate_stride, D, es)}, {post_weight, (size_t)D * es},
                      {pre_weight, (size_t)D * es}, {channel_scale, (size_t)D * es}};
  for (const Range& r : in)
    if (overlap(r, ho) || overlap(r, xo)) return fail(KDA_ERR_ALIAS, "an output overlaps an input");
  const Range hi{h_in, ho.n};
  if ((h_in != h_out && overlap(hi, ho)) || overlap(hi, xo) || overlap(ho, xo)) return fail(KDA_ERR_ALIAS, "h_in, h_out and x overlap");
  kda::ResidualNormArgs a{};
  a.y = y; a.y_stride = y_stride; a.gate = gate; a.gate_stride = gate_stride; a.post_weight = post_weight; a.channel_scale = channel_scale;
  a.res_scale = res_scale; a.h_in = h_in; a.h_out = h_out; a.h_stride = h_stride; a.h_dtype = h_dtype; a.pre_weight = pre_weight;
  a.eps = eps; a.act = act; a.x = x; a.T = T; a.D = D; a.dtype = dtype;
  return cuda_status(kda::launch_residual_norm(a, reinterpret_cast<cudaStream_t>(stream)), "kda_residual_norm launch");
}

}  // extern "C"
