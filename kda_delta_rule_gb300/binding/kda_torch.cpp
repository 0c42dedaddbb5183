// Calls that serve single tokens (the latent page cache's, linear attention's, the norms') from Python without Python's share of
// the work.
//
// kda.py passes its arguments on as they are.  When every one of them is what the call
// takes, this checks them, allocates what was not given and calls the C ABI; otherwise it
// returns None and kda.py, which then says what is wrong (or finds nothing wrong with an
// argument of a less common kind), goes its own way through ctypes.  These calls serve
// single tokens: of 25 us that the binding took for one sequence's attention, 14 were the
// tests and allocations made from Python and ctypes' conversions; from here the call takes 14 us in
// all, 11 of them on the device beside it.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <c10/util/Optional.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <vector>

#include "../../include/kda.h"

namespace {

using at::Tensor;

// A CUDA tensor argument: null for None, false if it is something else.
bool tensor(PyObject* o, const Tensor** t) {
  *t = nullptr;
  if (o == Py_None) return true;
  if (!THPVariable_Check(o)) return false;
  *t = &THPVariable_Unpack(o);
  return (*t)->is_cuda();
}
bool integer(PyObject* o, int64_t* v) {
  if (!PyLong_Check(o)) return false;
  int overflow = 0;
  *v = PyLong_AsLongLongAndOverflow(o, &overflow);
  return overflow == 0;
}
bool fits_int(int64_t v) { return v >= INT32_MIN && v <= INT32_MAX; }
bool number(PyObject* o, double* v) {
  if (!PyFloat_Check(o) && !PyLong_Check(o)) return false;
  *v = PyFloat_AsDouble(o);
  if (*v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  return true;
}
bool dense(const Tensor* t, at::ScalarType type, at::IntArrayRef shape) {
  return t && t->scalar_type() == type && t->sizes() == shape && t->is_contiguous();
}
// the last axis dense, the others anyhow
bool rows(const Tensor* t, at::ScalarType type, at::IntArrayRef shape) {
  return t && t->scalar_type() == type && t->sizes() == shape && (shape.back() <= 1 || t->stride(-1) == 1);
}
// Do all of these (those that are there) lie on one device?  A kernel given another GPU's memory
// would fault.
bool on_one_device(const Tensor& on, std::initializer_list<const Tensor*> others) {
  for (const Tensor* t : others)
    if (t && t->device() != on.device()) return false;
  return true;
}
int code(at::ScalarType t) { return t == at::kFloat ? KDA_F32 : t == at::kBFloat16 ? KDA_BF16 : -1; }
void* ptr(const Tensor* t) { return t ? t->data_ptr() : nullptr; }

// the stream: a handle, or None for the device's current one
bool stream_of(PyObject* o, const Tensor& on, kda_stream_t* s) {
  if (o == Py_None) {
    *s = reinterpret_cast<kda_stream_t>(c10::cuda::getCurrentCUDAStream(on.get_device()).stream());
    return true;
  }
  int64_t v;
  if (!integer(o, &v)) return false;
  *s = reinterpret_cast<kda_stream_t>(static_cast<uintptr_t>(v));
  return true;
}

// Memory allocated for a call belongs to the stream that its kernels run on: taken from the
// current stream's pool it could still be in use there, or be handed out again there before the
// kernels are done.
struct AllocateOn {
  c10::optional<c10::cuda::CUDAStreamGuard> guard;
  AllocateOn(PyObject* given, kda_stream_t s, const Tensor& on) {
    if (given != Py_None) guard.emplace(c10::cuda::getStreamFromExternal(reinterpret_cast<cudaStream_t>(s), on.get_device()));
  }
};

// past the dispatcher
Tensor empty(at::IntArrayRef shape, at::ScalarType type, const Tensor& on) {
  return Tensor(at::detail::empty_cuda(shape, type, on.device(), c10::nullopt));
}

// (pages, page_tokens, slots, positions, rope, c, k_pe, q_pe, q_pe_out, norm_weight, eps, style,
//  stream) -> (status, q_pe_out or None)
PyObject* mla_append(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const Tensor *pages, *slots, *positions, *rope, *c, *k_pe, *q_pe, *out, *weight;
  int64_t page_tokens, style;
  double eps;
  kda_stream_t s;
  if (n != 13 || !tensor(args[0], &pages) || !integer(args[1], &page_tokens) || !tensor(args[2], &slots) ||
      !tensor(args[3], &positions) || !tensor(args[4], &rope) || !tensor(args[5], &c) || !tensor(args[6], &k_pe) ||
      !tensor(args[7], &q_pe) || !tensor(args[8], &out) || !tensor(args[9], &weight) || !number(args[10], &eps) ||
      !integer(args[11], &style) || !c || c->dim() != 2 || !pages || pages->dim() != 2 ||
      !on_one_device(*c, {pages, slots, positions, rope, k_pe, q_pe, out, weight}) || !stream_of(args[12], *c, &s))
    Py_RETURN_NONE;
  const auto type = c->scalar_type();
  const int64_t T = c->size(0), d_c = c->size(1);
  int64_t d_r = 0, n_pos = 0, H = 0, k_stride = 0, qst = 0, qsh = 0;
  if (code(type) < 0 || !rows(c, type, {T, d_c}) || !dense(pages, at::kByte, pages->sizes()) || !dense(slots, at::kInt, {T})) Py_RETURN_NONE;
  // the stride of an axis of one entry says nothing: it may have any value
  const int64_t c_stride = T > 1 ? c->stride(0) : d_c;
  if (k_pe) {
    if (k_pe->dim() != 2 || !rope || rope->dim() != 2) Py_RETURN_NONE;
    d_r = k_pe->size(1);
    n_pos = rope->size(0);
    k_stride = T > 1 ? k_pe->stride(0) : d_r;
    if (!rows(k_pe, type, {T, d_r}) || !dense(positions, at::kInt, {T}) || !dense(rope, at::kFloat, {n_pos, d_r})) Py_RETURN_NONE;
  }
  if (weight && !dense(weight, type, {d_c})) Py_RETURN_NONE;
  Tensor made;
  if (q_pe) {
    if (q_pe->dim() != 3) Py_RETURN_NONE;
    H = q_pe->size(1);
    if (!rows(q_pe, type, {T, H, d_r}) || (out && !dense(out, type, {T, H, d_r}))) Py_RETURN_NONE;
    qst = T > 1 ? q_pe->stride(0) : 0;
    qsh = H > 1 ? q_pe->stride(1) : d_r;
  }
  if (!fits_int(page_tokens) || !fits_int(style) || !fits_int(T) || !fits_int(H) || !fits_int(d_c) || !fits_int(n_pos)) Py_RETURN_NONE;
  const c10::cuda::CUDAGuard device(c->device());   // the library asks the current one for its SMs, and launches there
  if (q_pe && !out) {
    const AllocateOn stream(args[12], s, *c);
    made = empty({T, H, d_r}, type, *c);
    out = &made;
  }
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = kda_mla_append(ptr(pages), pages->size(1), pages->size(0), (int)page_tokens, static_cast<const int32_t*>(ptr(slots)),
                          k_pe ? static_cast<const int32_t*>(ptr(positions)) : nullptr,
                          k_pe ? static_cast<const float*>(ptr(rope)) : nullptr, (int)n_pos, ptr(c), c_stride, ptr(k_pe),
                          k_stride, ptr(weight), (float)eps, ptr(q_pe), qst, qsh, q_pe ? ptr(out) : nullptr, (int)T, (int)H,
                          (int)d_c, (int)d_r, code(type), (int)style, s);
  Py_END_ALLOW_THREADS
  PyObject* result = !q_pe ? Py_NewRef(Py_None) : made.defined() ? THPVariable_Wrap(made) : Py_NewRef(args[8]);
  return Py_BuildValue("(iN)", status, result);
  END_HANDLE_TH_ERRORS
}

// (q, q_pe, pages, page_tokens, page_table, lens, scale, prefix_pages, prefix_len, o, lse,
//  workspace, stream) -> (status, o, lse); workspace None: allocated here
PyObject* mla_decode(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const Tensor *q, *q_pe, *pages, *table, *lens, *prefix, *o, *lse, *ws;
  int64_t page_tokens, prefix_len;
  double scale;
  kda_stream_t s;
  if (n != 13 || !tensor(args[0], &q) || !tensor(args[1], &q_pe) || !tensor(args[2], &pages) || !integer(args[3], &page_tokens) ||
      !tensor(args[4], &table) || !tensor(args[5], &lens) || !number(args[6], &scale) || !tensor(args[7], &prefix) ||
      !integer(args[8], &prefix_len) || !tensor(args[9], &o) || !tensor(args[10], &lse) || !tensor(args[11], &ws) || !q ||
      q->dim() != 4 || !pages || pages->dim() != 2 || !table || table->dim() != 2 ||
      !on_one_device(*q, {q_pe, pages, table, lens, prefix, o, lse, ws}) || !stream_of(args[12], *q, &s))
    Py_RETURN_NONE;
  const auto type = q->scalar_type();
  const int64_t B = q->size(0), n_q = q->size(1), H = q->size(2), d_c = q->size(3), max_pages = table->size(1);
  int64_t d_r = 0;
  if (code(type) < 0 || !q->is_contiguous() || !dense(pages, at::kByte, pages->sizes()) || !dense(table, at::kInt, {B, max_pages}) ||
      !dense(lens, at::kInt, {B}))
    Py_RETURN_NONE;
  if (q_pe) {
    if (q_pe->dim() != 4) Py_RETURN_NONE;
    d_r = q_pe->size(3);
    if (!dense(q_pe, type, {B, n_q, H, d_r})) Py_RETURN_NONE;
  }
  if (!fits_int(page_tokens) || !fits_int(B) || !fits_int(n_q) || !fits_int(H) || !fits_int(d_c) || page_tokens < 1) Py_RETURN_NONE;
  if (prefix_len > 0 && (!prefix || !dense(prefix, at::kInt, {prefix->numel()}) || prefix->numel() * page_tokens < prefix_len))
    Py_RETURN_NONE;
  if ((o && !dense(o, type, {B, n_q, H, d_c})) || (lse && !dense(lse, at::kFloat, {B, n_q, H})) ||
      (ws && !dense(ws, at::kByte, {ws->numel()})))
    Py_RETURN_NONE;
  const c10::cuda::CUDAGuard device(q->device());   // the library asks the current one for its SMs, and launches there
  Tensor made_o, made_lse, made_ws;
  c10::optional<AllocateOn> stream;
  if (!o || !lse || !ws) stream.emplace(args[12], s, *q);
  if (!o) { made_o = empty({B, n_q, H, d_c}, type, *q); o = &made_o; }
  if (!lse) { made_lse = empty({B, n_q, H}, at::kFloat, *q); lse = &made_lse; }
  if (!ws) {
    const int64_t need = kda_mla_decode_workspace_bytes((int)B, (int)n_q, (int)H, (int)d_c, prefix_len, code(type));
    if (need < 0) Py_RETURN_NONE;
    made_ws = empty({need > 0 ? need : 1}, at::kByte, *q);
    ws = &made_ws;
  }
  stream.reset();
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = kda_mla_decode(ptr(q), d_r ? ptr(q_pe) : nullptr, ptr(pages), pages->size(1), pages->size(0), (int)page_tokens,
                          prefix_len > 0 ? static_cast<const int32_t*>(ptr(prefix)) : nullptr, prefix_len,
                          static_cast<const int32_t*>(ptr(table)), max_pages, static_cast<const int32_t*>(ptr(lens)),
                          (float)scale, ptr(o), static_cast<float*>(ptr(lse)), (int)B, (int)n_q, (int)H, (int)d_c, (int)d_r,
                          code(type), ptr(ws), ws->numel(), s);
  Py_END_ALLOW_THREADS
  return Py_BuildValue("(iNN)", status, made_o.defined() ? THPVariable_Wrap(made_o) : Py_NewRef(args[9]),
                       made_lse.defined() ? THPVariable_Wrap(made_lse) : Py_NewRef(args[10]));
  END_HANDLE_TH_ERRORS
}

// (lead.., heads, d) rows: heads dense, rows a fixed distance apart
bool head_rows(const Tensor* t, at::ScalarType type, int64_t lead, int64_t heads, int64_t d, int64_t* stride) {
  if (!t || t->scalar_type() != type || t->dim() != lead + 2 || t->size(-1) != d || t->size(-2) != heads) return false;
  if ((d > 1 && t->stride(-1) != 1) || (heads > 1 && t->stride(-2) != d)) return false;
  int64_t n = 1;
  for (int64_t i = 0; i < lead; ++i) n *= t->size(i);
  if (n <= 1) {
    *stride = heads * d;
    return true;
  }
  *stride = t->size(lead - 1) > 1 ? t->stride(lead - 1) : t->stride(0);
  return lead < 2 || t->size(0) <= 1 || t->size(1) <= 1 || t->stride(0) == t->size(1) * *stride;
}
// fp32 log decays, (lead.., H) or (H,) for all rows
bool decays(const Tensor* t, at::IntArrayRef lead, int64_t H, int64_t* stride) {
  *stride = 0;
  if (!t || t->scalar_type() != at::kFloat || t->dim() < 1 || t->size(-1) != H || (H > 1 && t->stride(-1) != 1)) return false;
  if (t->dim() == 1) return true;
  if (t->dim() != (int64_t)lead.size() + 1) return false;
  int64_t n = 1;
  for (size_t i = 0; i < lead.size(); ++i) {
    if (t->size(i) != lead[i]) return false;
    n *= lead[i];
  }
  if (n <= 1) return true;
  *stride = lead.back() > 1 ? t->stride(lead.size() - 1) : t->stride(0);
  return *stride != 0 && (lead.size() < 2 || lead[0] <= 1 || lead[1] <= 1 || t->stride(0) == lead[1] * *stride);
}

// (S, q, k, v, g, scale, o, S_new, write_state, slot_in, slot_out, n_accepted, stream) -> (status, o)
PyObject* linattn_step(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const Tensor *S, *q, *k, *v, *g, *o, *to, *in, *out, *count;
  double scale;
  kda_stream_t s;
  if (n != 13 || !tensor(args[0], &S) || !tensor(args[1], &q) || !tensor(args[2], &k) || !tensor(args[3], &v) || !tensor(args[4], &g) ||
      !number(args[5], &scale) || !tensor(args[6], &o) || !tensor(args[7], &to) || !PyBool_Check(args[8]) || !tensor(args[9], &in) ||
      !tensor(args[10], &out) || !tensor(args[11], &count) || !v || (v->dim() != 3 && v->dim() != 4) || !S || S->dim() != 4 || !q || q->dim() < 2 ||
      !on_one_device(*v, {S, q, k, g, o, to, in, out, count}) || !stream_of(args[12], *v, &s))
    Py_RETURN_NONE;
  const auto type = v->scalar_type();
  const bool write = args[8] == Py_True;
  const int64_t nl = v->dim() - 2, H = v->size(-2), dv = v->size(-1), B = v->size(nl - 1), steps = nl == 2 ? v->size(0) : 1;
  const int64_t H_k = q->size(-2), dk = q->size(-1), n_slots = S->size(0);
  const auto lead = v->sizes().slice(0, nl);
  int64_t qs, ks, vs, gs;
  if (code(type) < 0 || !head_rows(v, type, nl, H, dv, &vs) || !head_rows(q, type, nl, H_k, dk, &qs) || q->sizes().slice(0, nl) != lead ||
      !head_rows(k, type, nl, H_k, dk, &ks) || k->sizes().slice(0, nl) != lead || !decays(g, lead, H, &gs) ||
      !dense(S, at::kFloat, {n_slots, H, dk, dv}) || (to && (!write || !dense(to, at::kFloat, {n_slots, H, dk, dv}))) ||
      (in && !dense(in, at::kInt, {B})) || (out && !dense(out, at::kInt, {B})) || (count && !dense(count, at::kInt, {B})) ||
      (o && !dense(o, type, v->sizes())) || !fits_int(steps) || !fits_int(B) || !fits_int(H) || !fits_int(H_k) || !fits_int(dk) || !fits_int(dv))
    Py_RETURN_NONE;
  const c10::cuda::CUDAGuard device(v->device());   // the library launches on the current one
  Tensor made;
  if (!o) {
    const AllocateOn stream(args[12], s, *v);
    made = empty(v->sizes(), type, *v);
    o = &made;
  }
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = kda_linattn_step(static_cast<const float*>(ptr(S)), write ? static_cast<float*>(ptr(to ? to : S)) : nullptr, n_slots,
                            static_cast<const int32_t*>(ptr(in)), static_cast<const int32_t*>(ptr(out)), ptr(q), qs, ptr(k), ks, ptr(v), vs,
                            static_cast<const float*>(ptr(g)), gs, static_cast<const int32_t*>(ptr(count)), (float)scale, ptr(o), (int)steps,
                            (int)B, (int)H, (int)H_k, (int)dk, (int)dv, code(type), s);
  Py_END_ALLOW_THREADS
  return Py_BuildValue("(iN)", status, made.defined() ? THPVariable_Wrap(made) : Py_NewRef(args[6]));
  END_HANDLE_TH_ERRORS
}

// (S0, q, k, v, g, cu_seqlens, scale, o, S_final, ckpt_stride, pages, ckpt_page_ids, ckpt_pos, workspace, stream) ->
// (status, o, S_final); cu_seqlens a list or None, workspace True: allocated here
PyObject* linattn_prefill(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const Tensor *S0, *q, *k, *v, *g, *o, *S, *pages, *ids, *pos, *ws = nullptr;
  double scale;
  int64_t stride;
  kda_stream_t s;
  if (n != 15 || !tensor(args[0], &S0) || !tensor(args[1], &q) || !tensor(args[2], &k) || !tensor(args[3], &v) || !tensor(args[4], &g) ||
      !number(args[6], &scale) || !tensor(args[7], &o) || !tensor(args[8], &S) || !integer(args[9], &stride) || !tensor(args[10], &pages) ||
      !tensor(args[11], &ids) || !tensor(args[12], &pos) || (args[13] != Py_True && !tensor(args[13], &ws)) || !v || v->dim() != 3 || !q ||
      q->dim() != 3 || !on_one_device(*v, {S0, q, k, g, o, S, pages, ids, pos, ws}) || !stream_of(args[14], *v, &s))
    Py_RETURN_NONE;
  std::vector<int32_t> cu;
  if (args[5] != Py_None) {
    if (!PyList_Check(args[5])) Py_RETURN_NONE;
    const Py_ssize_t len = PyList_GET_SIZE(args[5]);
    cu.reserve(len);
    for (Py_ssize_t i = 0; i < len; ++i) {
      int64_t x;
      if (!integer(PyList_GET_ITEM(args[5], i), &x) || !fits_int(x)) Py_RETURN_NONE;
      cu.push_back((int32_t)x);
    }
    if (cu.size() < 2) Py_RETURN_NONE;
  }
  const auto type = v->scalar_type();
  const int64_t T = v->size(0), H = v->size(1), dv = v->size(2), H_k = q->size(1), dk = q->size(2), N = cu.empty() ? 1 : (int64_t)cu.size() - 1;
  int64_t qs, ks, vs, gs;
  if (code(type) < 0 || q->size(0) != T || !k || k->dim() != 3 || k->size(0) != T || !head_rows(v, type, 1, H, dv, &vs) ||
      !head_rows(q, type, 1, H_k, dk, &qs) || !head_rows(k, type, 1, H_k, dk, &ks) || !decays(g, {T}, H, &gs) ||
      (S0 && !dense(S0, at::kFloat, {N, H, dk, dv})) || (o && !dense(o, type, {T, H, dv})) || (S && !dense(S, at::kFloat, {N, H, dk, dv})) ||
      (ids && (!dense(ids, at::kInt, {ids->numel()}) || !pages || pages->dim() != 2 || !dense(pages, at::kByte, pages->sizes()))) ||
      (pos && (!dense(pos, at::kInt, {pos->numel()}) || pos->numel() < (ids ? ids->numel() : 0))) || (ws && !dense(ws, at::kByte, {ws->numel()})) ||
      !fits_int(stride) || !fits_int(N) || !fits_int(H) || !fits_int(H_k) || !fits_int(dk) || !fits_int(dv))
    Py_RETURN_NONE;
  const c10::cuda::CUDAGuard device(v->device());   // the library launches on the current one
  Tensor made_o, made_S, made_ws;
  {
    const AllocateOn stream(args[14], s, *v);
    if (!o) { made_o = empty({T, H, dv}, type, *v); o = &made_o; }
    if (!S) { made_S = empty({N, H, dk, dv}, at::kFloat, *v); S = &made_S; }
    if (args[13] == Py_True) {
      const int64_t need = kda_linattn_prefill_workspace_bytes(cu.empty() ? nullptr : cu.data(), (int)N, T, (int)H, (int)dk, (int)dv, code(type));
      if (need < 0) Py_RETURN_NONE;
      if (need > 0) { made_ws = empty({need}, at::kByte, *v); ws = &made_ws; }
    }
  }
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = kda_linattn_prefill(static_cast<const float*>(ptr(S0)), ptr(q), qs, ptr(k), ks, ptr(v), vs, static_cast<const float*>(ptr(g)), gs,
                               cu.empty() ? nullptr : cu.data(), (int)N, T, (int)H, (int)H_k, (int)dk, (int)dv, code(type), (float)scale,
                               (int)stride, ptr(o), static_cast<float*>(ptr(S)), ids ? ptr(pages) : nullptr, ids ? pages->size(1) : 0,
                               static_cast<const int32_t*>(ptr(ids)), static_cast<int32_t*>(ptr(pos)), ids ? ids->numel() : 0, ptr(ws),
                               ws ? ws->numel() : 0, s);
  Py_END_ALLOW_THREADS
  return Py_BuildValue("(iNN)", status, made_o.defined() ? THPVariable_Wrap(made_o) : Py_NewRef(args[7]),
                       made_S.defined() ? THPVariable_Wrap(made_S) : Py_NewRef(args[8]));
  END_HANDLE_TH_ERRORS
}

// (x, weight, gate, eps, act, gate_first, y, stream) -> (status, y)
PyObject* gated_norm(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const Tensor *x, *weight, *gate, *y;
  double eps;
  int64_t act;
  kda_stream_t s;
  if (n != 8 || !tensor(args[0], &x) || !tensor(args[1], &weight) || !tensor(args[2], &gate) || !number(args[3], &eps) || !integer(args[4], &act) ||
      !PyBool_Check(args[5]) || !tensor(args[6], &y) || !x || x->dim() != 3 || !weight || !on_one_device(*x, {weight, gate, y}) ||
      !stream_of(args[7], *x, &s))
    Py_RETURN_NONE;
  const auto type = x->scalar_type();
  const int64_t T = x->size(0), H = x->size(1), d = x->size(2);
  const bool per_head = weight->dim() == 2;
  int64_t xs, zs = 0;
  if (code(type) < 0 || !head_rows(x, type, 1, H, d, &xs) || (gate && (!head_rows(gate, type, 1, H, d, &zs) || gate->size(0) != T)) ||
      !(per_head ? dense(weight, type, {H, d}) : dense(weight, type, {d})) || (y && !dense(y, type, {T, H, d})) || !fits_int(act) || !fits_int(H) ||
      !fits_int(d))
    Py_RETURN_NONE;
  const c10::cuda::CUDAGuard device(x->device());   // the library launches on the current one
  Tensor made;
  if (!y) {
    const AllocateOn stream(args[7], s, *x);
    made = empty({T, H, d}, type, *x);
    y = &made;
  }
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = kda_gated_norm(ptr(x), xs, ptr(gate), zs, ptr(weight), per_head ? d : 0, (float)eps, (int)act, args[5] == Py_True, ptr(y), T, (int)H,
                          (int)d, code(type), s);
  Py_END_ALLOW_THREADS
  return Py_BuildValue("(iN)", status, made.defined() ? THPVariable_Wrap(made) : Py_NewRef(args[6]));
  END_HANDLE_TH_ERRORS
}

// (h, y, pre_weight, post_weight, gate, channel_scale, res_scale, act, eps, h_out, x, stream) -> (status, h_out or h, x)
PyObject* residual_norm(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const Tensor *h, *y, *pre, *post, *gate, *channel, *to, *x;
  double res_scale, eps;
  int64_t act;
  kda_stream_t s;
  if (n != 12 || !tensor(args[0], &h) || !tensor(args[1], &y) || !tensor(args[2], &pre) || !tensor(args[3], &post) || !tensor(args[4], &gate) ||
      !tensor(args[5], &channel) || !number(args[6], &res_scale) || !integer(args[7], &act) || !number(args[8], &eps) || !tensor(args[9], &to) ||
      !tensor(args[10], &x) || !y || y->dim() != 2 || !h || !on_one_device(*y, {h, pre, post, gate, channel, to, x}) ||
      !stream_of(args[11], *y, &s))
    Py_RETURN_NONE;
  const auto type = y->scalar_type(), h_type = h->scalar_type();
  const int64_t T = y->size(0), D = y->size(1);
  if (code(type) < 0 || code(h_type) < 0 || !rows(y, type, {T, D}) || !rows(h, h_type, {T, D}) || (gate && !rows(gate, type, {T, D})) ||
      (to && (!rows(to, h_type, {T, D}) || (T > 1 && to->stride(0) != h->stride(0)))) || !dense(pre, type, {D}) || (post && !dense(post, type, {D})) ||
      (channel && !dense(channel, type, {D})) || (x && !dense(x, type, {T, D})) || !fits_int(act) || !fits_int(D))
    Py_RETURN_NONE;
  const c10::cuda::CUDAGuard device(y->device());   // the library launches on the current one
  Tensor made;
  if (!x) {
    const AllocateOn stream(args[11], s, *y);
    made = empty({T, D}, type, *y);
    x = &made;
  }
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = kda_residual_norm(ptr(y), T > 1 ? y->stride(0) : D, ptr(gate), gate && T > 1 ? gate->stride(0) : D, ptr(post), ptr(channel),
                             (float)res_scale, ptr(h), ptr(to ? to : h), T > 1 ? h->stride(0) : D, code(h_type), ptr(pre), (float)eps, (int)act,
                             ptr(x), T, (int)D, code(type), s);
  Py_END_ALLOW_THREADS
  return Py_BuildValue("(iNN)", status, Py_NewRef(args[to ? 9 : 0]), made.defined() ? THPVariable_Wrap(made) : Py_NewRef(args[10]));
  END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"linattn_step", reinterpret_cast<PyCFunction>(linattn_step), METH_FASTCALL, nullptr},
    {"linattn_prefill", reinterpret_cast<PyCFunction>(linattn_prefill), METH_FASTCALL, nullptr},
    {"gated_norm", reinterpret_cast<PyCFunction>(gated_norm), METH_FASTCALL, nullptr},
    {"residual_norm", reinterpret_cast<PyCFunction>(residual_norm), METH_FASTCALL, nullptr},
    {"mla_append", reinterpret_cast<PyCFunction>(mla_append), METH_FASTCALL, nullptr},
    {"mla_decode", reinterpret_cast<PyCFunction>(mla_decode), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kda_torch", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__kda_torch(void) { return PyModule_Create(&module); }
