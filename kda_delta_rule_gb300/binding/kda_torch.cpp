// The latent page cache's calls from Python without Python's share of the work.
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

PyMethodDef methods[] = {
    {"mla_append", reinterpret_cast<PyCFunction>(mla_append), METH_FASTCALL, nullptr},
    {"mla_decode", reinterpret_cast<PyCFunction>(mla_decode), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kda_torch", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__kda_torch(void) { return PyModule_Create(&module); }
