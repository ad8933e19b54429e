// Python binding of the attention-layer operators: checks of the tensors, allocation of the outputs, the
// current stream, and the call into libgdr. A decoding step makes these calls once a layer on kernels of
// a few microseconds, so the marshalling is compiled: the same checks written in Python with ctypes took
// 11 to 22 us a call on a Grace core. Only CPython's and torch's C++ interfaces are used; nothing is
// computed here.
#include <Python.h>
#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cmath>
#include <initializer_list>

#include "gdr.h"

namespace {

using at::Tensor;
struct Error {};   // a Python exception has been set

[[noreturn]] void refuse(const char* fmt, const char* name = "") {
  PyErr_Format(PyExc_ValueError, fmt, name);
  throw Error{};
}

// The library counts in 32 bits: nothing is cut to them.
int int32(int64_t x, const char* name) {
  if (x < INT_MIN || x > INT_MAX) refuse("%s does not fit in 32 bits", name);
  return (int)x;
}
int size(const Tensor& t, int dim, const char* name) { return int32(t.size(dim), name); }

// A call's arguments, of which the last is the launch stream: its raw handle, or None for the current one.
struct Call {
  PyObject* const* args;
  bool given;              // a stream
  cudaStream_t handle;
  mutable c10::DeviceIndex device = -1;   // the tensors'
  Call(PyObject* const* args, int last) : args(args), given(args[last] != Py_None), handle(nullptr) {
    if (given) handle = static_cast<cudaStream_t>(PyLong_AsVoidPtr(args[last]));
    if (PyErr_Occurred()) throw Error{};
  }
  // argument i (NULL for None where that is allowed)
  const Tensor* tensor(int i, const char* name, bool none = false) const {
    if (none && args[i] == Py_None) return nullptr;
    if (!THPVariable_Check(args[i])) refuse("%s must be a tensor", name);
    const Tensor& t = THPVariable_Unpack(args[i]);
    if (!t.is_cuda()) refuse("%s must be a CUDA tensor", name);
    if (device < 0) device = t.device().index();
    if (t.device().index() != device) refuse("%s must be on the device of the other tensors", name);
    return &t;
  }
  // contiguous, of this type and shape (empty: any)
  const Tensor* of(int i, const char* name, at::ScalarType type, at::IntArrayRef shape = {}, bool none = false) const {
    const Tensor* t = tensor(i, name, none);
    if (!t) return t;
    if (t->scalar_type() != type) refuse("%s has the wrong dtype", name);
    if (!t->is_contiguous()) refuse("%s must be contiguous", name);
    if (!shape.empty() && t->sizes() != shape) refuse("%s has the wrong shape", name);
    return t;
  }
  const Tensor* ints(int i, const char* name, at::IntArrayRef shape = {}, bool none = false) const {
    return of(i, name, at::kInt, shape, none);
  }
  double number(int i) const {
    const double x = PyFloat_AsDouble(args[i]);
    if (x == -1.0 && PyErr_Occurred()) throw Error{};
    return x;
  }
  int integer(int i, const char* name) const {
    const long x = PyLong_AsLong(args[i]);
    if (x == -1 && PyErr_Occurred()) throw Error{};
    return int32(x, name);
  }
  bool truth(int i) const {
    const int x = PyObject_IsTrue(args[i]);
    if (x < 0) throw Error{};
    return x == 1;
  }
  gdr_stream_t stream() const {
    if (c10::cuda::current_device() != device) refuse("the tensors must be on the current CUDA device");
    return reinterpret_cast<gdr_stream_t>(given ? handle : c10::cuda::getCurrentCUDAStream(device).stream());
  }
  // A new tensor, of the launch stream's memory: the allocator hands memory out again in the order of the
  // stream it was taken for, so a workspace that is dropped when the call returns, or an output that the
  // caller drops, is not given to anyone whose work does not come after the kernels. An output (kept) may be
  // read on the current stream as well, and is not handed out again before that stream is past the reads.
  Tensor empty(at::IntArrayRef shape, at::ScalarType type, const Tensor& near, bool kept) const {
    const auto options = near.options().dtype(type);
    if (!given) return at::empty(shape, options);
    struct Back {   // the current stream, set again on the way out
      c10::cuda::CUDAStream stream;
      ~Back() { c10::cuda::setCurrentCUDAStream(stream); }
    } back{c10::cuda::getCurrentCUDAStream(device)};
    c10::cuda::setCurrentCUDAStream(c10::cuda::getStreamFromExternal(handle, device));
    Tensor t = at::empty(shape, options);
    if (kept) t.record_stream(back.stream.unwrap());
    return t;
  }
  // an output: the caller's, or a new one like `near`
  Tensor output(int i, const char* name, at::IntArrayRef shape, at::ScalarType type, const Tensor& near) const {
    if (args[i] == Py_None) return empty(shape, type, near, true);
    return *of(i, name, type, shape);
  }
  Tensor workspace(int i, size_t bytes, const Tensor& near) const {
    if (args[i] == Py_None) return empty({(int64_t)(bytes < 16 ? 16 : bytes)}, at::kByte, near, false);
    const Tensor* t = tensor(i, "ws");   // (its elements have to be its memory: a workspace is written as bytes)
    if (!t->is_contiguous()) refuse("%s must be contiguous", "ws");
    return *t;
  }
};

void* ptr(const Tensor* t) { return t ? t->data_ptr() : nullptr; }
template <typename T>
T* ptr(const Tensor* t) { return static_cast<T*>(ptr(t)); }
size_t bytes_of(const Tensor& t) { return (size_t)t.numel() * t.element_size(); }

gdr_dtype dtype(const Tensor& t, const char* name) {
  if (t.scalar_type() == at::kBFloat16) return GDR_BF16;
  if (t.scalar_type() != at::kFloat) {
    PyErr_Format(PyExc_TypeError, "%s must be float32 or bfloat16", name);
    throw Error{};
  }
  return GDR_F32;
}

// Raises the library's error as the Python side does.
void check(gdr_status st) {
  if (st == GDR_OK) return;
  PyObject* m = PyImport_ImportModule("gated_deltanet_rule_gb300.gdr");
  PyObject* r = m ? PyObject_CallMethod(m, "_check", "i", (int)st) : nullptr;
  Py_XDECREF(r);
  Py_XDECREF(m);
  if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, gdr_status_string(st));
  throw Error{};
}

PyObject* wrap(std::initializer_list<Tensor> ts) {
  PyObject* t = PyTuple_New(ts.size());
  if (!t) throw Error{};
  Py_ssize_t i = 0;
  for (const Tensor& x : ts) {
    PyObject* o = THPVariable_Wrap(x);
    if (!o) {
      Py_DECREF(t);
      throw Error{};
    }
    PyTuple_SET_ITEM(t, i++, o);
  }
  return t;
}

// Strides (token, head) of [B, N, H, D], which may be a slice of a wider projection.
struct Heads {
  long long tok, head;
};
Heads heads(const Tensor& t, const char* name, const Tensor& like) {
  if (t.dim() != 4) refuse("%s must be [B, N, H, D]", name);
  const int64_t B = t.size(0), N = t.size(1), H = t.size(2), D = t.size(3);
  if (t.scalar_type() != like.scalar_type() || B != like.size(0) || N != like.size(1) || D != like.size(3))
    refuse("%s must share q's dtype, rows, tokens and head dimension", name);
  if (D > 1 && t.stride(3) != 1) refuse("%s: the last dimension must be contiguous", name);
  const int64_t tok = N > 1 ? t.stride(1) : B > 1 ? t.stride(0) : H * D;
  if (B > 1 && N > 1 && t.stride(0) != N * tok) refuse("%s: tokens of all rows must lie at one stride", name);
  return {tok, H > 1 ? t.stride(2) : D};
}

struct Rope {
  const Tensor *q, *k, *q_w, *k_w, *inv_freq, *pos;
  Heads qs, ks;
  int B, N, Hq, Hk, D, R;
  gdr_dtype dt;
  // arguments i .. i + 5: q, k, q_w, k_w, inv_freq, pos
  Rope(const Call& c, int i) {
    q = c.tensor(i, "q");
    k = c.tensor(i + 1, "k");
    qs = heads(*q, "q", *q);
    ks = heads(*k, "k", *q);
    B = size(*q, 0, "q's size");
    N = size(*q, 1, "q's size");
    Hq = size(*q, 2, "q's size");
    Hk = size(*k, 2, "k's size");
    D = size(*q, 3, "q's size");
    dt = dtype(*q, "q and k");
    q_w = c.of(i + 2, "q_w", at::kFloat, {q->size(3)});
    k_w = c.of(i + 3, "k_w", at::kFloat, {q->size(3)});
    inv_freq = c.of(i + 4, "inv_freq", at::kDouble);
    if (inv_freq->dim() != 1) refuse("inv_freq must be [R / 2]");
    pos = c.ints(i + 5, "pos", {q->size(0), q->size(1)});
    R = int32(2 * inv_freq->size(0), "inv_freq's size");
  }
};

struct Pages {
  const Tensor *k, *v, *table, *ctx;
  int P, page, Hk, M;
  // arguments i .. i + 3: k_pages, v_pages, table, ctx
  Pages(const Call& c, int i, const Tensor& q) {
    k = c.of(i, "k_pages", q.scalar_type());
    if (k->dim() != 4 || k->size(3) != q.size(3)) refuse("k_pages must be [P, page, Hk, D] with q's head dimension");
    v = c.of(i + 1, "v_pages", q.scalar_type(), k->sizes());
    table = c.ints(i + 2, "table");
    if (table->dim() != 2 || table->size(0) != q.size(0)) refuse("table must be [B, M]");
    ctx = c.ints(i + 3, "ctx", {q.size(0)});
    P = size(*k, 0, "k_pages' size");
    page = size(*k, 1, "k_pages' size");
    Hk = size(*k, 2, "k_pages' size");
    M = size(*table, 1, "table's size");
  }
};

// q, k, q_w, k_w, inv_freq, pos, eps, interleaved, q_out, k_out, stream
PyObject* norm_rope(const Call& c) {
  const Rope r(c, 0);
  const float eps = (float)c.number(6);
  const bool interleaved = c.truth(7);
  Tensor q_out = c.output(8, "q_out", r.q->sizes(), r.q->scalar_type(), *r.q);
  Tensor k_out = c.output(9, "k_out", r.k->sizes(), r.q->scalar_type(), *r.q);
  check(gdr_qk_norm_rope(ptr(r.q), ptr(r.k), ptr<float>(r.q_w), ptr<float>(r.k_w), ptr<double>(r.inv_freq),
                         ptr<int32_t>(r.pos), eps, interleaved, q_out.data_ptr(), k_out.data_ptr(), r.B, r.N,
                         r.Hq, r.Hk, r.D, r.R, r.qs.tok, r.qs.head, r.ks.tok, r.ks.head, r.dt, c.stream()));
  return wrap({q_out, k_out});
}

// q, k, q_w, k_w, inv_freq, pos, v, k_pages, v_pages, table, ctx, lengths, eps, interleaved, q_out, stream
PyObject* norm_rope_append(const Call& c) {
  const Rope r(c, 0);
  const float eps = (float)c.number(12);
  const bool interleaved = c.truth(13);
  const Tensor* v = c.tensor(6, "v");
  const Heads vs = heads(*v, "v", *r.q);
  const Pages p(c, 7, *r.q);
  if (v->size(2) != r.Hk || p.Hk != r.Hk) refuse("v and the pages must have k's heads");
  const Tensor* lengths = c.ints(11, "lengths", {r.q->size(0)}, true);
  Tensor q_out = c.output(14, "q_out", r.q->sizes(), r.q->scalar_type(), *r.q);
  check(gdr_qk_norm_rope_append(ptr(r.q), ptr(r.k), ptr(v), ptr<float>(r.q_w), ptr<float>(r.k_w), ptr<double>(r.inv_freq),
                                ptr<int32_t>(r.pos), eps, interleaved, q_out.data_ptr(), ptr(p.k), ptr(p.v),
                                ptr<int32_t>(p.table), ptr<int32_t>(p.ctx), ptr<int32_t>(lengths), p.P, p.page, p.M, r.B,
                                r.N, r.Hq, r.Hk, r.D, r.R, r.qs.tok, r.qs.head, r.ks.tok, r.ks.head, vs.tok, vs.head, r.dt,
                                c.stream()));
  return THPVariable_Wrap(q_out);
}

// q, k, q_w, k_w, inv_freq, pos, dq_out, dk_out, eps, interleaved, ws, stream
PyObject* norm_rope_backward(const Call& c) {
  const Rope r(c, 0);
  const float eps = (float)c.number(8);
  const bool interleaved = c.truth(9);
  const Tensor *dqo = c.of(6, "dq_out", r.q->scalar_type(), r.q->sizes()), *dko = c.of(7, "dk_out", r.q->scalar_type(), r.k->sizes());
  Tensor ws = c.workspace(10, gdr_qk_norm_rope_backward_workspace_bytes(r.D), *r.q);
  auto grad = [&](at::IntArrayRef shape) { return c.empty(shape, at::kFloat, *r.q, true); };
  Tensor dq = grad(r.q->sizes()), dk = grad(r.k->sizes()), dq_w = grad({r.q->size(3)}), dk_w = grad({r.q->size(3)});
  check(gdr_qk_norm_rope_backward(ptr(r.q), ptr(r.k), ptr<float>(r.q_w), ptr<float>(r.k_w), ptr<double>(r.inv_freq),
                                  ptr<int32_t>(r.pos), ptr(dqo), ptr(dko), eps, interleaved, ptr<float>(&dq),
                                  ptr<float>(&dk), ptr<float>(&dq_w), ptr<float>(&dk_w), r.B, r.N, r.Hq, r.Hk, r.D, r.R,
                                  r.qs.tok, r.qs.head, r.ks.tok, r.ks.head, r.dt, ws.data_ptr(), bytes_of(ws), c.stream()));
  return wrap({dq, dk, dq_w, dk_w});
}

// q, k_pages, v_pages, table, ctx, lengths, mask, scale, o, lse, want_lse, ws, stream
PyObject* tree_attn(const Call& c) {
  const Tensor* q = c.of(0, "q", at::kBFloat16);
  if (q->dim() != 4) refuse("q must be [B, N, Hq, D]");
  const int B = size(*q, 0, "q's size"), N = size(*q, 1, "q's size"), Hq = size(*q, 2, "q's size"), D = size(*q, 3, "q's size");
  const Pages p(c, 1, *q);
  const Tensor* lengths = c.ints(5, "lengths", {B}, true);
  const Tensor* mask = c.of(6, "mask", at::kLong, {B, N, ((int64_t)N + 63) / 64}, true);
  const double scale = c.args[7] == Py_None ? 1.0 / std::sqrt((double)D) : c.number(7);
  Tensor o = c.output(8, "o", q->sizes(), at::kBFloat16, *q), lse;
  const bool with_lse = c.args[9] != Py_None || c.truth(10);
  if (with_lse) lse = c.output(9, "lse", {B, N, Hq}, at::kFloat, *q);
  Tensor ws = c.workspace(11, gdr_tree_attn_workspace_bytes(D), *q);
  check(gdr_tree_attn(ptr(q), ptr(p.k), ptr(p.v), ptr<int32_t>(p.table), ptr<int32_t>(p.ctx), ptr<int32_t>(lengths),
                      ptr<uint64_t>(mask), (float)scale, o.data_ptr(), with_lse ? ptr<float>(&lse) : nullptr, B, N, Hq,
                      p.Hk, D, p.P, p.page, p.M, GDR_BF16, ws.data_ptr(), bytes_of(ws), c.stream()));
  return with_lse ? wrap({o, lse}) : THPVariable_Wrap(o);
}

// tokens, parents, lengths, p, q, u, u_next, path, n_path, next_token, stream
PyObject* verify(const Call& c) {
  const Tensor* p = c.tensor(3, "p");
  const gdr_dtype dt = dtype(*p, "p");
  if (p->dim() != 3 || !p->is_contiguous()) refuse("p must be a contiguous tensor [B, N, V]");
  const int B = size(*p, 0, "p's size"), N = size(*p, 1, "p's size"), V = size(*p, 2, "p's size");
  const Tensor* q = c.of(4, "q", p->scalar_type(), p->sizes(), true);
  const Tensor *tokens = c.ints(0, "tokens", {B, N}), *parents = c.ints(1, "parents", {B, N}), *lengths = c.ints(2, "lengths", {B});
  const Tensor *u = c.of(5, "u", at::kFloat, {B, N}), *u_next = c.of(6, "u_next", at::kFloat, {B});
  Tensor path = c.output(7, "path", {B, N}, at::kInt, *p), n_path = c.output(8, "n_path", {B}, at::kInt, *p);
  Tensor next = c.output(9, "next_token", {B}, at::kInt, *p);
  check(gdr_verify_draft(ptr<int32_t>(tokens), ptr<int32_t>(parents), ptr<int32_t>(lengths), ptr(p), ptr(q), ptr<float>(u),
                         ptr<float>(u_next), ptr<int32_t>(&path), ptr<int32_t>(&n_path), ptr<int32_t>(&next), B, N, V,
                         dt, c.stream()));
  return wrap({path, n_path, next});
}

struct Cache {
  const Tensor *k, *v;
  int layers, P, page;
  long long row_bytes;
  Cache(const Call& c, int i) {
    k = c.tensor(i, "k_cache");
    if (k->dim() != 5 || !k->is_contiguous()) refuse("k_cache must be a contiguous tensor [layers, P, page, Hk, D]");
    v = c.of(i + 1, "v_cache", k->scalar_type(), k->sizes());
    layers = size(*k, 0, "k_cache's size");
    P = size(*k, 1, "k_cache's size");
    page = size(*k, 2, "k_cache's size");
    row_bytes = (long long)k->size(3) * k->size(4) * k->element_size();
  }
};
struct Rows {
  const Tensor *table, *ctx, *refs, *list;
  int F, R, M, P;
  // arguments i .. i + 2: table, ctx, refs; j: the row list
  Rows(const Call& c, int i, int j, const char* name) {
    table = c.ints(i, "table");
    if (table->dim() != 2) refuse("table must be [rows, M]");
    ctx = c.ints(i + 1, "ctx", {table->size(0)});
    refs = c.ints(i + 2, "refs");
    list = c.ints(j, name);
    if (refs->dim() != 1 || list->dim() != 1) refuse("refs must be [P] and row lists [F]");
    F = size(*list, 0, name);
    R = size(*table, 0, "table's size");
    M = size(*table, 1, "table's size");
    P = size(*refs, 0, "refs' size");
  }
};

// table, ctx, refs, rows, extra, page, ws, stream
PyObject* cache_reserve(const Call& c) {
  const Rows r(c, 0, 3, "rows");
  const int extra = c.integer(4, "extra"), page = c.integer(5, "page");
  Tensor ws = c.workspace(6, gdr_cache_workspace_bytes(r.F, r.M), *r.table);
  check(gdr_cache_reserve(ptr<int32_t>(r.table), ptr<int32_t>(r.ctx), ptr<int32_t>(r.refs), ptr<int32_t>(r.list),
                          extra, r.F, r.R, r.M, r.P, page, ws.data_ptr(), bytes_of(ws), c.stream()));
  Py_RETURN_NONE;
}

// k_cache, v_cache, table, ctx, refs, src, dst, ws, stream
PyObject* cache_fork(const Call& c) {
  const Cache k(c, 0);
  const Rows r(c, 2, 6, "dst");
  const Tensor* src = c.ints(5, "src", r.list->sizes());
  if (r.P != k.P) refuse("refs must be [P]");
  Tensor ws = c.workspace(7, gdr_cache_workspace_bytes(r.F, r.M), *r.table);
  check(gdr_cache_fork(ptr(k.k), ptr(k.v), ptr<int32_t>(r.table), ptr<int32_t>(r.ctx), ptr<int32_t>(r.refs),
                       ptr<int32_t>(src), ptr<int32_t>(r.list), r.F, r.R, r.M, k.layers, k.P, k.page, k.row_bytes,
                       ws.data_ptr(), bytes_of(ws), c.stream()));
  Py_RETURN_NONE;
}

// table, ctx, refs, rows, stream
PyObject* cache_free(const Call& c) {
  const Rows r(c, 0, 3, "rows");
  check(gdr_cache_free(ptr<int32_t>(r.table), ptr<int32_t>(r.ctx), ptr<int32_t>(r.refs), ptr<int32_t>(r.list), r.F, r.R,
                       r.M, r.P, c.stream()));
  Py_RETURN_NONE;
}

// k_cache, v_cache, table, ctx, path, n_path, new_ctx, stream
PyObject* cache_compact(const Call& c) {
  const Cache k(c, 0);
  const Tensor* path = c.ints(4, "path");
  if (path->dim() != 2) refuse("path must be [B, W]");
  const int B = size(*path, 0, "path's size"), W = size(*path, 1, "path's size");
  const Tensor *table = c.ints(2, "table"), *ctx = c.ints(3, "ctx", {B}), *n_path = c.ints(5, "n_path", {B});
  if (table->dim() != 2 || table->size(0) != B) refuse("table must be [B, M]");
  const int M = size(*table, 1, "table's size");
  Tensor new_ctx = c.output(6, "new_ctx", {B}, at::kInt, *ctx);
  check(gdr_cache_compact(ptr(k.k), ptr(k.v), ptr<int32_t>(table), ptr<int32_t>(ctx), ptr<int32_t>(path),
                          ptr<int32_t>(n_path), ptr<int32_t>(&new_ctx), B, W, M, k.layers, k.P, k.page,
                          k.row_bytes, c.stream()));
  return THPVariable_Wrap(new_ctx);
}

// No C++ exception leaves a call.
template <PyObject* (*kFn)(const Call&), int kArgs>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != kArgs) {
    PyErr_Format(PyExc_TypeError, "%d arguments expected, %zd given", kArgs, n);
    return nullptr;
  }
  try {
    return kFn(Call(args, kArgs - 1));
  } catch (const Error&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

#define GDR_ENTRY(fn, n) {#fn, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(&entry<fn, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {GDR_ENTRY(norm_rope, 11),   GDR_ENTRY(norm_rope_append, 16), GDR_ENTRY(norm_rope_backward, 12),
                         GDR_ENTRY(tree_attn, 13),   GDR_ENTRY(verify, 11),           GDR_ENTRY(cache_reserve, 8),
                         GDR_ENTRY(cache_fork, 9),   GDR_ENTRY(cache_free, 5),        GDR_ENTRY(cache_compact, 8),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_gdr_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__gdr_bind(void) { return PyModule_Create(&module); }
