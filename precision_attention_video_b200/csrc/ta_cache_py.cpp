// ta_cache_py.cpp -- the Python entry of the cached-attention operators: reads
// tensors, checks them and calls the C ABI, in about a microsecond (marshalled
// in Python a call costs ten, more than a kernel for single tokens).  A call
// that a check refuses returns None without any work; the Python module then
// makes the same checks again and raises with the reason.
#include <Python.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "tiered_attn_cache.h"

namespace {

// What the Python PagedCache says of itself (the same layout as its ctypes
// structure).
struct CacheView {
  ta_cache c;
  int64_t stride[3];             // page, head, slot
  int64_t shape[4];              // n_pages, Hkv, page_size, d; zeros without keys
  int32_t format, device, has_mean, pad;
};

// The C ABI's entry points, set once by init().
decltype(&tiered_attn_cache_append) g_append;
decltype(&tiered_attn_cache_decode) g_decode;
decltype(&tiered_attn_cache_select) g_select;
decltype(&tiered_attn_cache_sparse) g_sparse;

bool read_struct(PyObject* o, void* dst, Py_ssize_t size) {
  Py_buffer b;
  if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE) != 0) {
    PyErr_Clear();
    return false;
  }
  const bool ok = b.len == size;
  if (ok) memcpy(dst, b.buf, size);
  PyBuffer_Release(&b);
  return ok;
}

struct Call {
  ta_cache_params p;
  CacheView v;
  void* stream;
  bool ok;

  const at::Tensor* tensor(PyObject* o) {
    if (!THPVariable_Check(o)) {
      ok = false;
      return nullptr;
    }
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.get_device() != v.device || t.layout() != at::kStrided) ok = false;
    return &t;
  }
  // A contiguous tensor of this type with these sizes.
  void* plain(PyObject* o, at::ScalarType type, std::initializer_list<int64_t> sizes) {
    const at::Tensor* t = tensor(o);
    if (!ok || t->scalar_type() != type || t->sizes() != at::IntArrayRef(sizes.begin(), sizes.size()) ||
        !t->is_contiguous()) {
      ok = false;
      return nullptr;
    }
    return t->data_ptr();
  }
  // A bf16 [rows, heads, d] tensor, d contiguous.
  void* rows(PyObject* o, int64_t heads, int64_t& st, int64_t& sh) {
    const at::Tensor* t = tensor(o);
    if (!ok || t->scalar_type() != at::kBFloat16 || t->dim() != 3 || t->size(0) != p.T ||
        t->size(1) != heads || t->size(2) != p.d || t->stride(2) != 1) {
      ok = false;
      return nullptr;
    }
    st = t->stride(0);
    sh = t->stride(1);
    return t->data_ptr();
  }
  const int32_t* table(PyObject* o) {
    const at::Tensor* t = tensor(o);
    if (!ok || t->scalar_type() != at::kInt || t->dim() != 2 || t->size(0) != p.S ||
        t->size(1) < p.max_pages || t->stride(1) != 1) {
      ok = false;
      return nullptr;
    }
    p.stride_table = t->stride(0);
    return t->data_ptr<int32_t>();
  }
  const int32_t* ints(PyObject* o, int64_t n) {
    return o == Py_None ? nullptr : static_cast<const int32_t*>(plain(o, at::kInt, {n}));
  }
  void* workspace(PyObject* o, size_t& bytes) {
    const at::Tensor* t = tensor(o);
    if (!ok || t->scalar_type() != at::kByte || t->dim() != 1 || !t->is_contiguous()) {
      ok = false;
      return nullptr;
    }
    bytes = t->numel();
    return t->data_ptr();
  }

  Call(PyObject* params, PyObject* cache, PyObject* strm, bool kv) : stream(nullptr), ok(false) {
    if (!read_struct(params, &p, sizeof p) || !read_struct(cache, &v, sizeof v)) return;
    if (v.device < 0 || v.device != c10::cuda::current_device()) return;
    if (kv && (v.shape[0] != p.n_pages || v.shape[1] != p.Hkv || v.shape[2] != p.page_size ||
               v.shape[3] != p.d || v.format != p.format))
      return;
    p.stride_page = v.stride[0];
    p.stride_head = v.stride[1];
    p.stride_slot = v.stride[2];
    if (strm == Py_None) {
      stream = c10::cuda::getCurrentCUDAStream(v.device).stream();
    } else if (PyLong_Check(strm)) {
      stream = PyLong_AsVoidPtr(strm);
      if (PyErr_Occurred()) {
        PyErr_Clear();
        return;
      }
    } else {
      return;
    }
    ok = true;
  }
};

template <typename F>
PyObject* finish(const Call& c, F f) {
  if (!c.ok) Py_RETURN_NONE;
  ta_status st;
  Py_BEGIN_ALLOW_THREADS
  st = f();
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}

// append(p, cache, K, V, table, lens, ws, cu, cos, sin, pos, Q, Q_out, stream)
PyObject* append(PyObject* const* a, Py_ssize_t n) {
  if (n != 14) Py_RETURN_NONE;
  Call c(a[0], a[1], a[13], true);
  if (!c.ok) Py_RETURN_NONE;
  ta_cache_params& p = c.p;
  size_t wn = 0;
  const void* k = c.rows(a[2], p.Hkv, p.stride_k_t, p.stride_k_h);
  const void* v = c.rows(a[3], p.Hkv, p.stride_v_t, p.stride_v_h);
  const int32_t* table = c.table(a[4]);
  const int32_t* lens = static_cast<int32_t*>(c.plain(a[5], at::kInt, {p.S}));
  void* ws = c.workspace(a[6], wn);
  const int32_t* cu = c.ints(a[7], (int64_t)p.S + 1);
  const float *cos = nullptr, *sin = nullptr;
  if (p.rot_dim) {
    const at::Tensor* t = c.tensor(a[8]);
    if (!c.ok || t->dim() != 2 || t->size(0) > 0x7fffffff) Py_RETURN_NONE;
    p.rot_rows = (int32_t)t->size(0);
    cos = static_cast<float*>(c.plain(a[8], at::kFloat, {p.rot_rows, p.rot_dim / 2}));
    sin = static_cast<float*>(c.plain(a[9], at::kFloat, {p.rot_rows, p.rot_dim / 2}));
  }
  const int32_t* pos = c.ints(a[10], p.T);
  const void* q = nullptr;
  void* qo = nullptr;
  if (a[11] != Py_None) {
    q = c.rows(a[11], p.H, p.stride_q_t, p.stride_q_h);
    qo = c.rows(a[12], p.H, p.stride_o_t, p.stride_o_h);
    if (q == qo && (p.stride_q_t != p.stride_o_t || p.stride_q_h != p.stride_o_h)) c.ok = false;
  }
  return finish(c, [&] { return g_append(&p, &c.v.c, k, v, q, qo, cos, sin, pos, cu, lens, table, ws, wn, c.stream); });
}

// decode(p, cache, Q, table, lens, ws, O, lse, stream)
PyObject* decode(PyObject* const* a, Py_ssize_t n) {
  if (n != 9) Py_RETURN_NONE;
  Call c(a[0], a[1], a[8], true);
  if (!c.ok) Py_RETURN_NONE;
  ta_cache_params& p = c.p;
  size_t wn = 0;
  const void* q = c.rows(a[2], p.H, p.stride_q_t, p.stride_q_h);
  const int32_t* table = c.table(a[3]);
  const int32_t* lens = static_cast<int32_t*>(c.plain(a[4], at::kInt, {p.S}));
  void* ws = c.workspace(a[5], wn);
  void* o = c.rows(a[6], p.H, p.stride_o_t, p.stride_o_h);
  float* lse = a[7] == Py_None ? nullptr : static_cast<float*>(c.plain(a[7], at::kFloat, {p.T, p.H}));
  return finish(c, [&] { return g_decode(&p, &c.v.c, q, lens, table, o, lse, ws, wn, c.stream); });
}

// select(p, cache, Q, table, lens, ws, sel, cu, stream)
PyObject* select(PyObject* const* a, Py_ssize_t n) {
  if (n != 9) Py_RETURN_NONE;
  Call c(a[0], a[1], a[8], false);
  if (!c.ok || !c.v.has_mean) Py_RETURN_NONE;
  ta_cache_params& p = c.p;
  if (c.v.shape[0] != p.n_pages || c.v.shape[1] != p.Hkv || c.v.shape[3] != p.d) Py_RETURN_NONE;
  size_t wn = 0;
  const void* q = c.rows(a[2], p.H, p.stride_q_t, p.stride_q_h);
  const int32_t* table = c.table(a[3]);
  const int32_t* lens = static_cast<int32_t*>(c.plain(a[4], at::kInt, {p.S}));
  void* ws = c.workspace(a[5], wn);
  int32_t* sel = static_cast<int32_t*>(c.plain(a[6], at::kInt, {p.T, p.Hkv, p.n_select}));
  const int32_t* cu = c.ints(a[7], (int64_t)p.S + 1);
  return finish(c, [&] { return g_select(&p, &c.v.c, q, cu, lens, table, sel, ws, wn, c.stream); });
}

// sparse(p, cache, Q, sel, table, lens, ws, O, cu, lse, stream)
PyObject* sparse(PyObject* const* a, Py_ssize_t n) {
  if (n != 11) Py_RETURN_NONE;
  Call c(a[0], a[1], a[10], true);
  if (!c.ok) Py_RETURN_NONE;
  ta_cache_params& p = c.p;
  size_t wn = 0;
  const void* q = c.rows(a[2], p.H, p.stride_q_t, p.stride_q_h);
  const int32_t* sel = static_cast<int32_t*>(c.plain(a[3], at::kInt, {p.T, p.Hkv, p.n_select}));
  const int32_t* table = c.table(a[4]);
  const int32_t* lens = static_cast<int32_t*>(c.plain(a[5], at::kInt, {p.S}));
  void* ws = c.workspace(a[6], wn);
  void* o = c.rows(a[7], p.H, p.stride_o_t, p.stride_o_h);
  const int32_t* cu = c.ints(a[8], (int64_t)p.S + 1);
  float* lse = a[9] == Py_None ? nullptr : static_cast<float*>(c.plain(a[9], at::kFloat, {p.T, p.H}));
  return finish(c, [&] { return g_sparse(&p, &c.v.c, q, sel, cu, lens, table, o, lse, ws, wn, c.stream); });
}

// init(append, decode, select, sparse): addresses of the C ABI's entry points
PyObject* init(PyObject*, PyObject* args) {
  unsigned long long f[4];
  if (!PyArg_ParseTuple(args, "KKKK", &f[0], &f[1], &f[2], &f[3])) return nullptr;
  g_append = reinterpret_cast<decltype(g_append)>(f[0]);
  g_decode = reinterpret_cast<decltype(g_decode)>(f[1]);
  g_select = reinterpret_cast<decltype(g_select)>(f[2]);
  g_sparse = reinterpret_cast<decltype(g_sparse)>(f[3]);
  Py_RETURN_NONE;
}

// No C++ exception leaves an entry: what a tensor's accessor throws (a tensor
// without storage, say) refuses the call like any other check.
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject*, PyObject* const* a, Py_ssize_t n) {
  try {
    return F(a, n);
  } catch (...) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
}
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<F>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    method<append>("append"),
    method<decode>("decode"),
    method<select>("select"),
    method<sparse>("sparse"),
    {"init", init, METH_VARARGS, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_cache_call", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__cache_call() { return PyModule_Create(&module); }
