// The serving calls on torch tensors without the interpreter's share of the
// work: module _serve (CPython), used by the package's functions of the same
// names.  A decoding step of one token takes the GPU 5 to 8 us; reading some
// forty attributes in Python, ctypes and torch.empty take 16, this 6.
//
// Each function checks its arguments as the package does and returns None,
// having done nothing, for any that it does not take: the package's own path
// then handles the call or says what is wrong with it.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "fa.h"

namespace {

decltype(&fa_kv4_write) g_write;
decltype(&fa_kv4_read) g_read;
decltype(&fa_fwd_kv4) g_fwd;
decltype(&fa_fwd_kv4_workspace_size) g_workspace_size;

// A plain contiguous CUDA tensor on device dev, or null.
const at::Tensor* plain(PyObject* x, int dev) {
  if (!THPVariable_CheckExact(x)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(x);
  return t.is_cuda() && t.get_device() == dev && t.is_contiguous() ? &t : nullptr;
}

bool fits(int64_t x) { return x >= 0 && x <= INT_MAX; }

// [B, heads, rows, d] of a 16-bit type on the current device.
struct Rows {
  const at::Tensor* t = nullptr;
  int dev = 0, B = 0, heads = 0, rows = 0, d = 0, dtype = 0;

  bool take(PyObject* x) {
    dev = c10::cuda::current_device();
    t = plain(x, dev);
    if (t == nullptr || t->dim() != 4) return false;
    for (int i = 0; i < 4; ++i)
      if (!fits(t->size(i))) return false;
    B = (int)t->size(0), heads = (int)t->size(1), rows = (int)t->size(2), d = (int)t->size(3);
    if (t->scalar_type() == at::kBFloat16)
      dtype = FA_BF16;
    else if (t->scalar_type() == at::kHalf)
      dtype = FA_FP16;
    else
      return false;
    return true;
  }
};

struct Cache {
  void* pool = nullptr;
  const int* table = nullptr;
  const int* start = nullptr;
  const int* count = nullptr;
  int n_pages = 0, heads = 0, page = 0, d = 0, max_pages = 0, B = 0;

  bool take(PyObject* pool_, PyObject* table_, PyObject* start_, PyObject* count_, int dev) {
    const at::Tensor* p = plain(pool_, dev);
    if (p == nullptr || p->scalar_type() != at::kByte || p->dim() != 4 || p->size(3) % 18 != 0) return false;
    const at::Tensor* t = plain(table_, dev);
    if (t == nullptr || t->scalar_type() != at::kInt || t->dim() != 2) return false;
    if (!fits(p->size(0)) || !fits(p->size(1)) || !fits(16 * p->size(2)) || !fits(p->size(3)) || !fits(t->size(0)) ||
        !fits(t->size(1)))
      return false;
    n_pages = (int)p->size(0), heads = (int)p->size(1), page = 16 * (int)p->size(2), d = (int)p->size(3) / 18;
    B = (int)t->size(0), max_pages = (int)t->size(1);
    pool = p->data_ptr();
    table = static_cast<const int*>(t->data_ptr());
    return per_sequence(start_, dev, &start) && (count_ == Py_None || per_sequence(count_, dev, &count));
  }

  bool per_sequence(PyObject* x, int dev, const int** out) const {
    const at::Tensor* t = plain(x, dev);
    if (t == nullptr || t->scalar_type() != at::kInt || t->dim() != 1 || t->size(0) != B) return false;
    *out = static_cast<const int*>(t->data_ptr());
    return true;
  }
};

void* current_stream(int dev) { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream(); }

// f() must not throw: pointers and streams are looked up before.
template <typename F>
int without_gil(F&& f) {
  int st;
  Py_BEGIN_ALLOW_THREADS
  st = f();
  Py_END_ALLOW_THREADS
  return st;
}

// write(k, v, pool, page_table, start, count) -> status
PyObject* serve_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Rows k, v;
  Cache c;
  if (n != 6 || !k.take(a[0]) || !v.take(a[1]) || !c.take(a[2], a[3], a[4], a[5], k.dev)) Py_RETURN_NONE;
  if (v.t->sizes() != k.t->sizes() || v.dtype != k.dtype) Py_RETURN_NONE;
  if (c.B != k.B || c.heads != k.heads || c.d != k.d) Py_RETURN_NONE;
  const void *pk = k.t->data_ptr(), *pv = v.t->data_ptr();
  void* const stream = current_stream(k.dev);
  return PyLong_FromLong(without_gil([&] {
    return g_write(pk, pv, c.pool, c.table, c.start, c.count, k.B, k.heads, k.rows, k.d, c.n_pages, c.page,
                   c.max_pages, k.dtype, stream);
  }));
  END_HANDLE_TH_ERRORS
}

// read(pool, page_table, start, count, N, dtype) -> (k, v) or status
PyObject* serve_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const int dev = c10::cuda::current_device();
  Cache c;
  if (n != 6 || !c.take(a[0], a[1], a[2], a[3], dev) || !PyLong_Check(a[4]) || !THPDtype_Check(a[5])) Py_RETURN_NONE;
  int over = 0;
  const long long rows = PyLong_AsLongLongAndOverflow(a[4], &over);
  const at::ScalarType type = reinterpret_cast<THPDtype*>(a[5])->scalar_type;
  if (over != 0 || rows <= 0 || !fits(rows) || (type != at::kBFloat16 && type != at::kHalf)) Py_RETURN_NONE;
  const auto options = at::TensorOptions().dtype(type).device(at::kCUDA, (c10::DeviceIndex)dev);
  const at::Tensor k = at::empty({c.B, c.heads, rows, c.d}, options), v = at::empty({c.B, c.heads, rows, c.d}, options);
  void *const pk = k.data_ptr(), *const pv = v.data_ptr(), *const stream = current_stream(dev);
  const int st = without_gil([&] {
    return g_read(c.pool, c.table, c.start, c.count, pk, pv, c.B, c.heads, (int)rows, c.d, c.n_pages, c.page,
                  c.max_pages, type == at::kBFloat16 ? FA_BF16 : FA_FP16, stream);
  });
  if (st != FA_OK) return PyLong_FromLong(st);
  return Py_BuildValue("(NN)", THPVariable_Wrap(k), THPVariable_Wrap(v));
  END_HANDLE_TH_ERRORS
}

// fwd(q, pool, page_table, start, count, o, lse, workspace, scale, causal, o_fp32) -> (o, lse) or status
PyObject* serve_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Rows q;
  Cache c;
  if (n != 11 || !q.take(a[0]) || !c.take(a[1], a[2], a[3], a[4], q.dev)) Py_RETURN_NONE;
  if (c.B != q.B || c.d != q.d || c.heads < 1 || q.heads % c.heads != 0) Py_RETURN_NONE;
  double scale = 1.0 / std::sqrt((double)q.d);
  if (a[8] != Py_None) {
    if (!PyFloat_Check(a[8])) Py_RETURN_NONE;
    scale = PyFloat_AsDouble(a[8]);
  }
  const int causal = PyObject_IsTrue(a[9]), o_fp32 = PyObject_IsTrue(a[10]);
  if (causal < 0 || o_fp32 < 0) return nullptr;

  const at::Tensor *o = nullptr, *lse = nullptr, *ws = nullptr;
  if (a[5] != Py_None) {
    o = plain(a[5], q.dev);
    if (o == nullptr || o->sizes() != q.t->sizes() ||
        (o->scalar_type() != q.t->scalar_type() && o->scalar_type() != at::kFloat))
      Py_RETURN_NONE;
  }
  if (a[6] != Py_None) {
    lse = plain(a[6], q.dev);
    if (lse == nullptr || lse->scalar_type() != at::kFloat || lse->dim() != 3 || lse->size(0) != q.B ||
        lse->size(1) != q.heads || lse->size(2) != q.rows)
      Py_RETURN_NONE;
  }
  if (a[7] != Py_None && (ws = plain(a[7], q.dev)) == nullptr) Py_RETURN_NONE;

  const auto options = at::TensorOptions().device(at::kCUDA, (c10::DeviceIndex)q.dev);
  at::Tensor new_o, new_lse, new_ws;
  if (o == nullptr) {
    new_o = at::empty(q.t->sizes(), options.dtype(o_fp32 ? at::kFloat : q.t->scalar_type()));
    o = &new_o;
  }
  if (lse == nullptr) {
    new_lse = at::empty({q.B, q.heads, q.rows}, options.dtype(at::kFloat));
    lse = &new_lse;
  }
  if (ws == nullptr) {
    new_ws = at::empty({(int64_t)g_workspace_size(q.B, q.heads, c.heads, q.rows, q.d)}, options.dtype(at::kByte));
    ws = &new_ws;
  }
  const bool o32 = o->scalar_type() == at::kFloat;
  const int dtype = q.dtype == FA_BF16 ? (o32 ? FA_BF16_O_F32 : FA_BF16) : (o32 ? FA_FP16_O_F32 : FA_FP16);
  const void* const pq = q.t->data_ptr();
  void *const po = o->data_ptr(), *const pl = lse->data_ptr(), *const pw = ws->data_ptr();
  void* const stream = current_stream(q.dev);
  const size_t ws_bytes = ws->nbytes();
  const int st = without_gil([&] {
    return g_fwd(pq, c.pool, c.table, c.start, c.count, po, static_cast<float*>(pl), pw, ws_bytes, q.B, q.heads,
                 c.heads, q.rows, q.d, c.n_pages, c.page, c.max_pages, (float)scale, causal, dtype, stream);
  });
  if (st != FA_OK) return PyLong_FromLong(st);
  return Py_BuildValue("(NN)", a[5] != Py_None ? Py_NewRef(a[5]) : THPVariable_Wrap(new_o),
                       a[6] != Py_None ? Py_NewRef(a[6]) : THPVariable_Wrap(new_lse));
  END_HANDLE_TH_ERRORS
}

// connect(write, read, fwd, workspace_size): the library's entry points, as addresses.
PyObject* serve_connect(PyObject*, PyObject* args) {
  unsigned long long w, r, f, s;
  if (!PyArg_ParseTuple(args, "KKKK", &w, &r, &f, &s)) return nullptr;
  g_write = reinterpret_cast<decltype(g_write)>(w);
  g_read = reinterpret_cast<decltype(g_read)>(r);
  g_fwd = reinterpret_cast<decltype(g_fwd)>(f);
  g_workspace_size = reinterpret_cast<decltype(g_workspace_size)>(s);
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"connect", serve_connect, METH_VARARGS, "connect(write, read, fwd, workspace_size): addresses of the entry points"},
    {"write", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(serve_write)), METH_FASTCALL,
     "write(k, v, pool, page_table, start, count) -> status, or None"},
    {"read", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(serve_read)), METH_FASTCALL,
     "read(pool, page_table, start, count, N, dtype) -> (k, v), status or None"},
    {"fwd", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(serve_fwd)), METH_FASTCALL,
     "fwd(q, pool, page_table, start, count, o, lse, workspace, scale, causal, o_fp32) -> (o, lse), status or None"},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_serve", "Serving calls on torch tensors.", -1, methods,
                      nullptr,               nullptr,  nullptr,                           nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serve() { return PyModule_Create(&module); }
