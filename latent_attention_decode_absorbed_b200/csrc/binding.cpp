// Python entry points of the drafted-step calls: each takes its arguments in
// the order of include/mla.h (tensors, integer addresses or None for
// pointers) and returns the status code.  A serving loop makes these calls
// every step and layer, and their kernels take a few microseconds: marshalling
// through ctypes costs about as much as the launch itself (append by slot on a
// B200, back to back: 6.5 us a call through ctypes, 3.5 us through here).
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "mla.h"

namespace {

PyObject* g_data_ptr = nullptr;      // "data_ptr"
PyObject* g_cuda_stream = nullptr;   // "cuda_stream"
PyObject* g_device = nullptr;        // callables set by set_stream_getters: the current device,
PyObject* g_raw_stream = nullptr;    // and a device's current stream as an integer

// Reads the arguments of one call in order; `ok` goes false at the first bad
// one, with the Python error set.
struct Reader {
  PyObject* const* args;
  Py_ssize_t at = 0;
  bool ok = true;

  void* ptr() {
    PyObject* a = args[at++];
    if (!ok || a == Py_None) return nullptr;
    if (PyLong_Check(a)) return address(a);
    PyObject* r = PyObject_CallMethodNoArgs(a, g_data_ptr);
    if (!r) {
      ok = false;
      return nullptr;
    }
    void* p = address(r);
    Py_DECREF(r);
    return p;
  }
  int num() {
    PyObject* a = args[at++];
    if (!ok) return 0;
    int over = 0;
    const long v = PyLong_AsLongAndOverflow(a, &over);
    if (v == -1 && PyErr_Occurred()) ok = false;
    else if (over || v != (long)(int)v) {
      PyErr_SetString(PyExc_OverflowError, "argument does not fit a C int");
      ok = false;
    }
    return (int)v;
  }
  float real() {
    PyObject* a = args[at++];
    if (!ok) return 0.f;
    const double v = PyFloat_AsDouble(a);
    if (v == -1.0 && PyErr_Occurred()) ok = false;
    return (float)v;
  }
  // None: the current stream of the current device
  cudaStream_t stream() {
    PyObject* a = args[at++];
    if (!ok) return nullptr;
    if (PyLong_Check(a)) return static_cast<cudaStream_t>(address(a));
    PyObject* r = nullptr;
    if (a != Py_None) {
      r = PyObject_GetAttr(a, g_cuda_stream);
    } else if (!g_raw_stream) {
      PyErr_SetString(PyExc_RuntimeError, "no stream given and no current stream known");
    } else if (PyObject* dev = PyObject_CallNoArgs(g_device)) {
      r = PyObject_CallOneArg(g_raw_stream, dev);
      Py_DECREF(dev);
    }
    if (!r) {
      ok = false;
      return nullptr;
    }
    auto st = static_cast<cudaStream_t>(address(r));
    Py_DECREF(r);
    return st;
  }
  template <typename T>
  T* as() { return static_cast<T*>(ptr()); }
  mla_dtype dtype() { return static_cast<mla_dtype>(num()); }

 private:
  void* address(PyObject* a) {
    void* p = PyLong_AsVoidPtr(a);
    if (!p && PyErr_Occurred()) ok = false;
    return p;
  }
};

// Calls F on the arguments that `read` takes from the reader, in order.
#define MLA_ENTRY(name, count, ...)                                                                   \
  PyObject* name(PyObject*, PyObject* const* args, Py_ssize_t n) {                                    \
    if (n != (count)) {                                                                               \
      PyErr_Format(PyExc_TypeError, "mla_" #name " takes %d arguments, got %zd", (int)(count), n);    \
      return nullptr;                                                                                 \
    }                                                                                                 \
    Reader r{args};                                                                                   \
    __VA_ARGS__                                                                                       \
  }
// (other threads run meanwhile: a launch may wait for room in the stream's queue)
#define MLA_CALL(expr)        \
  if (!r.ok) return nullptr;  \
  mla_status status;          \
  Py_BEGIN_ALLOW_THREADS      \
  status = (expr);            \
  Py_END_ALLOW_THREADS        \
  return PyLong_FromLong(static_cast<long>(status));

MLA_ENTRY(step_plan, 23, {
  auto* lens = r.as<const int32_t>(); auto* counts = r.as<const int32_t>(); auto* parents = r.as<const int32_t>();
  const int batch = r.num(), max_rows = r.num(), words = r.num();
  auto* held_in = r.as<const int32_t>(); auto* held_out = r.as<int32_t>(); auto* free_pages = r.as<int32_t>();
  auto* fc_in = r.as<const int32_t>(); auto* fc_out = r.as<int32_t>(); auto* table = r.as<int32_t>();
  const int max_pages = r.num(), page = r.num(), num_pages = r.num();
  auto* row_start = r.as<int32_t>(); auto* kv_lens = r.as<int32_t>(); auto* seq_ids = r.as<int32_t>();
  auto* positions = r.as<int32_t>(); auto* slots = r.as<int32_t>(); auto* mask = r.as<uint64_t>();
  auto* err = r.as<int32_t>(); auto stream = r.stream();
  MLA_CALL(mla_step_plan(lens, counts, parents, batch, max_rows, words, held_in, held_out, free_pages, fc_in, fc_out,
                         table, max_pages, page, num_pages, row_start, kv_lens, seq_ids, positions, slots, mask, err,
                         stream))
})

MLA_ENTRY(cache_append_slots, 16, {
  auto* kv = r.as<const void>(); const mla_dtype kv_dtype = r.dtype(); const int n = r.num();
  auto* slots = r.as<const int32_t>(); auto* positions = r.as<const int32_t>(); auto* gain = r.as<const float>();
  const float eps = r.real();
  auto* cos = r.as<const float>(); auto* sin = r.as<const float>(); const int max_pos = r.num();
  auto* cache = r.as<void>(); auto* scale = r.as<float>(); const mla_dtype dtype = r.dtype();
  const int num_pages = r.num();
  auto* err = r.as<int32_t>(); auto stream = r.stream();
  MLA_CALL(mla_cache_append_slots(kv, kv_dtype, n, slots, positions, gain, eps, cos, sin, max_pos, cache, scale,
                                  dtype, num_pages, err, stream))
})

MLA_ENTRY(decode_tree, 23, {
  auto* q = r.as<const void>(); const mla_dtype q_dtype = r.dtype();
  auto* cache = r.as<const void>(); auto* scale = r.as<const float>(); const mla_dtype dtype = r.dtype();
  const int num_pages = r.num();
  auto* table = r.as<const int32_t>(); const int max_pages = r.num(), page = r.num();
  auto* kv_lens = r.as<const int32_t>(); auto* row_start = r.as<const int32_t>();
  const int batch = r.num(), max_rows = r.num(), heads = r.num();
  auto* mask = r.as<const uint64_t>(); const int words = r.num(); const float softmax_scale = r.real();
  auto* ws = r.as<void>(); auto* o = r.as<void>(); const mla_dtype o_dtype = r.dtype(); auto* lse = r.as<float>();
  auto* err = r.as<int32_t>(); auto stream = r.stream();
  MLA_CALL(mla_decode_tree(q, q_dtype, cache, scale, dtype, num_pages, table, max_pages, page, kv_lens, row_start,
                           batch, max_rows, heads, mask, words, softmax_scale, ws, o, o_dtype, lse, err, stream))
})

MLA_ENTRY(cache_commit, 16, {
  auto* kv_lens = r.as<const int32_t>(); auto* row_start = r.as<const int32_t>();
  const int batch = r.num(), max_rows = r.num();
  auto* counts = r.as<const int32_t>(); auto* nodes = r.as<const int32_t>();
  auto* table = r.as<const int32_t>(); const int max_pages = r.num(), page = r.num();
  auto* cache = r.as<void>(); auto* scale = r.as<float>(); const mla_dtype dtype = r.dtype();
  const int num_pages = r.num();
  auto* lens_out = r.as<int32_t>(); auto* err = r.as<int32_t>(); auto stream = r.stream();
  MLA_CALL(mla_cache_commit(kv_lens, row_start, batch, max_rows, counts, nodes, table, max_pages, page, cache, scale,
                            dtype, num_pages, lens_out, err, stream))
})

PyObject* set_stream_getters(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 2) {
    PyErr_SetString(PyExc_TypeError, "set_stream_getters takes two callables");
    return nullptr;
  }
  Py_XSETREF(g_device, Py_NewRef(args[0]));
  Py_XSETREF(g_raw_stream, Py_NewRef(args[1]));
  Py_RETURN_NONE;
}

#define MLA_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(name)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {MLA_METHOD(step_plan), MLA_METHOD(cache_append_slots), MLA_METHOD(decode_tree),
                           MLA_METHOD(cache_commit), MLA_METHOD(set_stream_getters), {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_native", "Fast argument marshalling for libmla.so.", -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() {
  g_data_ptr = PyUnicode_InternFromString("data_ptr");
  g_cuda_stream = PyUnicode_InternFromString("cuda_stream");
  return g_data_ptr && g_cuda_stream ? PyModule_Create(&g_module) : nullptr;
}
