// The INT4 cache calls from Python: argument checks and marshalling in native code.
//
// On the device these calls take 2 to 6 us for a decode step's few rows.  Through ctypes one costs the host about
// 10 us (checking the attributes of nine tensors one by one in Python 5 us, converting 16 to 24 arguments 1.3 us, the
// launch 2.9 us); through this module about 3 us.  Each function takes tensors, reads their types, shapes, strides and
// addresses here, and calls the C entry it is bound to.  It returns the entry's status, or kWrong if an argument is
// not as it has to be (nothing is called; the Python side then finds the words), or kWorkspace if decode is to get a
// workspace first.  No exception leaves a function.

#include <Python.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "paged_attn.h"

namespace {

constexpr int kWrong = 1, kWorkspace = 2;

struct {
  decltype(&pa_write_kv_int4) write;
  decltype(&pa_rope_write_kv_int4) rope;
  decltype(&pa_copy_blocks_int4) copy;
  decltype(&pa_load_blocks_int4) load;
  decltype(&pa_decode_int4) decode;
} entry;

// A tensor argument; null for anything else.
const at::Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

// One call's checks: all tensors on device dev, contiguous.
struct Check {
  at::ScalarType dt = at::kFloat;  // the 16-bit type
  int dev = -1;
  bool ok = true;
  int64_t NB = 0, Hkv = 0, bs = 0, D = 0;

  void need(bool b) { ok = ok && b; }
  // The first tensor: sets type and device.
  const at::Tensor* lead(PyObject* o, int dim) {
    const at::Tensor* t = tensor(o);
    need(t && t->is_cuda() && t->dim() == dim && t->is_contiguous());
    if (!ok) return nullptr;
    dt = t->scalar_type();
    dev = t->get_device();
    return t;
  }
  void sixteen_bit() { need(dt == at::kBFloat16 || dt == at::kHalf); }
  void* like(PyObject* o, at::ScalarType type, at::IntArrayRef sizes, bool optional = false) {
    if (!ok || (optional && o == Py_None)) return nullptr;
    const at::Tensor* t = tensor(o);
    need(t && t->is_cuda() && t->get_device() == dev && t->scalar_type() == type && t->sizes() == sizes &&
         t->is_contiguous());
    return ok ? t->data_ptr() : nullptr;
  }
  // The four tensors of a cache.
  void cache(PyObject* const* o, void** at) {
    if (!ok) return;
    const at::Tensor* c = tensor(o[0]);
    need(c && c->dim() == 4 && c->size(3) % 32 == 0);
    if (!ok) return;
    NB = c->size(0), Hkv = c->size(1), bs = c->size(2), D = c->size(3) * 2;
    const int64_t params[5] = {NB, Hkv, bs, D / 64, 2};
    at[0] = like(o[0], at::kByte, c->sizes());
    at[1] = like(o[1], at::kByte, c->sizes());
    at[2] = like(o[2], dt, at::IntArrayRef(params, 5));
    at[3] = like(o[3], dt, at::IntArrayRef(params, 5));
    need(NB < INT32_MAX && Hkv < INT32_MAX && bs < INT32_MAX && D < INT32_MAX);
  }
  int number(PyObject* o) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) PyErr_Clear(), ok = false;
    need(v >= INT32_MIN && v <= INT32_MAX);
    return (int)v;
  }
  int code() const { return dt == at::kBFloat16 ? PA_BF16 : PA_F16; }
  // dev is the current device; the stream given by handle, or the current one.
  void* stream(PyObject* o) {
    if (!ok) return nullptr;
    need(c10::cuda::current_device() == dev);
    if (!ok) return nullptr;
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream(dev).stream();
    void* s = PyLong_AsVoidPtr(o);
    if (PyErr_Occurred()) PyErr_Clear(), ok = false;
    return s;
  }
};

int small(int64_t n) { return n > INT32_MAX ? -1 : (int)n; }  // a size the entries refuse in place of one they cannot take

PyObject* answer(int v) { return PyLong_FromLong(v); }

template <int N, typename F>
PyObject* guarded(Py_ssize_t n, F&& f) {
  if (n != N) return answer(kWrong);
  try {
    return answer(f());
  } catch (...) {  // a tensor of an unusual layout: the Python side finds the words
    return answer(kWrong);
  }
}

// k, v, slots, cache x 4, k_out, v_out, stream
PyObject* write_kv_int4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded<10>(n, [&] {
    Check c;
    void* m[4];
    const at::Tensor* k = c.lead(a[0], 3);
    c.sixteen_bit();
    c.cache(a + 3, m);
    if (!c.ok || k->size(1) != c.Hkv || k->size(2) != c.D) return kWrong;
    const auto rows = k->sizes();
    void* v = c.like(a[1], c.dt, rows);
    void* slots = c.like(a[2], at::kLong, rows.slice(0, 1));
    void *ko = c.like(a[7], c.dt, rows, true), *vo = c.like(a[8], c.dt, rows, true), *st = c.stream(a[9]);
    if (!c.ok) return kWrong;
    return entry.write(k->data_ptr(), v, (const int64_t*)slots, small(rows[0]), m[0], m[1], m[2], m[3], ko, vo,
                       (int)c.NB, (int)c.bs, (int)c.Hkv, (int)c.D, c.code(), st);
  });
}

// q, k, v, positions, cos, sin, slots, cache x 4, q_out, k_out, v_out, stream
PyObject* rope_write_kv_int4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded<15>(n, [&] {
    Check c;
    void* m[4];
    const at::Tensor* q = c.lead(a[0], 3);
    c.sixteen_bit();
    c.cache(a + 7, m);
    const at::Tensor* cos = tensor(a[4]);
    if (!c.ok || !cos || cos->dim() != 2 || q->size(2) != c.D || cos->size(1) * 2 != c.D) return kWrong;
    const int64_t T = q->size(0), rows[3] = {T, c.Hkv, c.D};
    void *k = c.like(a[1], c.dt, at::IntArrayRef(rows, 3)), *v = c.like(a[2], c.dt, at::IntArrayRef(rows, 3));
    void *pos = c.like(a[3], at::kLong, at::IntArrayRef(rows, 1)), *slots = c.like(a[6], at::kLong, at::IntArrayRef(rows, 1));
    void *ct = c.like(a[4], at::kFloat, cos->sizes()), *si = c.like(a[5], at::kFloat, cos->sizes());
    void* qo = c.like(a[11], c.dt, q->sizes());
    void *ko = c.like(a[12], c.dt, at::IntArrayRef(rows, 3), true), *vo = c.like(a[13], c.dt, at::IntArrayRef(rows, 3), true);
    void* st = c.stream(a[14]);
    if (!c.ok) return kWrong;
    return entry.rope(q->data_ptr(), qo, k, v, (const int64_t*)pos, (const float*)ct, (const float*)si,
                      small(cos->size(0)), (const int64_t*)slots, small(T), small(q->size(1)), m[0], m[1], m[2], m[3], ko,
                      vo, (int)c.NB, (int)c.bs, (int)c.Hkv, (int)c.D, c.code(), st);
  });
}

// pairs, cache x 4, stream
PyObject* copy_blocks_int4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded<6>(n, [&] {
    Check c;
    void* m[4];
    const at::Tensor *pairs = c.lead(a[0], 2), *params = tensor(a[3]);
    if (!c.ok || !params || c.dt != at::kInt || pairs->size(1) != 2) return kWrong;
    c.dt = params->scalar_type();
    c.sixteen_bit();
    c.cache(a + 1, m);
    void* st = c.stream(a[5]);
    if (!c.ok) return kWrong;
    return entry.copy((const int32_t*)pairs->data_ptr(), small(pairs->size(0)), m[0], m[1], m[2], m[3], (int)c.NB,
                      (int)c.bs, (int)c.Hkv, (int)c.D, st);
  });
}

// pairs, cache x 4, k_cache, v_cache, stream
PyObject* load_blocks_int4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded<8>(n, [&] {
    Check c;
    void* m[4];
    const at::Tensor *pairs = c.lead(a[0], 2), *k16 = tensor(a[5]);
    if (!c.ok || !k16 || k16->dim() != 4 || c.dt != at::kInt || pairs->size(1) != 2) return kWrong;
    c.dt = k16->scalar_type();
    c.sixteen_bit();
    c.cache(a + 1, m);
    const int64_t blocks[4] = {k16->size(0), c.bs, c.Hkv, c.D};
    void *k = c.like(a[5], c.dt, at::IntArrayRef(blocks, 4)), *v = c.like(a[6], c.dt, at::IntArrayRef(blocks, 4));
    void* st = c.stream(a[7]);
    if (!c.ok) return kWrong;
    return entry.load((const int32_t*)pairs->data_ptr(), small(pairs->size(0)), m[0], m[1], m[2], m[3], (int)c.NB, k, v,
                      small(blocks[0]), (int)c.bs, (int)c.Hkv, (int)c.D, c.code(), st);
  });
}

// q, cache x 4, block_tables, context_lens, max_context_len, scale, out, lse, workspace, num_partitions, stream
PyObject* decode_int4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded<14>(n, [&] {
    Check c;
    void* m[4];
    const at::Tensor* q = c.lead(a[0], 3);
    c.sixteen_bit();
    c.cache(a + 1, m);
    const at::Tensor* bt = tensor(a[5]);
    if (!c.ok || !bt || bt->dim() != 2 || bt->size(0) != q->size(0) || q->size(2) != c.D) return kWrong;
    void *tables = c.like(a[5], at::kInt, bt->sizes()), *lens = c.like(a[6], at::kInt, q->sizes().slice(0, 1));
    const int max_len = c.number(a[7]), parts = c.number(a[12]);
    const double scale = PyFloat_AsDouble(a[8]);
    if (PyErr_Occurred()) PyErr_Clear(), c.ok = false;
    void *out = c.like(a[9], c.dt, q->sizes()), *lse = c.like(a[10], at::kFloat, q->sizes().slice(0, 2), true);
    void* st = c.stream(a[13]);
    if (!c.ok) return kWrong;
    if (a[11] == Py_None) return kWorkspace;
    const at::Tensor* ws = tensor(a[11]);
    if (!ws || !ws->is_cuda() || ws->get_device() != c.dev || !ws->is_contiguous()) return kWrong;
    return entry.decode(q->data_ptr(), m[0], m[1], m[2], m[3], (const int32_t*)tables, small(bt->size(1)),
                        (const int32_t*)lens, small(q->size(0)), small(q->size(1)), (int)c.Hkv, (int)c.D, (int)c.bs,
                        (int)c.NB, max_len, (float)scale, c.code(), ws->data_ptr(), ws->nbytes(), parts, out, (float*)lse,
                        st);
  });
}

// The addresses of the five C entries, in the order above.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  void* p[5];
  if (n != 5) {
    PyErr_SetString(PyExc_TypeError, "bind takes five addresses");
    return nullptr;
  }
  for (int i = 0; i < 5; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  entry = {(decltype(entry.write))p[0], (decltype(entry.rope))p[1], (decltype(entry.copy))p[2],
           (decltype(entry.load))p[3], (decltype(entry.decode))p[4]};
  Py_RETURN_NONE;
}

#define PA_METHOD(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {PA_METHOD(write_kv_int4), PA_METHOD(rope_write_kv_int4), PA_METHOD(copy_blocks_int4),
                         PA_METHOD(load_blocks_int4), PA_METHOD(decode_int4), PA_METHOD(bind),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls(void) { return PyModule_Create(&module); }
