// The paged cache's calls from Python without Python's own cost.
//
// A decode step's calls run on the GPU for 3 to 10 microseconds; checking a handful of
// tensors, allocating the outputs and marshalling 17 arguments takes the interpreter 10
// to 25.  Each function here makes the same checks as its method in paged.py, allocates the
// same outputs and calls the same C entry point (whose address the binding hands over,
// so the loaded library is the one that is used).  Anything out of the ordinary - a
// failed check, a tensor subclass - returns None, and the method goes its own way, which
// names what is wrong.
//
// Returns: None (not taken), an int (the failed call's kvs_status), or the result.
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAStream.h>

#include "../../include/kvs.h"

namespace {

decltype(&kvs_paged_plan) g_plan;
decltype(&kvs_paged_append) g_append;
decltype(&kvs_paged_gather) g_gather;
decltype(&kvs_paged_attend) g_attend;
decltype(&kvs_paged_attend_scratch_bytes) g_scratch;

// What a cache's tensors have to look like.
struct Cache {
  kvs_paged* pc;
  int64_t device, hkv, hq, d;
  at::ScalarType dtype;
};

bool read_cache(PyObject* o, Cache* c) {            // (handle, device, Hkv, Hq, D, bf16?)
  if (!PyTuple_CheckExact(o) || PyTuple_GET_SIZE(o) != 6) return false;
  c->pc = static_cast<kvs_paged*>(PyLong_AsVoidPtr(PyTuple_GET_ITEM(o, 0)));
  c->device = PyLong_AsLong(PyTuple_GET_ITEM(o, 1));
  c->hkv = PyLong_AsLong(PyTuple_GET_ITEM(o, 2));
  c->hq = PyLong_AsLong(PyTuple_GET_ITEM(o, 3));
  c->d = PyLong_AsLong(PyTuple_GET_ITEM(o, 4));
  c->dtype = PyTuple_GET_ITEM(o, 5) == Py_True ? at::kBFloat16 : at::kFloat;
  return !PyErr_Occurred();
}

const at::Tensor* tensor(PyObject* o, const Cache& c, at::ScalarType dtype, int64_t dims) {
  if (!THPVariable_CheckExact(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (t.scalar_type() != dtype || t.dim() != dims || !t.is_cuda() || t.get_device() != c.device || !t.is_contiguous())
    return nullptr;
  return &t;
}
bool rows_of(const at::Tensor* t, int64_t n, int64_t h, int64_t d) {
  return t && t->size(0) == n && t->size(1) == h && t->size(2) == d;
}

kvs_stream_t stream_of(const Cache& c) {
  return reinterpret_cast<kvs_stream_t>(c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)c.device).stream());
}
at::Tensor fresh(const Cache& c, at::IntArrayRef shape, at::ScalarType dtype) {
  return at::empty(shape, at::TensorOptions().dtype(dtype).device(at::kCUDA, (c10::DeviceIndex)c.device));
}
int32_t* i32(const at::Tensor* t) { return t ? static_cast<int32_t*>(t->data_ptr()) : nullptr; }

// Everything from torch may throw; nothing passes into the interpreter.
template <typename F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (const std::exception& e) {
    PyErr_Clear();
    Py_RETURN_NONE;                                 // the method meets it again, with torch's own translation
  }
}

#define TAKE(x) if (!(x)) { PyErr_Clear(); Py_RETURN_NONE; }

// append(cache, layer, k, v, slots)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded([&]() -> PyObject* {
    Cache c;
    TAKE(n_args == 5 && read_cache(a[0], &c));
    const long layer = PyLong_AsLong(a[1]);
    TAKE(layer != -1 || !PyErr_Occurred());
    const at::Tensor* slots = tensor(a[4], c, at::kInt, 1);
    TAKE(slots && slots->numel() <= INT32_MAX && layer >= INT32_MIN && layer <= INT32_MAX);
    const int64_t n = slots->numel();
    const at::Tensor *k = tensor(a[2], c, c.dtype, 3), *v = tensor(a[3], c, c.dtype, 3);
    TAKE(rows_of(k, n, c.hkv, c.d) && rows_of(v, n, c.hkv, c.d));
    return PyLong_FromLong(g_append(c.pc, (int32_t)layer, (int32_t)n, i32(slots), k->data_ptr(), v->data_ptr(), stream_of(c)));
  });
}

// gather(cache, layer, slots) -> (k, v)
PyObject* gather(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded([&]() -> PyObject* {
    Cache c;
    TAKE(n_args == 3 && read_cache(a[0], &c));
    const long layer = PyLong_AsLong(a[1]);
    TAKE(layer != -1 || !PyErr_Occurred());
    const at::Tensor* slots = tensor(a[2], c, at::kInt, 1);
    TAKE(slots && slots->numel() <= INT32_MAX && layer >= INT32_MIN && layer <= INT32_MAX);
    const int64_t n = slots->numel();
    at::Tensor k = fresh(c, {n, c.hkv, c.d}, c.dtype), v = fresh(c, {n, c.hkv, c.d}, c.dtype);
    const kvs_status st = g_gather(c.pc, (int32_t)layer, (int32_t)n, i32(slots), k.data_ptr(), v.data_ptr(), stream_of(c));
    if (st != KVS_OK) return PyLong_FromLong(st);
    PyObject* both[2] = {THPVariable_Wrap(std::move(k)), THPVariable_Wrap(std::move(v))};
    PyObject* r = both[0] && both[1] ? PyTuple_New(2) : nullptr;
    for (int i = 0; i < 2; ++i) {
      if (r) PyTuple_SET_ITEM(r, i, both[i]);
      else Py_XDECREF(both[i]);
    }
    return r;
  });
}

// plan(cache, ctx_len, new_len, block_table, free_pages, free_count, free_count_out, row_capacity)
//   -> (row_start, kv_len, slots, positions, denied)
PyObject* plan(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded([&]() -> PyObject* {
    Cache c;
    TAKE(n_args == 8 && read_cache(a[0], &c));
    const at::Tensor *ctx = tensor(a[1], c, at::kInt, 1), *add = tensor(a[2], c, at::kInt, 1),
                     *table = tensor(a[3], c, at::kInt, 2), *pages = tensor(a[4], c, at::kInt, 1),
                     *count = tensor(a[5], c, at::kInt, 1), *out = tensor(a[6], c, at::kInt, 1);
    TAKE(ctx && add && table && pages && count && out);
    const int64_t n = ctx->numel(), stride = table->size(1);
    TAKE(add->numel() == n && table->size(0) == n && count->numel() == 1 && out->numel() == 1);
    const long rows = PyLong_AsLong(a[7]);
    TAKE(rows >= 0 && rows <= (1 << 30) && n <= (1 << 20) && stride <= INT32_MAX && pages->numel() <= INT32_MAX);
    // one allocation, slots and positions on 16-byte boundaries; all that may fail comes before the call, which takes
    // pages: the method must not make it again
    const int64_t pos = rows + (-rows & 3), start = pos + rows, len = start + n + 1, den = len + n;
    at::Tensor buf = fresh(c, {den + 1}, at::kInt);
    PyObject* r = PyTuple_New(5);
    if (!r) return nullptr;
    {
      at::AutoDispatchBelowADInplaceOrView below;   // whole numbers: nothing to differentiate
      const int64_t part[5][2] = {{start, n + 1}, {len, n}, {0, rows}, {pos, rows}, {den, 1}};
      try {
        for (int i = 0; i < 5; ++i) {
          PyObject* view = THPVariable_Wrap(buf.as_strided({part[i][1]}, {1}, part[i][0]));
          if (!view) {
            Py_DECREF(r);
            return nullptr;
          }
          PyTuple_SET_ITEM(r, i, view);
        }
      } catch (...) {
        Py_DECREF(r);
        throw;
      }
    }
    int32_t* p = i32(&buf);
    const kvs_status st = g_plan(c.pc, (int32_t)n, i32(ctx), i32(add), i32(table), (int32_t)stride, i32(pages),
                                 (int32_t)pages->numel(), i32(count), i32(out), p + start, p + len, p, p + pos,
                                 (int32_t)rows, p + den, stream_of(c));
    if (st == KVS_OK) return r;
    Py_DECREF(r);
    return PyLong_FromLong(st);
  });
}

// attend(cache, layer, q, block_table, kv_len, q_start or None, max_q_len, window, block_mass or None) -> out
PyObject* attend(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded([&]() -> PyObject* {
    Cache c;
    TAKE(n_args == 9 && read_cache(a[0], &c));
    const long layer = PyLong_AsLong(a[1]), most = PyLong_AsLong(a[6]), window = PyLong_AsLong(a[7]);
    TAKE(!PyErr_Occurred() && layer >= 0 && layer <= INT32_MAX && most >= 1 && most <= INT32_MAX && window >= 0 && window <= INT32_MAX);
    const at::Tensor *q = tensor(a[2], c, c.dtype, 3), *table = tensor(a[3], c, at::kInt, 2), *len = tensor(a[4], c, at::kInt, 1);
    TAKE(q && table && len);
    const int64_t n = len->numel(), stride = table->size(1), rows = q->size(0);
    TAKE(table->size(0) == n && rows_of(q, rows, c.hq, c.d) && n <= (1 << 20) && rows <= (1 << 28) && stride <= (1 << 22));
    const at::Tensor *start = nullptr, *mass = nullptr;
    if (a[5] != Py_None) {
      start = tensor(a[5], c, at::kInt, 1);
      TAKE(start && start->numel() == n + 1);
    }
    if (a[8] != Py_None) {
      mass = tensor(a[8], c, at::kFloat, 2);
      TAKE(mass && mass->size(0) == n && mass->size(1) == stride);
    }
    const size_t need = g_scratch(c.pc, (int32_t)n, (int32_t)stride, (int32_t)rows, (int32_t)most, mass != nullptr);
    TAKE(need > 0);
    at::Tensor out = fresh(c, q->sizes(), c.dtype), scratch = fresh(c, {(int64_t)need}, at::kByte);
    const kvs_status st = g_attend(c.pc, (int32_t)layer, (int32_t)n, i32(table), (int32_t)stride, i32(len), i32(start),
                                   (int32_t)rows, (int32_t)most, (int32_t)window, q->data_ptr(), out.data_ptr(),
                                   mass ? static_cast<float*>(mass->data_ptr()) : nullptr, scratch.data_ptr(), need, stream_of(c));
    if (st != KVS_OK) return PyLong_FromLong(st);
    return THPVariable_Wrap(std::move(out));
  });
}

// bind(addresses of kvs_paged_plan, _append, _gather, _attend, _attend_scratch_bytes)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 5) {
    PyErr_SetString(PyExc_TypeError, "bind takes five addresses");
    return nullptr;
  }
  void* p[5];
  for (int i = 0; i < 5; ++i)
    if (!(p[i] = PyLong_AsVoidPtr(a[i]))) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a null address");
      return nullptr;
    }
  g_plan = reinterpret_cast<decltype(g_plan)>(p[0]);
  g_append = reinterpret_cast<decltype(g_append)>(p[1]);
  g_gather = reinterpret_cast<decltype(g_gather)>(p[2]);
  g_attend = reinterpret_cast<decltype(g_attend)>(p[3]);
  g_scratch = reinterpret_cast<decltype(g_scratch)>(p[4]);
  Py_RETURN_NONE;
}

#define FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(bind), FAST(plan), FAST(append), FAST(gather), FAST(attend), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_paged_call", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged_call() { return PyModule_Create(&module_def); }
