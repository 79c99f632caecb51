// binding.cpp - the Python module `_native`: tensors in, addresses and sizes to
// the C entry points of the 8-bit cache and of the rotary positions.
//
// A call of these costs the host about 4 us in the library (most of it the
// launch); checking seven tensors and calling through ctypes cost another 4 us,
// as long as a small kernel runs.  Here it is 0.5 us.  The module links neither
// libswa.so nor the CUDA runtime: bind() receives the entry points' addresses
// from whoever loaded the library.
//
// Every function checks its tensors (type, shape, device, density) before
// anything is launched and raises ValueError; it returns the entry point's code.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <sstream>
#include <string>

#include "swa.h"

namespace {

decltype(&swa_q8_append) g_append = nullptr;
decltype(&swa_q8_prefill_chunk) g_prefill = nullptr;
decltype(&swa_q8_decode) g_decode = nullptr;
decltype(&swa_rope) g_rope = nullptr;

// What a CacheQ8 or a Rope keeps for this module (a Dims: swa_dims), at the address in its
// `_cache_addr`, `_rope_addr` (`_dims_addr`).
struct CacheRecord {
  swa_q8_cache c;
  int32_t batch, n_kv_heads, window, head_dim, device;
};
struct RopeRecord {
  swa_rope_spec c;
  int32_t device;
};

struct Refused {};   // a Python exception is set

PyObject *g_dims_addr, *g_cache_addr, *g_rope_addr;   // the attributes' names

template <typename T>
const T* record(PyObject* o, PyObject* name) {
  PyObject* a = PyObject_GetAttr(o, name);
  if (a == nullptr) throw Refused();
  void* p = PyLong_AsVoidPtr(a);
  Py_DECREF(a);
  if (p == nullptr) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a record at address 0");
    throw Refused();
  }
  return static_cast<const T*>(p);
}

const at::Tensor& tensor(const char* name, PyObject* o) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s: expected a torch.Tensor, got %s", name, Py_TYPE(o)->tp_name);
    throw Refused();
  }
  return THPVariable_Unpack(o);
}

[[noreturn]] void refuse(const char* name, const at::Tensor& t, const char* what, at::ScalarType type,
                         c10::IntArrayRef shape, int device) {
  std::ostringstream s;
  s << name << ": expected a " << what << " " << toString(type) << " tensor of shape " << shape << " on cuda:" << device
    << ", got " << t.scalar_type() << " " << t.sizes() << " with strides " << t.strides() << " on " << t.device();
  PyErr_SetString(PyExc_ValueError, s.str().c_str());
  throw Refused();
}

bool on(const at::Tensor& t, int device) { return t.is_cuda() && t.get_device() == device; }

// Address of a dense tensor of this shape, type and device.
void* dense(const char* name, PyObject* o, at::ScalarType type, c10::IntArrayRef shape, int device) {
  const at::Tensor& t = tensor(name, o);
  if (t.scalar_type() != type || !on(t, device) || t.sizes() != shape || !t.is_contiguous())
    refuse(name, t, "contiguous", type, shape, device);
  return t.data_ptr();
}

// Address of q or k [B, T, H, d] with dense heads and evenly spaced rows, and the elements from row to row.
void* rows(const char* name, PyObject* o, c10::IntArrayRef shape, int device, int64_t* stride) {
  const at::Tensor& t = tensor(name, o);
  const int64_t B = shape[0], T = shape[1], H = shape[2], d = shape[3];
  if (t.scalar_type() == at::kBFloat16 && on(t, device) && t.sizes() == shape) {
    const auto s = t.strides();
    const int64_t row = T > 1 ? s[1] : B > 1 ? s[0] : H * d;
    if ((d == 1 || s[3] == 1) && (H == 1 || s[2] == d) && (B == 1 || s[0] == T * row)) {
      *stride = row;
      return t.data_ptr();
    }
  }
  refuse(name, t, "evenly spaced", at::kBFloat16, shape, device);
}

std::pair<void*, size_t> scratch(PyObject* o, int device) {
  const at::Tensor& t = tensor("workspace", o);
  if (!on(t, device) || !t.is_contiguous()) refuse("workspace", t, "contiguous", t.scalar_type(), t.sizes(), device);
  return {t.data_ptr(), t.nbytes()};
}

int64_t tokens(const char* name, PyObject* o) {
  const at::Tensor& t = tensor(name, o);
  if (t.dim() != 4) {
    std::ostringstream s;
    s << name << ": expected [B, T, heads, d], got " << t.sizes();
    PyErr_SetString(PyExc_ValueError, s.str().c_str());
    throw Refused();
  }
  if (t.size(1) > INT32_MAX) {
    PyErr_Format(PyExc_ValueError, "%s: too many tokens", name);
    throw Refused();
  }
  return t.size(1);
}

at::ScalarType out_type(const swa_dims* d) { return d->out_dtype == SWA_DTYPE_F32 ? at::kFloat : at::kBFloat16; }

const CacheRecord* cache_for(PyObject* o, const swa_dims* d) {
  const CacheRecord* c = record<CacheRecord>(o, g_cache_addr);
  if (c->batch != d->batch || c->n_kv_heads != d->n_kv_heads || c->window != d->window || c->head_dim != d->head_dim) {
    PyErr_Format(PyExc_ValueError, "cache of [B, Hkv, W, d] = [%d, %d, %d, %d] for dims of [%d, %d, %d, %d]", c->batch,
                 c->n_kv_heads, c->window, c->head_dim, d->batch, d->n_kv_heads, d->window, d->head_dim);
    throw Refused();
  }
  return c;
}

// Calls f(stream) with `device` current, on the stream of this handle or, for None, the device's current one.
template <typename F>
PyObject* launch(int device, PyObject* stream, F f) {
  void* s = nullptr;
  if (stream == Py_None) {
    s = c10::cuda::getCurrentCUDAStream(device).stream();
  } else {
    s = PyLong_AsVoidPtr(stream);
    if (s == nullptr && PyErr_Occurred()) throw Refused();
  }
  std::optional<c10::cuda::CUDAGuard> guard;
  if (c10::cuda::current_device() != device) guard.emplace(device);
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = f(s);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(rc);
}

// Runs a call's body; C++ exceptions become Python ones.
template <typename F>
PyObject* guarded(const char* name, Py_ssize_t n, Py_ssize_t want, F f) {
  if (n != want) return PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, got %zd", name, want, n);
  try {
    return f();
  } catch (const Refused&) {
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// append(dims, cache, k, v, start_pos, n_tokens, stream)
PyObject* py_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("append", n, 7, [&] {
    const swa_dims* d = record<swa_dims>(a[0], g_dims_addr);
    const CacheRecord* c = cache_for(a[1], d);
    const int dev = c->device;
    const int64_t T = tokens("k", a[2]), kv[] = {d->batch, T, d->n_kv_heads, d->head_dim}, b[] = {d->batch};
    void *k = dense("k", a[2], at::kBFloat16, kv, dev), *v = dense("v", a[3], at::kBFloat16, kv, dev);
    auto* s = static_cast<int32_t*>(dense("start_pos", a[4], at::kInt, b, dev));
    auto* m = static_cast<int32_t*>(dense("n_tokens", a[5], at::kInt, b, dev));
    return launch(dev, a[6], [=](void* stream) { return g_append(d, &c->c, k, v, (int32_t)T, s, m, stream); });
  });
}

// prefill(dims, out, q, k, v, cache, start_pos, n_tokens, workspace, stream)
PyObject* py_prefill(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("prefill", n, 10, [&] {
    const swa_dims* d = record<swa_dims>(a[0], g_dims_addr);
    const CacheRecord* c = cache_for(a[5], d);
    const int dev = c->device;
    const int64_t T = tokens("q", a[2]), b[] = {d->batch};
    const int64_t qs[] = {d->batch, T, d->n_q_heads, d->head_dim}, kv[] = {d->batch, T, d->n_kv_heads, d->head_dim};
    void *out = dense("out", a[1], out_type(d), qs, dev), *q = dense("q", a[2], at::kBFloat16, qs, dev);
    void *k = dense("k", a[3], at::kBFloat16, kv, dev), *v = dense("v", a[4], at::kBFloat16, kv, dev);
    auto* s = static_cast<int32_t*>(dense("start_pos", a[6], at::kInt, b, dev));
    auto* m = static_cast<int32_t*>(dense("n_tokens", a[7], at::kInt, b, dev));
    const auto ws = scratch(a[8], dev);
    return launch(dev, a[9], [=](void* stream) {
      return g_prefill(d, out, q, k, v, (int32_t)T, &c->c, s, m, ws.first, ws.second, stream);
    });
  });
}

// decode(dims, out, q, k_new, v_new, cache, pos, workspace, stream)
PyObject* py_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("decode", n, 9, [&] {
    const swa_dims* d = record<swa_dims>(a[0], g_dims_addr);
    const CacheRecord* c = cache_for(a[5], d);
    const int dev = c->device;
    const int64_t qs[] = {d->batch, d->n_q_heads, d->head_dim}, kv[] = {d->batch, d->n_kv_heads, d->head_dim}, b[] = {d->batch};
    void *out = dense("out", a[1], out_type(d), qs, dev), *q = dense("q", a[2], at::kBFloat16, qs, dev);
    void *k = dense("k_new", a[3], at::kBFloat16, kv, dev), *v = dense("v_new", a[4], at::kBFloat16, kv, dev);
    auto* p = static_cast<int32_t*>(dense("pos", a[6], at::kInt, b, dev));
    const auto ws = scratch(a[7], dev);
    return launch(dev, a[8], [=](void* stream) { return g_decode(d, out, q, k, v, &c->c, p, ws.first, ws.second, stream); });
  });
}

// rope(dims, spec, q_out, k_out, q, k, start_pos, n_tokens, transpose, stream); k and k_out, n_tokens may be None
PyObject* py_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("rope", n, 10, [&] {
    const swa_dims* d = record<swa_dims>(a[0], g_dims_addr);
    const RopeRecord* r = record<RopeRecord>(a[1], g_rope_addr);
    const int dev = r->device;
    const int64_t T = tokens("q", a[4]), b[] = {d->batch};
    const int64_t qs[] = {d->batch, T, d->n_q_heads, d->head_dim}, kv[] = {d->batch, T, d->n_kv_heads, d->head_dim};
    int64_t q_stride = 0, k_stride = 0;
    void *q_out = dense("q_out", a[2], at::kBFloat16, qs, dev), *q = rows("q", a[4], qs, dev, &q_stride);
    void *k_out = nullptr, *k = nullptr;
    if ((a[3] == Py_None) != (a[5] == Py_None)) {
      PyErr_SetString(PyExc_ValueError, "k and k_out: both or neither");
      throw Refused();
    }
    if (a[5] != Py_None) {
      k_out = dense("k_out", a[3], at::kBFloat16, kv, dev);
      k = rows("k", a[5], kv, dev, &k_stride);
    }
    auto* s = static_cast<int32_t*>(dense("start_pos", a[6], at::kInt, b, dev));
    auto* m = a[7] == Py_None ? nullptr : static_cast<int32_t*>(dense("n_tokens", a[7], at::kInt, b, dev));
    const int transpose = PyObject_IsTrue(a[8]);
    if (transpose < 0) throw Refused();
    return launch(dev, a[9], [=](void* stream) {
      return g_rope(d, &r->c, q_out, k_out, q, k, q_stride, k_stride, (int32_t)T, s, m, transpose, stream);
    });
  });
}

// bind(append, prefill, decode, rope): addresses of the C entry points
PyObject* py_bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("bind", n, 4, [&]() -> PyObject* {
    void* p[4];
    for (int i = 0; i < 4; ++i) {
      p[i] = PyLong_AsVoidPtr(a[i]);
      if (p[i] == nullptr) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "an entry point at address 0");
        throw Refused();
      }
    }
    g_append = reinterpret_cast<decltype(g_append)>(p[0]);
    g_prefill = reinterpret_cast<decltype(g_prefill)>(p[1]);
    g_decode = reinterpret_cast<decltype(g_decode)>(p[2]);
    g_rope = reinterpret_cast<decltype(g_rope)>(p[3]);
    Py_RETURN_NONE;
  });
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
constexpr PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {method<py_append>("append"), method<py_prefill>("prefill"), method<py_decode>("decode"),
                           method<py_rope>("rope"),     method<py_bind>("bind"),       {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native(void) {
  g_dims_addr = PyUnicode_InternFromString("_dims_addr");
  g_cache_addr = PyUnicode_InternFromString("_cache_addr");
  g_rope_addr = PyUnicode_InternFromString("_rope_addr");
  return g_dims_addr && g_cache_addr && g_rope_addr ? PyModule_Create(&g_module) : nullptr;
}
