// Python calls of the operators around the cache (rotary, reading back, group
// index and selection, decode over listed groups): argument checks on the
// tensors themselves, then the C ABI.  These are called once per layer and
// step, and through ctypes the checks and the marshalling of a call took 4 to
// 7 us, as long as the kernel; here they take well under 1 us.
//
// Every function returns the oscar_status of the C call (0: done) and raises
// TypeError or ValueError for what the C ABI cannot see behind a pointer:
// dtype, shape, contiguity, the cache's KV heads (those of the handle, always;
// an argument hkv >= 0 is the caller's own expectation and checked beside them).
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <algorithm>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <stdexcept>
#include <string>
#include <vector>

#include <ATen/core/CachingHostAllocator.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/oscar.h"

namespace {

struct Refused : std::runtime_error {
  PyObject* type;
  Refused(PyObject* t, const std::string& m) : std::runtime_error(m), type(t) {}
};

[[noreturn]] void refuse(PyObject* type, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  throw Refused(type, buf);
}

// A Python error is already set.
struct Raised {};

constexpr int64_t kDim = 128;

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a torch.Tensor", name);
  return THPVariable_Unpack(o);
}

std::string text(at::IntArrayRef shape) {
  std::string s = "(";
  for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + (shape[i] < 0 ? "any" : std::to_string(shape[i]));
  return s + ")";
}

const char* type_name(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "torch.bfloat16";
    case at::kFloat: return "torch.float32";
    case at::kInt: return "torch.int32";
    case at::kByte: return "torch.uint8";
    default: return c10::toString(t);
  }
}

void* dense(const at::Tensor& t, at::ScalarType type, at::IntArrayRef shape, const char* name) {
  if (t.scalar_type() != type) refuse(PyExc_ValueError, "%s must be %s, got %s", name, type_name(type), type_name(t.scalar_type()));
  if (!t.is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous", name);
  bool ok = t.dim() == (int64_t)shape.size();
  for (size_t i = 0; ok && i < shape.size(); ++i)
    ok = shape[i] < 0 || (i == 0 ? t.size(0) >= shape[0] : t.size((int64_t)i) == shape[i]);
  if (!ok)
    refuse(PyExc_ValueError, "%s has shape %s, expected %s (leading dimension at least)", name, text(t.sizes()).c_str(),
           text(shape).c_str());
  return t.data_ptr();
}

int32_t float_type(const at::Tensor& t, const char* name) {
  if (t.scalar_type() == at::kBFloat16) return OSCAR_BF16;
  if (t.scalar_type() == at::kFloat) return OSCAR_F32;
  refuse(PyExc_ValueError, "%s must be torch.bfloat16 or torch.float32, got %s", name, type_name(t.scalar_type()));
}

// KV heads of the cache; -1 for a NULL handle, which the C call refuses.
int64_t cache_heads(const oscar_cache* cache) {
  oscar_cache_config cfg;
  return cache != nullptr && oscar_cache_get_config(cache, &cfg) == OSCAR_OK ? cfg.num_kv_heads : -1;
}

// The KV-head dimension of a buffer: the kernels index it with the cache's
// number, so a smaller one would be read or written past its end.
void heads(const at::Tensor& t, int64_t dim, int64_t hkv, const oscar_cache* cache, const char* name) {
  for (const int64_t want : {hkv, cache_heads(cache)})
    if (want >= 0 && t.dim() > dim && t.size(dim) != want)
      refuse(PyExc_ValueError, "%s has %lld KV heads, the cache %lld", name, (long long)t.size(dim), (long long)want);
}

int64_t integer(PyObject* o) {
  const int64_t v = PyLong_Check(o) ? PyLong_AsLongLong(o) : [&] {
    PyObject* i = PyNumber_Index(o);
    if (!i) throw Raised();
    const int64_t r = PyLong_AsLongLong(i);
    Py_DECREF(i);
    return r;
  }();
  if (v == -1 && PyErr_Occurred()) throw Raised();
  return v;
}

int32_t integer32(PyObject* o, const char* name) {
  const int64_t v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) refuse(PyExc_ValueError, "%s out of range: %lld", name, (long long)v);
  return (int32_t)v;
}

std::vector<int32_t> integers(PyObject* o, const char* name) {
  PyObject* s = PySequence_Fast(o, "expected a sequence of integers");
  if (!s) throw Raised();
  const Py_ssize_t n = PySequence_Fast_GET_SIZE(s);
  std::vector<int32_t> r((size_t)n);
  try {
    for (Py_ssize_t i = 0; i < n; ++i) r[(size_t)i] = integer32(PySequence_Fast_GET_ITEM(s, i), name);
  } catch (...) {
    Py_DECREF(s);
    throw;
  }
  Py_DECREF(s);
  return r;
}

template <typename T = void>
T* address(PyObject* o) {   // a handle (c_void_p) or an integer address
  if (o == Py_None) return nullptr;
  if (PyLong_Check(o)) return reinterpret_cast<T*>((uintptr_t)PyLong_AsUnsignedLongLong(o));
  PyObject* v = PyObject_GetAttrString(o, "value");
  if (!v) throw Raised();
  T* p = v == Py_None ? nullptr : reinterpret_cast<T*>((uintptr_t)PyLong_AsUnsignedLongLong(v));
  Py_DECREF(v);
  return p;
}

// None: the current stream of the current device; a torch stream; a raw handle.
void* stream_of(PyObject* o) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream().stream();
  if (PyLong_Check(o)) return reinterpret_cast<void*>((uintptr_t)PyLong_AsUnsignedLongLong(o));
  PyObject* v = PyObject_GetAttrString(o, "cuda_stream");
  if (!v) throw Raised();
  void* p = reinterpret_cast<void*>((uintptr_t)PyLong_AsUnsignedLongLong(v));
  Py_DECREF(v);
  return p;
}

// The C call, without the interpreter lock (as ctypes makes its calls).
template <typename F>
oscar_status unlocked(F f) {
  if (PyErr_Occurred()) throw Raised();   // an address that does not convert
  PyThreadState* state = PyEval_SaveThread();
  const oscar_status s = f();
  PyEval_RestoreThread(state);
  return s;
}

template <typename F>
PyObject* call(Py_ssize_t got, Py_ssize_t want, F f) {
  if (got != want) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, got);
    return nullptr;
  }
  try {
    return PyLong_FromLong((long)f());
  } catch (const Raised&) {
    return nullptr;
  } catch (const Refused& e) {
    PyErr_SetString(e.type, e.what());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// x [n, heads, 128] with contiguous channels, and where its rows go (None: in place)
bool rotary_rows(PyObject* xo, PyObject* oo, int64_t n, at::ScalarType type, const char* name, oscar_rotary_rows* r) {
  if (xo == Py_None) return false;
  const std::string out_name = std::string(name) + "_out";
  const at::Tensor& x = tensor(xo, name);
  if (x.dim() != 3 || x.size(0) != n || x.size(2) != kDim)
    refuse(PyExc_ValueError, "%s has shape %s, expected (%lld, heads, 128)", name, text(x.sizes()).c_str(), (long long)n);
  const at::Tensor& y = oo == Py_None ? x : tensor(oo, out_name.c_str());
  if (y.sizes() != x.sizes())
    refuse(PyExc_ValueError, "%s has shape %s, expected %s", out_name.c_str(), text(y.sizes()).c_str(),
           text(x.sizes()).c_str());
  for (const at::Tensor* t : {&x, &y}) {
    const char* what = t == &x ? name : out_name.c_str();
    if (t->scalar_type() != type)
      refuse(PyExc_ValueError, "%s must be %s, got %s", what, type_name(type), type_name(t->scalar_type()));
    if (t->stride(2) != 1) refuse(PyExc_ValueError, "%s must have contiguous channels", what);
  }
  if (x.size(1) > INT32_MAX) refuse(PyExc_ValueError, "%s has too many heads", name);
  *r = oscar_rotary_rows{x.data_ptr(), y.data_ptr(), x.stride(0), x.stride(1), y.stride(0), y.stride(1),
                         (int32_t)x.size(1)};
  return true;
}

// table, positions, q, k, q_out, k_out, transpose, stream
PyObject* rotary(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 8, [&] {
    const at::Tensor& q = tensor(a[2], "q");
    const int32_t type = float_type(q, "q");
    if (q.dim() != 3) refuse(PyExc_ValueError, "q has shape %s, expected (tokens, heads, 128)", text(q.sizes()).c_str());
    const int64_t tokens = q.size(0);
    const void* pos = dense(tensor(a[1], "positions"), at::kInt, {tokens}, "positions");
    oscar_rotary_rows rq, rk;
    rotary_rows(a[2], a[4], tokens, q.scalar_type(), "q", &rq);
    const bool has_k = rotary_rows(a[3], a[5], tokens, q.scalar_type(), "k", &rk);
    const int transpose = PyObject_IsTrue(a[6]);
    if (transpose < 0) throw Raised();
    const auto* table = address<const oscar_rotary_table>(a[0]);
    void* stream = stream_of(a[7]);
    return unlocked([&] {
      return oscar_rotary(table, tokens, static_cast<const int32_t*>(pos), type, &rq, has_k ? &rk : nullptr, transpose,
                          stream);
    });
  });
}

// handle, hkv, seq_ids, start, end, k_out, v_out, stream
PyObject* read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 8, [&] {
    auto* cache = address<oscar_cache>(a[0]);
    const int64_t hkv = integer(a[1]);
    const std::vector<int32_t> ids = integers(a[2], "seq_ids"), start = integers(a[3], "start"),
                               end = integers(a[4], "end");
    if (start.size() != ids.size() || end.size() != ids.size())
      refuse(PyExc_ValueError, "seq_ids, start and end must have the same length");
    int64_t rows = 0;
    for (size_t i = 0; i < ids.size(); ++i) rows += std::max<int64_t>(0, (int64_t)end[i] - start[i]);
    void* out[2] = {nullptr, nullptr};
    int32_t type = OSCAR_BF16;
    const at::Tensor* first = nullptr;
    for (int i = 0; i < 2; ++i) {
      const char* name = i ? "v_out" : "k_out";
      if (a[5 + i] == Py_None) continue;
      const at::Tensor& t = tensor(a[5 + i], name);
      if (!first) {
        first = &t;
        type = float_type(t, name);
      }
      heads(t, 1, hkv, cache, name);
      out[i] = dense(t, first->scalar_type(), {rows, first->dim() == 3 ? first->size(1) : (int64_t)1, kDim}, name);
    }
    void* stream = stream_of(a[7]);
    return unlocked([&] {
      return oscar_cache_read(cache, (int32_t)ids.size(), ids.data(), start.data(), end.data(), type, out[0], out[1],
                              stream);
    });
  });
}

// handle, seq_ids, rebuild, stream
PyObject* index_update(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 4, [&] {
    const std::vector<int32_t> ids = integers(a[1], "seq_ids");
    const int rebuild = PyObject_IsTrue(a[2]);
    if (rebuild < 0) throw Raised();
    auto* cache = address<oscar_cache>(a[0]);
    void* stream = stream_of(a[3]);
    return unlocked([&] { return oscar_index_update(cache, (int32_t)ids.size(), ids.data(), rebuild, stream); });
  });
}

// A group list [n, kv heads, entries]
int32_t* group_list(PyObject* o, int64_t n, int64_t hkv, const oscar_cache* cache, int32_t* entries) {
  const at::Tensor& t = tensor(o, "groups");
  heads(t, 1, hkv, cache, "groups");
  void* p = dense(t, at::kInt, {n, -1, -1}, "groups");
  if (t.size(2) > INT32_MAX) refuse(PyExc_ValueError, "groups has too many entries");
  *entries = (int32_t)t.size(2);
  return static_cast<int32_t*>(p);
}

// handle, hkv, seq_ids, q, num_q_heads, groups, keep_first, keep_last, stream
PyObject* select_groups(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 9, [&] {
    const std::vector<int32_t> ids = integers(a[2], "seq_ids");
    const int32_t hq = integer32(a[4], "num_q_heads");
    const void* q = dense(tensor(a[3], "q"), at::kBFloat16, {(int64_t)ids.size(), hq, kDim}, "q");
    int32_t entries = 0;
    auto* cache = address<oscar_cache>(a[0]);
    int32_t* groups = group_list(a[5], (int64_t)ids.size(), integer(a[1]), cache, &entries);
    const int32_t first = integer32(a[6], "keep_first"), last = integer32(a[7], "keep_last");
    void* stream = stream_of(a[8]);
    return unlocked([&] {
      return oscar_select_groups(cache, (int32_t)ids.size(), ids.data(), q, hq, entries, first, last, groups, stream);
    });
  });
}

// handle, hkv, seq_ids, q, num_q_heads, softmax_scale, groups, out, workspace, lse, stream
PyObject* sparse_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 11, [&] {
    const std::vector<int32_t> ids = integers(a[2], "seq_ids");
    const int64_t b = (int64_t)ids.size();
    const int32_t hq = integer32(a[4], "num_q_heads");
    const double scale = PyFloat_AsDouble(a[5]);
    if (scale == -1.0 && PyErr_Occurred()) throw Raised();
    const void* q = dense(tensor(a[3], "q"), at::kBFloat16, {b, hq, kDim}, "q");
    int32_t entries = 0;
    auto* cache = address<oscar_cache>(a[0]);
    const int32_t* groups = group_list(a[6], b, integer(a[1]), cache, &entries);
    const at::Tensor& o = tensor(a[7], "out");
    const int32_t type = float_type(o, "out");
    void* out = dense(o, o.scalar_type(), {b, hq, kDim}, "out");
    const at::Tensor& ws = tensor(a[8], "workspace");
    void* w = dense(ws, at::kByte, ws.sizes(), "workspace");
    float* lse = a[9] == Py_None ? nullptr : static_cast<float*>(dense(tensor(a[9], "lse"), at::kFloat, {b, hq}, "lse"));
    const size_t w_bytes = (size_t)ws.numel();
    void* stream = stream_of(a[10]);
    return unlocked([&] {
      return oscar_sparse_decode_attention(cache, (int32_t)b, ids.data(), q, hq, (float)scale, groups, entries, type, out,
                                           lse, w, w_bytes, stream);
    });
  });
}

// tensor, stream id, device index, device type (as torch streams name
// themselves): the stream uses a page-locked tensor until what is enqueued on
// it now has run.  Its memory, if it came from torch, is not handed out again
// before (record_stream, which torch offers for device tensors only).
PyObject* host_in_use(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 4, [&] {
    const at::Tensor& t = tensor(a[0], "tensor");
    const c10::Stream stream = c10::Stream::unpack3(integer(a[1]), (c10::DeviceIndex)integer(a[2]),
                                                    (c10::DeviceType)integer(a[3]));
    at::getHostAllocator(at::kCUDA)->record_event(t.data_ptr(), t.storage().data_ptr().get_context(), stream);
    return OSCAR_OK;
  });
}

#define OSCAR_FAST(f) {#f, (PyCFunction)(void (*)(void))f, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {OSCAR_FAST(rotary),        OSCAR_FAST(read),         OSCAR_FAST(index_update),
                         OSCAR_FAST(select_groups), OSCAR_FAST(sparse_decode), OSCAR_FAST(host_in_use),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", "Calls of liboscar.so on torch tensors.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls(void) { return PyModule_Create(&module); }
