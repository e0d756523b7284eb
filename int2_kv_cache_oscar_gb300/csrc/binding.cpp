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

// x [>= n, heads (-1: any), 128] in bf16 with contiguous channels
oscar_rows rows(const at::Tensor& x, int64_t n, int64_t heads, const char* name) {
  if (x.scalar_type() != at::kBFloat16)
    refuse(PyExc_ValueError, "%s must be torch.bfloat16, got %s", name, type_name(x.scalar_type()));
  if (x.dim() != 3 || x.size(0) < n || (heads >= 0 && x.size(1) != heads) || x.size(2) != kDim)
    refuse(PyExc_ValueError, "%s has shape %s, expected %s (leading dimension at least)", name, text(x.sizes()).c_str(),
           text({n, heads, kDim}).c_str());
  if (x.stride(2) != 1) refuse(PyExc_ValueError, "%s must have contiguous channels", name);
  if (x.size(1) > INT32_MAX) refuse(PyExc_ValueError, "%s has too many heads", name);
  return oscar_rows{x.data_ptr(), x.stride(0), x.stride(1)};
}

double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised();
  return v;
}

// A score rule from cap and slopes (None or float32 [hq])
oscar_score_rule score_rule(PyObject* cap, PyObject* slopes, int64_t hq) {
  oscar_score_rule r{(float)real(cap), 0, nullptr};
  if (slopes != Py_None) {
    const at::Tensor& t = tensor(slopes, "slopes");
    if (t.dim() != 1 || t.size(0) != hq)
      refuse(PyExc_ValueError, "slopes has shape %s, expected (%lld)", text(t.sizes()).c_str(), (long long)hq);
    r.slopes = static_cast<const float*>(dense(t, at::kFloat, {hq}, "slopes"));
  }
  return r;
}

// cu_seqlens, prefix, q, k, v, softmax_scale, cap, slopes, prior_out, prior_lse, out, lse, stream
PyObject* chunk(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 13, [&] {
    const std::vector<int32_t> cu = integers(a[0], "cu_seqlens");
    if (cu.empty()) refuse(PyExc_ValueError, "cu_seqlens must have an entry more than there are documents");
    const size_t docs = cu.size() - 1;
    std::vector<int32_t> prefix;
    if (a[1] != Py_None) {
      prefix = integers(a[1], "prefix");
      if (prefix.size() != docs) refuse(PyExc_ValueError, "prefix must have an entry for each document");
    }
    const int64_t tokens = *std::max_element(cu.begin(), cu.end());
    const at::Tensor &q = tensor(a[2], "q"), &k = tensor(a[3], "k"), &v = tensor(a[4], "v");
    const oscar_rows rq = rows(q, tokens, -1, "q"), rk = rows(k, tokens, -1, "k"), rv = rows(v, tokens, k.size(1), "v");
    const int64_t hq = q.size(1), hkv = k.size(1);
    const double scale = real(a[5]);
    const oscar_score_rule rule = score_rule(a[6], a[7], hq);
    auto row_buffer = [&](PyObject* o, const char* name) -> void* {
      return o == Py_None ? nullptr : dense(tensor(o, name), at::kBFloat16, {tokens, hq, kDim}, name);
    };
    auto lse_buffer = [&](PyObject* o, const char* name) -> float* {
      return o == Py_None ? nullptr : static_cast<float*>(dense(tensor(o, name), at::kFloat, {tokens, hq}, name));
    };
    const void* prior_out = row_buffer(a[8], "prior_out");
    const float* prior_lse = lse_buffer(a[9], "prior_lse");
    if (a[10] == Py_None) refuse(PyExc_TypeError, "out must be a torch.Tensor");
    void* out = row_buffer(a[10], "out");
    float* lse = lse_buffer(a[11], "lse");
    void* stream = stream_of(a[12]);
    return unlocked([&] {
      return oscar_chunk_attention((int32_t)docs, cu.data(), prefix.empty() ? nullptr : prefix.data(), &rq, &rk, &rv,
                                   (int32_t)hq, (int32_t)hkv, (float)scale, &rule, prior_out, prior_lse, out, lse, stream);
    });
  });
}

// handle, seq_ids, q, num_q_heads, softmax_scale, cap, slopes, out, workspace, stream
PyObject* scored_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 10, [&] {
    const std::vector<int32_t> ids = integers(a[1], "seq_ids");
    const int64_t b = (int64_t)ids.size();
    const int32_t hq = integer32(a[3], "num_q_heads");
    const void* q = dense(tensor(a[2], "q"), at::kBFloat16, {b, hq, kDim}, "q");
    const double scale = real(a[4]);
    const oscar_score_rule rule = score_rule(a[5], a[6], hq);
    const at::Tensor& o = tensor(a[7], "out");
    const int32_t type = float_type(o, "out");
    void* out = dense(o, o.scalar_type(), {b, hq, kDim}, "out");
    const at::Tensor& ws = tensor(a[8], "workspace");
    void* w = dense(ws, at::kByte, ws.sizes(), "workspace");
    const size_t w_bytes = (size_t)ws.numel();
    auto* cache = address<oscar_cache>(a[0]);
    void* stream = stream_of(a[9]);
    return unlocked([&] {
      return oscar_scored_decode_attention(cache, (int32_t)b, ids.data(), q, hq, (float)scale, &rule, type, out, w,
                                           w_bytes, stream);
    });
  });
}

// handle, seq, q, num_q_heads, softmax_scale, cap, slopes, out, lse, workspace, stream
PyObject* scored_prefill(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 11, [&] {
    const int32_t seq = integer32(a[1], "seq"), hq = integer32(a[3], "num_q_heads");
    const at::Tensor& qt = tensor(a[2], "q");
    const void* q = dense(qt, at::kBFloat16, {-1, hq, kDim}, "q");
    const int32_t rows = (int32_t)std::min<int64_t>(qt.size(0), INT32_MAX);
    const double scale = real(a[4]);
    const oscar_score_rule rule = score_rule(a[5], a[6], hq);
    void* out = dense(tensor(a[7], "out"), at::kBFloat16, {rows, hq, kDim}, "out");
    float* lse = a[8] == Py_None ? nullptr : static_cast<float*>(dense(tensor(a[8], "lse"), at::kFloat, {rows, hq}, "lse"));
    void* w = nullptr;
    size_t w_bytes = 0;
    if (a[9] != Py_None) {
      const at::Tensor& ws = tensor(a[9], "workspace");
      w = dense(ws, at::kByte, ws.sizes(), "workspace");
      w_bytes = (size_t)ws.numel();
    }
    auto* cache = address<oscar_cache>(a[0]);
    void* stream = stream_of(a[10]);
    return unlocked([&] {
      return oscar_scored_prefill_attention(cache, seq, rows, q, hq, (float)scale, &rule, out, lse, w, w_bytes, stream);
    });
  });
}

// Slots to read from and to write to, one of each a pair
void pairs(PyObject* so, PyObject* dst_o, std::vector<int32_t>* src, std::vector<int32_t>* dst) {
  *src = integers(so, "src");
  *dst = integers(dst_o, "dst");
  if (src->size() != dst->size()) refuse(PyExc_ValueError, "src and dst must have the same length");
}

// handle, src, dst, length, stream
PyObject* fork(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 5, [&] {
    std::vector<int32_t> src, dst;
    pairs(a[1], a[2], &src, &dst);
    const std::vector<int32_t> length = integers(a[3], "length");
    if (length.size() != src.size()) refuse(PyExc_ValueError, "length must have an entry for each pair");
    auto* cache = address<oscar_cache>(a[0]);
    void* stream = stream_of(a[4]);
    return unlocked([&] { return oscar_cache_fork(cache, (int32_t)src.size(), src.data(), dst.data(), length.data(), stream); });
  });
}

// handle, src, dst, groups (a sequence for each pair), stream
PyObject* keep_groups(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 5, [&] {
    std::vector<int32_t> src, dst;
    pairs(a[1], a[2], &src, &dst);
    PyObject* lists = PySequence_Fast(a[3], "groups must be a sequence of sequences of integers");
    if (!lists) throw Raised();
    std::vector<int32_t> groups, cu{0};
    try {
      for (Py_ssize_t i = 0; i < PySequence_Fast_GET_SIZE(lists); ++i) {
        const std::vector<int32_t> g = integers(PySequence_Fast_GET_ITEM(lists, i), "groups");
        groups.insert(groups.end(), g.begin(), g.end());
        if (groups.size() > (size_t)INT32_MAX) refuse(PyExc_ValueError, "groups has too many entries");
        cu.push_back((int32_t)groups.size());
      }
    } catch (...) {
      Py_DECREF(lists);
      throw;
    }
    Py_DECREF(lists);
    if (cu.size() != src.size() + 1) refuse(PyExc_ValueError, "groups must have a list for each pair");
    auto* cache = address<oscar_cache>(a[0]);
    void* stream = stream_of(a[4]);
    return unlocked([&] {
      return oscar_cache_keep_groups(cache, (int32_t)src.size(), src.data(), dst.data(), cu.data(), groups.data(), stream);
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
                         OSCAR_FAST(select_groups), OSCAR_FAST(sparse_decode), OSCAR_FAST(chunk),
                         OSCAR_FAST(scored_decode), OSCAR_FAST(scored_prefill), OSCAR_FAST(fork),
                         OSCAR_FAST(keep_groups),
                         OSCAR_FAST(host_in_use),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", "Calls of liboscar.so on torch tensors.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls(void) { return PyModule_Create(&module); }
