// Python calls of the cache operators: a call's tensors are checked (device, type, layout,
// size) and handed to the C entry points as addresses. The same checks in Python took
// longer than the smaller calls' kernels (7 of 12 us), and ctypes another 1.2 us.
// Holds no state but the entry points' addresses, which the package sets after it has
// loaded the library (the ordinary or the bounds-checking one).
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <exception>

#include "magicpig.h"

namespace {

decltype(&mp_cache_append) g_append = nullptr;
decltype(&mp_chunk_attention) g_attend = nullptr;
decltype(&mp_cache_weights) g_weights = nullptr;
decltype(&mp_cache_evict) g_evict = nullptr;
decltype(&mp_cache_plan) g_plan = nullptr;
decltype(&mp_prefix_attention) g_prefix = nullptr;
decltype(&mp_cache_rotate) g_rotate = nullptr;

struct Refused {};  // a Python exception is set

// Arguments of one call, taken in order.
class Args {
 public:
  Args(PyObject* const* a, Py_ssize_t n, Py_ssize_t want) : a_(a) {
    if (n != want) {
      PyErr_Format(PyExc_TypeError, "%zd arguments, %zd are needed", n, want);
      throw Refused();
    }
  }
  // the bytes of a ctypes structure, copied
  template <typename T>
  T structure(const char* name) {
    PyObject* o = a_[i_++];
    Py_buffer view;
    if (PyObject_GetBuffer(o, &view, PyBUF_SIMPLE) != 0) throw Refused();
    if (view.len != Py_ssize_t(sizeof(T))) {
      PyBuffer_Release(&view);
      PyErr_Format(PyExc_ValueError, "%s has another size than the library's structure", name);
      throw Refused();
    }
    T t = *static_cast<const T*>(view.buf);
    PyBuffer_Release(&view);
    return t;
  }
  int32_t number(const char* name) {
    const long long v = PyLong_AsLongLong(a_[i_++]);
    if (v == -1 && PyErr_Occurred()) throw Refused();
    if (v < INT_MIN || v > INT_MAX) {
      PyErr_Format(PyExc_ValueError, "%s = %lld does not fit 32 bits", name, v);
      throw Refused();
    }
    return int32_t(v);
  }
  // the first tensor: it says which device the call is for, and that has to be the current one
  const at::Tensor& first(const char* name) {
    const at::Tensor& t = tensor(a_[i_], name);
    if (!t.is_cuda()) {
      PyErr_SetString(PyExc_ValueError, "tensor arguments must be CUDA tensors (device memory)");
      throw Refused();
    }
    device_ = t.get_device();
    const int current = c10::cuda::current_device();
    if (device_ != current) {
      PyErr_Format(PyExc_ValueError, "tensors are on cuda:%d, the current device is cuda:%d", device_, current);
      throw Refused();
    }
    return t;
  }
  // address of a dense tensor of at least `numel` elements (None: nullptr, where allowed)
  void* dense(const char* name, at::ScalarType type, int64_t numel, bool none = false) {
    PyObject* o = a_[i_++];
    if (o == Py_None) {
      if (none) return nullptr;
      PyErr_Format(PyExc_ValueError, "%s is needed", name);
      throw Refused();
    }
    const at::Tensor& t = checked(o, name, type);
    if (!t.is_contiguous()) {
      PyErr_Format(PyExc_ValueError, "%s must be contiguous (dense row-major layout)", name);
      throw Refused();
    }
    if (t.numel() < numel) {
      PyErr_Format(PyExc_ValueError, "%s has %lld elements, the call uses %lld", name, (long long)t.numel(), (long long)numel);
      throw Refused();
    }
    return t.data_ptr();
  }
  // the same of a tensor whose first dimension counts `rows` rows of `width` elements: with more
  // elements (a leading dimension of one, say) the rows behind would be left out unnoticed
  void* rows_of(const char* name, at::ScalarType type, int64_t rows, int64_t width) {
    void* p = dense(name, type, rows * width);
    const at::Tensor& t = THPVariable_Unpack(a_[i_ - 1]);
    if (t.numel() != rows * width) {
      PyErr_Format(PyExc_ValueError, "%s has %lld elements, %lld rows of the call take %lld", name, (long long)t.numel(), (long long)rows,
                   (long long)(rows * width));
      throw Refused();
    }
    return p;
  }
  // address and row stride of a [rows, heads, d] tensor whose rows may lie apart
  void* rows(const char* name, at::ScalarType type, int64_t rows, int64_t heads, int64_t d, int64_t* stride) {
    const at::Tensor& t = checked(a_[i_++], name, type);
    if (t.dim() != 3 || t.size(0) != rows || t.size(1) != heads || t.size(2) != d) {
      PyErr_Format(PyExc_ValueError, "%s must be (%lld, %lld, %lld)", name, (long long)rows, (long long)heads, (long long)d);
      throw Refused();
    }
    if (t.stride(2) != 1 || (heads != 1 && t.stride(1) != d)) {
      PyErr_Format(PyExc_ValueError, "%s: the heads of a row must be dense", name);
      throw Refused();
    }
    *stride = rows > 1 ? t.stride(0) : heads * d;  // one row has no stride of its own
    return t.data_ptr();
  }
  // address of a dense [batch, heads, columns] tensor (None: nullptr), whose last two sizes come out
  void* per_slot(const char* name, at::ScalarType type, int64_t batch, int32_t* heads, int32_t* columns) {
    PyObject* o = a_[i_++];
    if (o == Py_None) return nullptr;
    const at::Tensor& t = checked(o, name, type);
    const bool fits = t.dim() == 3 && t.size(0) == batch && t.size(1) <= INT_MAX && t.size(2) <= INT_MAX;
    if (!fits || !t.is_contiguous()) {
      PyErr_Format(PyExc_ValueError, "%s must be a contiguous (%lld, heads, slots)", name, (long long)batch);
      throw Refused();
    }
    if (*columns >= 0 && (t.size(1) != *heads || t.size(2) != *columns)) {
      PyErr_Format(PyExc_ValueError, "%s has another shape than the other positions", name);
      throw Refused();
    }
    *heads = int32_t(t.size(1));
    *columns = int32_t(t.size(2));
    return t.data_ptr();
  }
  float real() {
    const double v = PyFloat_AsDouble(a_[i_++]);
    if (v == -1.0 && PyErr_Occurred()) throw Refused();
    return float(v);
  }
  size_t bytes_of_last() const { return a_[i_ - 1] == Py_None ? 0 : size_t(THPVariable_Unpack(a_[i_ - 1]).numel()); }
  // None: PyTorch's current stream; else a cudaStream_t as a number
  void* stream() {
    PyObject* o = a_[i_++];
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream(c10::DeviceIndex(device_)).stream();
    void* p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred()) throw Refused();
    return p;
  }

 private:
  const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) {
      PyErr_Format(PyExc_ValueError, "%s must be a CUDA tensor", name);
      throw Refused();
    }
    return THPVariable_Unpack(o);
  }
  const at::Tensor& checked(PyObject* o, const char* name, at::ScalarType type) {
    const at::Tensor& t = tensor(o, name);
    if (!t.is_cuda() || t.get_device() != device_) {
      PyErr_Format(PyExc_ValueError, "%s is not on cuda:%d", name, device_);
      throw Refused();
    }
    if (t.scalar_type() != type) {
      PyErr_Format(PyExc_ValueError, "%s must be %s, got %s", name, c10::toString(type), c10::toString(t.scalar_type()));
      throw Refused();
    }
    return t;
  }

  PyObject* const* a_;
  Py_ssize_t i_ = 0;
  int device_ = -1;
};

at::ScalarType type_of(const mp_cache_config& c) {
  if (c.dtype == MP_DTYPE_BF16) return at::kBFloat16;
  if (c.dtype == MP_DTYPE_F32) return at::kFloat;
  PyErr_SetString(PyExc_ValueError, "config.dtype is neither MP_DTYPE_F32 nor MP_DTYPE_BF16");
  throw Refused();
}
int64_t pool_of(const mp_cache_config& c) { return int64_t(c.n_pages) * c.kv_heads * c.page_size * c.head_dim; }

// The library call lets other threads have the interpreter: a launch waits where the device's queue
// is full. (The caller's references hold the tensors meanwhile.)
template <typename F>
int unlocked(F f) {
  struct Release {
    PyThreadState* state = PyEval_SaveThread();
    ~Release() { PyEval_RestoreThread(state); }
  } release;
  return f();
}

int append(Args a) {
  const auto cfg = a.structure<mp_cache_config>("config");
  const auto rotary = a.structure<mp_rotary>("rotary");
  const auto t = type_of(cfg);
  const int64_t rows = a.first("q").dim() ? a.first("q").size(0) : 0, d = cfg.head_dim;
  int64_t qs, ks, vs;
  const void* q = a.rows("q", t, rows, cfg.q_heads, d, &qs);
  const void* k = a.rows("k", t, rows, cfg.kv_heads, d, &ks);
  const void* v = a.rows("v", t, rows, cfg.kv_heads, d, &vs);
  const void* q_norm = a.dense("q_norm", t, d, true);
  const void* k_norm = a.dense("k_norm", t, d, true);
  const void* inv_freq = a.dense("inv_freq", at::kDouble, rotary.rot_dim / 2, true);
  const void* positions = a.dense("positions", at::kInt, rows, true);
  const void* cu_q = a.dense("cu_q", at::kInt, int64_t(cfg.batch) + 1);
  const void* kv_len = a.dense("kv_len", at::kInt, cfg.batch);
  void* keys = a.dense("keys", t, pool_of(cfg));
  void* values = a.dense("values", t, pool_of(cfg));
  const void* table = a.dense("page_table", at::kInt, int64_t(cfg.batch) * cfg.max_pages, true);
  void* q_out = a.dense("q_out", t, rows * cfg.q_heads * d);
  void* status = a.dense("status", at::kInt, 1, true);
  void* stream = a.stream();
  return unlocked([&] {
    return g_append(&cfg, &rotary, q, qs, k, ks, v, vs, q_norm, k_norm, static_cast<const double*>(inv_freq),
                    static_cast<const int32_t*>(positions), static_cast<const int32_t*>(cu_q),
                    static_cast<const int32_t*>(kv_len), int32_t(rows), keys, values, static_cast<const int32_t*>(table), q_out,
                    static_cast<uint32_t*>(status), stream);
  });
}

int attend(Args a) {
  const auto cfg = a.structure<mp_cache_config>("config");
  const auto t = type_of(cfg);
  const int64_t rows = a.first("q").dim() ? a.first("q").size(0) : 0, width = int64_t(cfg.q_heads) * cfg.head_dim;
  const void* q = a.rows_of("q", t, rows, width);
  const void* cu_q = a.dense("cu_q", at::kInt, int64_t(cfg.batch) + 1);
  const void* kv_len = a.dense("kv_len", at::kInt, cfg.batch);
  const int32_t max_q = a.number("max_q"), max_kv = a.number("max_kv");
  const void* keys = a.dense("keys", t, pool_of(cfg));
  const void* values = a.dense("values", t, pool_of(cfg));
  const void* table = a.dense("page_table", at::kInt, int64_t(cfg.batch) * cfg.max_pages, true);
  void* out = a.dense("out", t, rows * width);
  void* lse = a.dense("lse", at::kFloat, rows * cfg.q_heads, true);
  void* workspace = a.dense("workspace", at::kByte, 0, true);
  const size_t bytes = a.bytes_of_last();
  void* status = a.dense("status", at::kInt, 1, true);
  void* stream = a.stream();
  return unlocked([&] {
    return g_attend(&cfg, q, static_cast<const int32_t*>(cu_q), static_cast<const int32_t*>(kv_len), int32_t(rows), max_q, max_kv,
                    keys, values, static_cast<const int32_t*>(table), out, static_cast<float*>(lse), workspace, bytes,
                    static_cast<uint32_t*>(status), stream);
  });
}

int weights(Args a) {
  const auto cfg = a.structure<mp_cache_config>("config");
  const auto t = type_of(cfg);
  const int64_t rows = a.first("q").dim() ? a.first("q").size(0) : 0;
  const void* q = a.rows_of("q", t, rows, int64_t(cfg.q_heads) * cfg.head_dim);
  const void* lse = a.dense("lse", at::kFloat, rows * cfg.q_heads);
  const void* cu_q = a.dense("cu_q", at::kInt, int64_t(cfg.batch) + 1);
  const void* kv_len = a.dense("kv_len", at::kInt, cfg.batch);
  const int32_t max_q = a.number("max_q"), max_kv = a.number("max_kv");
  const void* keys = a.dense("keys", t, pool_of(cfg));
  const void* table = a.dense("page_table", at::kInt, int64_t(cfg.batch) * cfg.max_pages, true);
  void* scores = a.dense("scores", at::kFloat, int64_t(cfg.batch) * cfg.kv_heads * cfg.max_pages * cfg.page_size);
  void* status = a.dense("status", at::kInt, 1, true);
  void* stream = a.stream();
  return unlocked([&] {
    return g_weights(&cfg, q, static_cast<const float*>(lse), static_cast<const int32_t*>(cu_q),
                     static_cast<const int32_t*>(kv_len), int32_t(rows), max_q, max_kv, keys, static_cast<const int32_t*>(table),
                     static_cast<float*>(scores), static_cast<uint32_t*>(status), stream);
  });
}

int evict(Args a) {
  const auto cfg = a.structure<mp_cache_config>("config"), dst = a.structure<mp_cache_config>("destination config");
  const auto t = type_of(cfg);
  a.first("keys");
  const int64_t units = int64_t(cfg.batch) * cfg.kv_heads;
  const void* keys = a.dense("keys", t, pool_of(cfg));
  const void* values = a.dense("values", t, pool_of(cfg));
  const void* table = a.dense("page_table", at::kInt, int64_t(cfg.batch) * cfg.max_pages, true);
  const void* kv_len = a.dense("kv_len", at::kInt, cfg.batch);
  const int32_t max_kv = a.number("max_kv");
  const void* scores = a.dense("scores", at::kFloat, units * cfg.max_pages * cfg.page_size);
  const int32_t n_sink = a.number("n_sink"), window = a.number("window"), budget = a.number("budget");
  void* dst_keys = a.dense("dst_keys", t, pool_of(dst));
  void* dst_values = a.dense("dst_values", t, pool_of(dst));
  const void* dst_table = a.dense("dst_page_table", at::kInt, int64_t(cfg.batch) * dst.max_pages, true);
  void* dst_scores = a.dense("dst_scores", at::kFloat, units * dst.max_pages * dst.page_size, true);
  void* dst_len = a.dense("dst_len", at::kInt, cfg.batch);
  void* kept = a.dense("kept", at::kInt, units * (budget > 0 ? budget : 0), true);
  void* workspace = a.dense("workspace", at::kByte, 0);
  const size_t bytes = a.bytes_of_last();
  void* status = a.dense("status", at::kInt, 1, true);
  void* stream = a.stream();
  return unlocked([&] {
    return g_evict(&cfg, &dst, keys, values, static_cast<const int32_t*>(table), static_cast<const int32_t*>(kv_len), max_kv,
                   static_cast<const float*>(scores), n_sink, window, budget, dst_keys, dst_values,
                   static_cast<const int32_t*>(dst_table), static_cast<float*>(dst_scores), static_cast<int32_t*>(dst_len),
                   static_cast<int32_t*>(kept), workspace, bytes, static_cast<uint32_t*>(status), stream);
  });
}

int plan(Args a) {
  const auto cfg = a.structure<mp_cache_config>("config");
  a.first("change");
  const int64_t batch = cfg.batch;
  const void* change = a.dense("change", at::kInt, batch);
  const void* base = a.dense("base", at::kInt, batch, true);
  const void* kv_len = a.dense("kv_len", at::kInt, batch);
  const void* n_free = a.dense("n_free", at::kInt, 1, true);
  const int32_t max_rows = a.number("max_rows");
  void* table = a.dense("page_table", at::kInt, batch * cfg.max_pages, true);
  void* free_pages = a.dense("free_pages", at::kInt, cfg.n_pages, true);
  void* new_len = a.dense("new_len", at::kInt, batch);
  void* new_free = a.dense("new_free", at::kInt, 1, true);
  void* cu_q = a.dense("cu_q", at::kInt, batch + 1);
  void* positions = a.dense("positions", at::kInt, max_rows, true);
  void* slots = a.dense("slots", at::kInt, max_rows, true);
  void* row_seq = a.dense("row_seq", at::kInt, max_rows, true);
  void* status = a.dense("status", at::kInt, 1, true);
  void* stream = a.stream();
  return unlocked([&] {
    return g_plan(&cfg, static_cast<const int32_t*>(change), static_cast<const int32_t*>(base), static_cast<const int32_t*>(kv_len),
                  static_cast<const int32_t*>(n_free), max_rows, static_cast<int32_t*>(table), static_cast<int32_t*>(free_pages),
                  static_cast<int32_t*>(new_len), static_cast<int32_t*>(new_free), static_cast<int32_t*>(cu_q),
                  static_cast<int32_t*>(positions), static_cast<int32_t*>(slots), static_cast<int32_t*>(row_seq),
                  static_cast<uint32_t*>(status), stream);
  });
}

int prefix(Args a) {
  const auto cfg = a.structure<mp_cache_config>("config"), pre = a.structure<mp_cache_config>("prefix config");
  const auto t = type_of(cfg);
  const int64_t rows = a.first("q").dim() ? a.first("q").size(0) : 0, width = int64_t(cfg.q_heads) * cfg.head_dim;
  const void* q = a.rows_of("q", t, rows, width);
  const void* cu_q = a.dense("cu_q", at::kInt, int64_t(cfg.batch) + 1);
  const void* kv_len = a.dense("kv_len", at::kInt, cfg.batch);
  const int32_t max_q = a.number("max_q"), max_kv = a.number("max_kv");
  const void* keys = a.dense("keys", t, pool_of(cfg));
  const void* values = a.dense("values", t, pool_of(cfg));
  const void* table = a.dense("page_table", at::kInt, int64_t(cfg.batch) * cfg.max_pages, true);
  const void* cu_group = a.dense("cu_group", at::kInt, int64_t(pre.batch) + 1);
  const void* prefix_len = a.dense("prefix_len", at::kInt, pre.batch);
  const int32_t max_group_q = a.number("max_group_q"), max_prefix = a.number("max_prefix");
  const void* prefix_keys = a.dense("prefix_keys", t, pool_of(pre));
  const void* prefix_values = a.dense("prefix_values", t, pool_of(pre));
  const void* prefix_table = a.dense("prefix_table", at::kInt, int64_t(pre.batch) * pre.max_pages, true);
  void* out = a.rows_of("out", t, rows, width);
  void* lse = a.dense("lse", at::kFloat, rows * cfg.q_heads, true);
  void* workspace = a.dense("workspace", at::kByte, 0, true);
  const size_t bytes = a.bytes_of_last();
  void* status = a.dense("status", at::kInt, 1, true);
  void* stream = a.stream();
  return unlocked([&] {
    return g_prefix(&cfg, &pre, q, static_cast<const int32_t*>(cu_q), static_cast<const int32_t*>(kv_len), int32_t(rows), max_q,
                    max_kv, keys, values, static_cast<const int32_t*>(table), static_cast<const int32_t*>(cu_group),
                    static_cast<const int32_t*>(prefix_len), max_group_q, max_prefix, prefix_keys, prefix_values,
                    static_cast<const int32_t*>(prefix_table), out, static_cast<float*>(lse), workspace, bytes,
                    static_cast<uint32_t*>(status), stream);
  });
}

int rotate(Args a) {
  const auto cfg = a.structure<mp_cache_config>("config");
  const auto rotary = a.structure<mp_rotary>("rotary");
  const auto t = type_of(cfg);
  a.first("keys");
  void* keys = a.dense("keys", t, pool_of(cfg));
  const void* table = a.dense("page_table", at::kInt, int64_t(cfg.batch) * cfg.max_pages, true);
  const void* kv_len = a.dense("kv_len", at::kInt, cfg.batch);
  const int32_t max_kv = a.number("max_kv");
  const void* from_freq = a.dense("from_freq", at::kDouble, rotary.rot_dim / 2, true);
  const void* to_freq = a.dense("to_freq", at::kDouble, rotary.rot_dim / 2, true);
  int32_t heads = 1, columns = -1;
  const void* from = a.per_slot("from_positions", at::kInt, cfg.batch, &heads, &columns);
  const void* to = a.per_slot("to_positions", at::kInt, cfg.batch, &heads, &columns);
  const float scale = a.real();
  void* status = a.dense("status", at::kInt, 1, true);
  void* stream = a.stream();
  return unlocked([&] {
    return g_rotate(&cfg, &rotary, keys, static_cast<const int32_t*>(table), static_cast<const int32_t*>(kv_len), max_kv,
                    static_cast<const double*>(from_freq), static_cast<const double*>(to_freq), static_cast<const int32_t*>(from),
                    static_cast<const int32_t*>(to), heads, columns < 0 ? 0 : columns, scale, static_cast<uint32_t*>(status), stream);
  });
}

// METH_FASTCALL entry: the library's return code, or a Python exception
template <int (*F)(Args), int N>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  try {
    return PyLong_FromLong(F(Args(args, n, N)));
  } catch (const Refused&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// The entry points' addresses, in the order of `to`.
template <int N>
PyObject* take(PyObject* const* args, Py_ssize_t n, void** const (&to)[N]) {
  void* p[N];
  if (n != N) return PyErr_Format(PyExc_TypeError, "%d addresses are needed", N);
  for (int i = 0; i < N; ++i) {
    p[i] = PyLong_AsVoidPtr(args[i]);
    if (!p[i]) return PyErr_Occurred() ? nullptr : PyErr_Format(PyExc_ValueError, "a null address");
  }
  for (int i = 0; i < N; ++i) *to[i] = p[i];
  Py_RETURN_NONE;
}
template <typename F>
void** place(F& f) {
  return reinterpret_cast<void**>(&f);
}
// bind(append, attend, weights, evict)
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return take<4>(args, n, {place(g_append), place(g_attend), place(g_weights), place(g_evict)});
}
// bind_shared(plan, prefix, rotate)
PyObject* bind_shared(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return take<3>(args, n, {place(g_plan), place(g_prefix), place(g_rotate)});
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f))
PyMethodDef methods[] = {{"bind", FAST(bind), METH_FASTCALL, nullptr},
                         {"bind_shared", FAST(bind_shared), METH_FASTCALL, nullptr},
                         {"append", FAST((call<append, 17>)), METH_FASTCALL, nullptr},
                         {"attend", FAST((call<attend, 14>)), METH_FASTCALL, nullptr},
                         {"weights", FAST((call<weights, 12>)), METH_FASTCALL, nullptr},
                         {"evict", FAST((call<evict, 20>)), METH_FASTCALL, nullptr},
                         {"plan", FAST((call<plan, 16>)), METH_FASTCALL, nullptr},
                         {"prefix", FAST((call<prefix, 22>)), METH_FASTCALL, nullptr},
                         {"rotate", FAST((call<rotate, 13>)), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_mp_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mp_calls() { return PyModule_Create(&module); }
