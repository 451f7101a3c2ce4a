// Python marshalling of the serving calls (module _serving): tensors become
// device pointers and strides, checked once, and the C entry point is called.
//
// These calls come once per layer and decode step and their kernels take a few
// microseconds; the same checks written in Python with a ctypes call behind them
// took 8 of a small call's 12.  Each function returns the entry point's code; a
// tensor that does not fit raises what the `fail` function given to set_fail makes.
#include <Python.h>
#include <c10/core/DeviceGuard.h>
#include <torch/csrc/autograd/python_variable.h>

#include <vector>

#include "cpkv.h"

namespace {

// The pools as the binding's PoolTable describes them (the same fields there).
struct Table {
  uint64_t addresses, caps;
  int64_t row_bytes, key_offset, value_offset;
  int32_t page_size, cp_size, code, flags, device;
  void *const *pools() const { return reinterpret_cast<void *const *>(addresses); }
  const int64_t *cap_pages() const { return reinterpret_cast<const int64_t *>(caps); }
};

PyObject *g_fail = nullptr;

// An error is set; the caller returns.
struct Failed {};

[[noreturn]] void fail(const char *name, const char *what) {
  PyObject *e = g_fail ? PyObject_CallFunction(g_fail, "ss", name, what) : nullptr;
  if (e != nullptr) {
    PyErr_SetObject(reinterpret_cast<PyObject *>(Py_TYPE(e)), e);
    Py_DECREF(e);
  } else if (!PyErr_Occurred()) {
    PyErr_Format(PyExc_ValueError, "%s: %s is wanted", name, what);
  }
  throw Failed();
}

const at::Tensor &tensor(PyObject *o, const char *name, const Table &t, at::ScalarType type, const char *what) {
  if (!THPVariable_Check(o)) fail(name, what);
  const at::Tensor &x = THPVariable_Unpack(o);
  if (!x.is_cuda() || x.device().index() != t.device || x.scalar_type() != type) fail(name, what);
  return x;
}

at::ScalarType element(const Table &t) { return t.code == CPKV_BF16 ? at::kBFloat16 : at::kHalf; }

// A [tokens, heads, dim] tensor whose heads are contiguous within a token.
struct Rows {
  void *at;
  int64_t stride, n, heads, dim;
  bool same_shape(const Rows &o) const { return n == o.n && heads == o.heads && dim == o.dim; }
};

Rows rows(PyObject *o, const char *name, const Table &t) {
  static const char *const what = "[tokens, heads, dim] of the pools' type on their device, a token's heads side by side";
  const at::Tensor &x = tensor(o, name, t, element(t), what);
  if (x.dim() != 3) fail(name, what);
  const auto size = x.sizes(), stride = x.strides();
  if ((stride[2] != 1 && size[2] > 1) || (stride[1] != size[2] && size[1] > 1)) fail(name, what);
  const int64_t width = size[1] * size[2];  // also the stride of a single token, which has none
  return Rows{x.data_ptr(), size[0] > 1 ? stride[0] : width, size[0], size[1], size[2]};
}

// A contiguous device list.
template <typename T>
T *list(PyObject *o, const char *name, const Table &t, at::ScalarType type, int64_t *n) {
  static const char *const what = "a contiguous list of its whole-number type on the pools' device";
  const at::Tensor &x = tensor(o, name, t, type, what);
  if (x.dim() != 1 || !x.is_contiguous()) fail(name, what);
  *n = x.size(0);
  return static_cast<T *>(x.data_ptr());
}

// A [requests, pages] table.
struct PageRows {
  const int32_t *at;
  int64_t stride, pages;
};

PageRows page_rows(PyObject *o, const char *name, const Table &t, int64_t requests) {
  static const char *const what = "int32 on the pools' device, a contiguous row of page ids per request";
  const at::Tensor &x = tensor(o, name, t, at::kInt, what);
  if (x.dim() != 2 || x.size(0) != requests || (x.stride(1) != 1 && x.size(1) > 1)) fail(name, what);
  if (requests > 1 && x.stride(0) < x.size(1)) fail(name, what);
  return PageRows{static_cast<const int32_t *>(x.data_ptr()), requests > 1 ? x.stride(0) : x.size(1), x.size(1)};
}

float *lse_of(PyObject *o, const Table &t, const Rows &q) {
  if (o == Py_None) return nullptr;
  static const char *const what = "contiguous float32 [tokens, heads]";
  const at::Tensor &x = tensor(o, "lse", t, at::kFloat, what);
  if (x.dim() != 2 || x.size(0) != q.n || x.size(1) != q.heads || !x.is_contiguous()) fail("lse", what);
  return static_cast<float *>(x.data_ptr());
}

// A workspace and its bytes.
void *memory(PyObject *o, const Table &t, int64_t *bytes) {
  *bytes = 0;
  if (o == Py_None) return nullptr;
  static const char *const what = "a contiguous tensor on the pools' device";
  if (!THPVariable_Check(o)) fail("workspace", what);
  const at::Tensor &x = THPVariable_Unpack(o);
  if (!x.is_cuda() || x.device().index() != t.device || !x.is_contiguous()) fail("workspace", what);
  *bytes = static_cast<int64_t>(x.nbytes());
  return x.data_ptr();
}

int32_t *status_word(PyObject *o, const Table &t) {
  static const char *const what = "an int32 on the pools' device";
  const at::Tensor &x = tensor(o, "status", t, at::kInt, what);
  if (x.numel() < 1) fail("status", what);
  return static_cast<int32_t *>(x.data_ptr());
}

// Host lengths: an int32 array as it is, other sequences copied.
class Lengths {
 public:
  explicit Lengths(PyObject *o) {
    if (o == Py_None) return;
    if (PyObject_CheckBuffer(o)) {
      if (PyObject_GetBuffer(o, &view_.buffer, PyBUF_ND | PyBUF_FORMAT | PyBUF_C_CONTIGUOUS) == 0) {
        view_.held = true;
        const Py_buffer &v = view_.buffer;
        if (v.ndim == 1 && v.itemsize == 4 && v.format != nullptr && (v.format[0] == 'i' || v.format[0] == 'l')) {
          at_ = static_cast<const int32_t *>(v.buf);
          count_ = v.shape[0];
          return;
        }
      } else {
        PyErr_Clear();
      }
    }
    PyObject *seq = PySequence_Fast(o, "lengths: a sequence of whole numbers is wanted");
    if (seq == nullptr) throw Failed();
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(seq);
    copy_.resize(n);
    for (Py_ssize_t i = 0; i < n && !PyErr_Occurred(); ++i) {
      const long long v = PyLong_AsLongLong(PySequence_Fast_GET_ITEM(seq, i));
      copy_[i] = v < INT32_MIN || v > INT32_MAX ? -1 : static_cast<int32_t>(v);
    }
    Py_DECREF(seq);
    if (PyErr_Occurred()) throw Failed();
    at_ = copy_.data();
    count_ = n;
  }
  const int32_t *at() const { return at_; }
  int64_t count() const { return count_; }

 private:
  struct View {  // released also when the constructor above throws
    Py_buffer buffer;
    bool held = false;
    View() = default;
    View(const View &) = delete;
    ~View() {
      if (held) PyBuffer_Release(&buffer);
    }
  };
  View view_;
  std::vector<int32_t> copy_;
  const int32_t *at_ = nullptr;
  int64_t count_ = 0;
};

int64_t whole(PyObject *o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Failed();
  return v;
}

int small(PyObject *o, const char *name) {
  const int64_t v = whole(o);
  if (v < INT32_MIN || v > INT32_MAX) fail(name, "a 32-bit number");
  return static_cast<int>(v);
}

// An address that Python holds as a number.
template <typename T>
T address(PyObject *o) {
  const unsigned long long v = PyLong_AsUnsignedLongLong(o);
  if (v == static_cast<unsigned long long>(-1) && PyErr_Occurred()) throw Failed();
  return reinterpret_cast<T>(static_cast<uintptr_t>(v));
}

const Table &table(PyObject *o) {
  const Table *t = address<const Table *>(o);
  if (t == nullptr) fail("table", "a PoolTable's address");
  return *t;
}

cpkv_stream_t stream_of(PyObject *o) { return address<cpkv_stream_t>(o); }

double real(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Failed();
  return v;
}

// Runs a call, its first argument the table, with the pools' device current: the entry
// points launch on the current device, and their stream handle is one of the pools'.
// Python sees an exception instead of C++.
template <typename F>
PyObject *guarded(PyObject *const *a, Py_ssize_t got, Py_ssize_t wanted, F f) {
  if (got != wanted) {
    PyErr_Format(PyExc_TypeError, "%zd arguments: %zd are wanted", got, wanted);
    return nullptr;
  }
  try {
    const Table &t = table(a[0]);
    const c10::DeviceGuard current(c10::Device(c10::kCUDA, static_cast<c10::DeviceIndex>(t.device)));
    const int rc = f(t);
    if (PyErr_Occurred()) return nullptr;
    return PyLong_FromLong(rc);
  } catch (const Failed &) {
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown error");
  }
  return nullptr;
}

// (table, kv_heads, key_dim, value_dim, k, v, slots, positions, cos_sin, status, q, q_out, axis_of_freq, interleaved, stream)
PyObject *append_rotary(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(a, n, 15, [&](const Table &t) {
    const Rows k = rows(a[4], "k", t), v = rows(a[5], "v", t);
    if (k.heads != whole(a[1]) || k.dim != whole(a[2])) fail("k", "[tokens, kv_heads, key_dim] of the cache");
    if (v.n != k.n || v.heads != k.heads || v.dim != whole(a[3])) fail("v", "[tokens, kv_heads, value_dim] of the cache, k's tokens");
    int64_t count = 0;
    const int64_t *slots = list<int64_t>(a[6], "slots", t, at::kLong, &count);
    if (count != k.n) fail("slots", "a slot per token");
    static const char *const of_positions = "int32 [tokens] or [axes, tokens] on the pools' device";
    const at::Tensor &pos = tensor(a[7], "positions", t, at::kInt, of_positions);
    if (pos.dim() < 1 || pos.dim() > 2 || pos.size(-1) != k.n || (pos.stride(-1) != 1 && k.n > 1)) fail("positions", of_positions);
    const int64_t axes = pos.dim() == 1 ? 1 : pos.size(0), between = pos.dim() == 1 ? k.n : pos.stride(0);
    static const char *const of_table = "contiguous float32 [positions, rot_dim] on the pools' device";
    const at::Tensor &turns = tensor(a[8], "cos_sin", t, at::kFloat, of_table);
    if (turns.dim() != 2 || !turns.is_contiguous() || axes > INT32_MAX || turns.size(1) > INT32_MAX) fail("cos_sin", of_table);
    int32_t *status = status_word(a[9], t);
    Rows q = {nullptr, 0, 0, 0, k.dim}, q_out = q;
    if (a[10] != Py_None) {
      q = rows(a[10], "q", t);
      q_out = rows(a[11], "q_out", t);
      if (!q.same_shape(q_out) || q.n != k.n || q.dim != k.dim) fail("q and q_out", "k's tokens and width, alike");
    }
    const uint8_t *axis = nullptr;
    if (a[12] != Py_None) {
      if (!PyBytes_Check(a[12]) || PyBytes_GET_SIZE(a[12]) != turns.size(1) / 2) fail("axis_of_freq", "an axis per frequency");
      axis = reinterpret_cast<const uint8_t *>(PyBytes_AS_STRING(a[12]));
    }
    const int interleaved = PyObject_IsTrue(a[13]);
    if (interleaved < 0) throw Failed();
    const int flags = t.flags | (interleaved ? CPKV_ROTARY_INTERLEAVED : 0);
    return cpkv_append_rotary(k.n, t.page_size, t.cp_size, t.code, static_cast<int>(q.heads), static_cast<int>(k.heads),
                              static_cast<int>(k.dim), static_cast<int>(v.dim), t.row_bytes, t.key_offset, t.value_offset,
                              t.pools(), t.cap_pages(), k.at, k.stride, v.at, v.stride, q.at, q.stride, q_out.at, q_out.stride,
                              slots, static_cast<const int32_t *>(pos.data_ptr()), between, static_cast<int>(axes), axis,
                              static_cast<const float *>(turns.data_ptr()), turns.size(0), static_cast<int>(turns.size(1)),
                              flags, status, stream_of(a[14]));
  });
}

// (table, kv_heads, q, q_lens, page_table, kv_lens, max_kv_len, window, sinks, scale, out, lse, workspace, status, stream)
PyObject *attend_window(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(a, n, 15, [&](const Table &t) {
    const Rows q = rows(a[2], "q", t), out = rows(a[10], "out", t);
    if (!q.same_shape(out)) fail("out", "q's shape");
    int64_t requests = 0, bytes = 0;
    const int32_t *kv_lens = list<int32_t>(a[5], "kv_lens", t, at::kInt, &requests);
    const PageRows pages = page_rows(a[4], "page_table", t, requests);
    const Lengths q_lens(a[3]);
    if (q_lens.at() != nullptr && q_lens.count() != requests) fail("q_lens", "a length per request");
    const int64_t max_kv = whole(a[6]);
    if (max_kv > pages.pages * t.page_size) return CPKV_ERR_CAPACITY;
    const double scale = real(a[9]);
    float *lse = lse_of(a[11], t, q);
    void *workspace = memory(a[12], t, &bytes);
    int32_t *status = status_word(a[13], t);
    if (requests > INT32_MAX || q.heads > INT32_MAX || q.dim > INT32_MAX) return CPKV_ERR_LIMIT;
    return cpkv_attend_window(static_cast<int>(requests), t.page_size, t.cp_size, t.code, static_cast<int>(q.heads),
                              small(a[1], "kv_heads"), static_cast<int>(q.dim), t.row_bytes, t.key_offset, t.value_offset,
                              q_lens.at(), max_kv, t.pools(), t.cap_pages(), pages.at, pages.stride, kv_lens, q.n, q.at,
                              q.stride, static_cast<float>(scale), small(a[7], "window"), small(a[8], "sinks"), out.at,
                              out.stride, lse, workspace, bytes, t.flags, status, stream_of(a[14]));
  });
}

// (table, kv_heads, q, group_sizes, prefix_lens, prefix_pages, page_table, suffix_lens, max_suffix_len, scale, out, lse, workspace, status, stream)
PyObject *attend_shared(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(a, n, 15, [&](const Table &t) {
    const Rows q = rows(a[2], "q", t), out = rows(a[10], "out", t);
    if (!q.same_shape(out)) fail("out", "q's shape");
    int64_t requests = 0, prefix_pages = 0, bytes = 0;
    const int32_t *suffix_lens = list<int32_t>(a[7], "suffix_lens", t, at::kInt, &requests);
    const int32_t *prefix = list<int32_t>(a[5], "prefix_pages", t, at::kInt, &prefix_pages);
    const PageRows pages = page_rows(a[6], "page_table", t, requests);
    const Lengths sizes(a[3]), lens(a[4]);
    if (q.n != requests || sizes.count() != lens.count()) fail("q, group_sizes and prefix_lens", "a query per request, a prefix length per group");
    const int64_t max_suffix = whole(a[8]);
    if (max_suffix > pages.pages * t.page_size) return CPKV_ERR_CAPACITY;
    const double scale = real(a[9]);
    float *lse = lse_of(a[11], t, q);
    void *workspace = memory(a[12], t, &bytes);
    int32_t *status = status_word(a[13], t);
    if (requests > INT32_MAX || q.heads > INT32_MAX || q.dim > INT32_MAX || sizes.count() > INT32_MAX) return CPKV_ERR_LIMIT;
    return cpkv_attend_shared(static_cast<int>(requests), static_cast<int>(sizes.count()), t.page_size, t.cp_size, t.code,
                              static_cast<int>(q.heads), small(a[1], "kv_heads"), static_cast<int>(q.dim), t.row_bytes,
                              t.key_offset, t.value_offset, sizes.at(), lens.at(), max_suffix, t.pools(), t.cap_pages(),
                              prefix, prefix_pages, pages.at, pages.stride, suffix_lens, q.at, q.stride,
                              static_cast<float>(scale), out.at, out.stride, lse, workspace, bytes, t.flags, status,
                              stream_of(a[14]));
  });
}

// (stream) -> whether calls on it go into a CUDA graph; not where that cannot be told (the
// default stream beside a capture).
PyObject *captures(PyObject *, PyObject *stream) {
  int yes = 0;
  try {
    if (cpkv_stream_is_capturing(stream_of(stream), &yes) != CPKV_OK) yes = 0;
  } catch (const Failed &) {
    return nullptr;
  }
  return PyBool_FromLong(yes);
}

// The function (name, what is wanted) that makes an exception.
PyObject *set_fail(PyObject *, PyObject *f) {
  Py_INCREF(f);
  Py_XSETREF(g_fail, f);
  Py_RETURN_NONE;
}

template <typename F>
PyCFunction as_method(F *f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(f));
}

PyMethodDef methods[] = {{"append_rotary", as_method(append_rotary), METH_FASTCALL, nullptr},
                         {"attend_window", as_method(attend_window), METH_FASTCALL, nullptr},
                         {"attend_shared", as_method(attend_shared), METH_FASTCALL, nullptr},
                         {"captures", captures, METH_O, nullptr},
                         {"set_fail", set_fail, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_serving", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serving() {
  PyObject *m = PyModule_Create(&module);
  if (m != nullptr && PyModule_AddStringConstant(m, "built_for", BUILT_FOR) < 0) Py_CLEAR(m);
  return m;
}
