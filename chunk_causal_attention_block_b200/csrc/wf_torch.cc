// Python entry of the batch calls for torch tensors: checks and passes on the
// arguments of wf_batch_tables, wf_batch_append and wf_batch_attn (wf.py holds
// the functions that users call).
//
// These calls run once a step or a layer on as little as one token, where the
// host is what takes the time: asking each of up to 14 tensors for its layout,
// type, size, device and address from Python took 4 us of a call, ctypes
// another 1.2 us.  Here it is a few field reads per tensor.  (A call with the
// stream's lookup, 3.2 us, and its launches: tables of 5 requests 13.7 -> 8.4
// us, append of 32 tokens 12.2 -> 8.0 us, attention of one token 16.3 -> 11.1
// us.)
//
// An argument is a CUDA tensor, dense, of the type and at least the size that
// the call may touch and on the device of the plan (the current one, if the plan
// is an address: the library looks where that lies); None; or a raw address,
// which its owner vouches for.  A tensor of more dimensions than one also has
// to have rows of the documented length: one with longer rows (spare table
// columns, more heads) would hold enough elements and be read at the wrong
// stride.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/core/impl/VirtualGuardImpl.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <cstring>
#include <sstream>
#include <string>

#include "wf_batch.h"

namespace {

decltype(&wf_batch_tables) g_tables = nullptr;
decltype(&wf_batch_append) g_append = nullptr;
decltype(&wf_batch_attn) g_attn = nullptr;

struct Refused {
  std::string why;
};

constexpr int kAnyDevice = -1, kCurrentDevice = -2;
constexpr auto kInt = at::ScalarType::Int, kFloat = at::ScalarType::Float, kBf16 = at::ScalarType::BFloat16;
constexpr auto kBytes = at::ScalarType::Undefined;  // memory without a type of its own: elements of one byte

// Rows that a tensor consists of: `row` elements, their last dimension `inner`
// (or all of the row, or `flat`, several rows in one).
struct Rows {
  int64_t row, inner, flat;
  explicit Rows(int64_t n) : row(n), inner(n), flat(n) {}
  Rows(int64_t n, int64_t last) : row(n), inner(last), flat(n) {}
  Rows(int64_t n, int64_t last, int64_t all) : row(n), inner(last), flat(all) {}

  // Of n elements that the call may touch; with a single row, its end does not matter.
  bool fit(const at::Tensor& t, int64_t n) const {
    const auto sizes = t.sizes();
    size_t dims = sizes.size();
    while (dims > 1 && sizes[dims - 1] == 1) --dims;
    if (dims < 2 || n <= row) return true;
    const int64_t last = sizes[dims - 1];
    if (last == flat || last == row) return true;
    int64_t product = 1;
    for (size_t i = dims; i-- > 0;)
      if ((product *= sizes[i]) == row) return last == inner;
    return false;
  }
};

// Turns arguments into addresses.
struct Reader {
  const char* const* names;
  PyObject* const* args;
  int device = kAnyDevice;

  static const at::Tensor* tensor(PyObject* x) { return THPVariable_Check(x) ? &THPVariable_Unpack(x) : nullptr; }

  // The call's plan settles the device of all its tensors.  (Kernels that read one find out by themselves whether
  // it was built for the call's description.)
  void* plan(int i) {
    void* p = address(i, WF_BATCH_PLAN_HEAD, kBytes);
    const at::Tensor* t = tensor(args[i]);
    device = t ? t->get_device() : kCurrentDevice;
    return p;
  }

  bool here(const at::Tensor& t) const {
    if (!t.is_cuda() || device == kAnyDevice) return t.is_cuda();
    return t.get_device() == (device == kCurrentDevice
                                  ? c10::impl::VirtualGuardImpl(c10::DeviceType::CUDA).getDevice().index()
                                  : device);
  }

  void* address(int i, int64_t n, at::ScalarType type, const Rows* rows = nullptr) const {
    PyObject* x = args[i];
    if (x == Py_None) return nullptr;
    if (const at::Tensor* t = tensor(x)) {
      if (type == kBytes ? t->itemsize() != 1 : t->scalar_type() != type)
        throw Refused{std::string(names[i]) + " is of type " + c10::toString(t->scalar_type()) + " where " +
                      (type == kBytes ? "bytes" : c10::toString(type)) + " is needed"};
      if (rows && !rows->fit(*t, n)) {
        std::ostringstream s;
        s << names[i] << " is of shape " << t->sizes() << " where rows of " << rows->row << " elements are needed";
        throw Refused{s.str()};
      }
      const bool dense = t->layout() == at::kStrided && t->is_contiguous();
      if (dense && t->numel() >= n && here(*t)) return t->data_ptr();
      std::ostringstream s;
      s << names[i] << " has " << t->numel() << " elements on " << t->device() << (dense ? "" : ", not dense")
        << " where " << n << " are needed on " << (device == kAnyDevice       ? "a GPU"
                                                   : device == kCurrentDevice ? "the current GPU"
                                                                              : "the plan's GPU");
      throw Refused{s.str()};
    }
    if (!PyLong_Check(x)) throw Refused{std::string(names[i]) + " is neither a tensor nor an address nor None"};
    void* p = PyLong_AsVoidPtr(x);
    if (PyErr_Occurred()) throw Refused{std::string(names[i]) + " is not an address"};
    return p;
  }

  // A number, or what the tensor args[of] holds if it is None.  No more than that is believed.
  int64_t number(int i, int of, bool bytes) const {
    const at::Tensor* t = tensor(args[of]);
    if (args[i] != Py_None) {
      const int64_t v = PyLong_AsLongLong(args[i]);
      if (v == -1 && PyErr_Occurred()) throw Refused{std::string(names[i]) + " is not a number"};
      if (t && v > (bytes ? int64_t(t->nbytes()) : t->numel()))
        throw Refused{std::string(names[i]) + " is more than " + names[of] + " holds"};
      return v;
    }
    if (args[of] == Py_None) return 0;
    if (!t) throw Refused{std::string(names[i]) + " is needed where " + names[of] + " is an address"};
    return bytes ? int64_t(t->nbytes()) : t->numel();
  }
};

bool read_desc(PyObject* x, wf_batch_desc* d) {
  Py_buffer b;
  if (PyObject_GetBuffer(x, &b, PyBUF_SIMPLE) != 0) return false;
  const bool ok = b.len == Py_ssize_t(sizeof(*d));
  if (ok) std::memcpy(d, b.buf, sizeof(*d));
  PyBuffer_Release(&b);
  if (!ok) PyErr_SetString(PyExc_TypeError, "not a batch description");
  return ok;
}

// Runs f(desc, reader) -> call; returns the call's status, or the reason why it was not made.
template <int N, typename F>
PyObject* guarded(const char* const (&names)[N], PyObject* const* args, Py_ssize_t nargs, F f) {
  if (nargs != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments, not %d", N, int(nargs));
    return nullptr;
  }
  wf_batch_desc d;
  if (!read_desc(args[0], &d)) return nullptr;
  try {
    return PyLong_FromLong(f(d, Reader{names, args}));
  } catch (const Refused& r) {
    PyErr_Clear();
    return PyUnicode_FromString(r.why.c_str());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

template <typename F>
wf_status without_gil(F f) {
  wf_status s;
  Py_BEGIN_ALLOW_THREADS
  s = f();
  Py_END_ALLOW_THREADS
  return s;
}

PyObject* tables(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  static const char* const names[] = {"desc", "plan", "cached", "fresh", "prefix_len", "held", "free_pages", "num_free",
                                      "free_head", "free_head_out", "held_out", "block_table", "token_start",
                                      "slot_map", "positions", "plan_bytes", "stream"};
  return guarded(names, args, nargs, [](const wf_batch_desc& d, Reader r) {
    const int64_t plan_bytes = r.number(15, 1, true);
    void* plan = r.plan(1);
    auto i32 = [&](int i, int64_t n) { return static_cast<int32_t*>(r.address(i, n, kInt)); };
    const int64_t B = d.max_requests, T = d.max_tokens;
    const Rows columns(d.max_request_pages);
    int32_t *cached = i32(2, B), *fresh = i32(3, B), *prefix_len = i32(4, 1), *held = i32(5, B);
    const int64_t num_free = r.number(7, 6, false);
    if (num_free > INT32_MAX || num_free < INT32_MIN) throw Refused{"num_free does not fit"};
    int32_t *free_pages = i32(6, num_free), *head = i32(8, 1), *head_out = i32(9, 1), *held_out = i32(10, B);
    int32_t *table = static_cast<int32_t*>(r.address(11, B * d.max_request_pages, kInt, &columns)),
            *start = i32(12, B + 1), *slots = i32(13, T), *pos = i32(14, T);
    auto stream = static_cast<wf_stream_t>(r.address(16, 0, kBytes));
    return without_gil([&] {
      return g_tables(&d, cached, fresh, prefix_len, held, free_pages, int32_t(num_free), head, head_out, held_out, table,
                      start, slots, pos, plan, plan_bytes < 0 ? 0 : size_t(plan_bytes), stream);
    });
  });
}

PyObject* append(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  static const char* const names[] = {"desc", "plan", "slot_map", "rope", "q", "k", "v", "q_rot", "k_pool", "v_pool",
                                      "stream"};
  return guarded(names, args, nargs, [](const wf_batch_desc& d, Reader r) {
    void* plan = r.plan(1);
    // a step may hold fewer tokens than max_tokens: only the device knows, so room for all is asked for
    const int64_t T = d.max_tokens, kv = int64_t(d.num_kv_heads) * d.head_dim, q_size = T * d.num_heads * d.head_dim;
    const int64_t pool = int64_t(d.pool_pages) * d.page_tokens * kv;
    const Rows q_rows(int64_t(d.num_heads) * d.head_dim, d.head_dim), kv_rows(kv, d.head_dim),
        pool_rows(kv, d.head_dim, d.page_tokens * kv), rope_rows(d.head_dim, 2);
    auto slots = static_cast<const int32_t*>(r.address(2, T, kInt));
    auto rope = static_cast<const float*>(r.address(3, T * d.head_dim, kFloat, &rope_rows));
    void *q = r.address(4, q_size, kBf16, &q_rows), *q_rot = r.address(7, q_size, kBf16, &q_rows);
    void *k = r.address(5, T * kv, kBf16, &kv_rows), *v = r.address(6, T * kv, kBf16, &kv_rows);
    void *k_pool = r.address(8, pool, kBf16, &pool_rows), *v_pool = r.address(9, pool, kBf16, &pool_rows);
    auto stream = static_cast<wf_stream_t>(r.address(10, 0, kBytes));
    return without_gil([&] { return g_append(&d, plan, slots, rope, q, k, v, q_rot, k_pool, v_pool, stream); });
  });
}

PyObject* attn(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  static const char* const names[] = {"desc", "plan", "block_table", "prefix_table", "q", "k_pool", "v_pool", "out",
                                      "lse", "softmax_scale", "workspace", "workspace_bytes", "stream"};
  return guarded(names, args, nargs, [args](const wf_batch_desc& d, Reader r) {
    void* plan = r.plan(1);
    const int64_t T = d.max_tokens, kv = int64_t(d.num_kv_heads) * d.head_dim, q_size = T * d.num_heads * d.head_dim;
    const int64_t pool = int64_t(d.pool_pages) * d.page_tokens * kv;
    const Rows q_rows(int64_t(d.num_heads) * d.head_dim, d.head_dim), pool_rows(kv, d.head_dim, d.page_tokens * kv),
        columns(d.max_request_pages), lse_rows(T);
    auto table = static_cast<const int32_t*>(r.address(2, int64_t(d.max_requests) * d.max_request_pages, kInt, &columns));
    auto prefix = static_cast<const int32_t*>(r.address(3, d.max_prefix_pages, kInt));
    void *q = r.address(4, q_size, kBf16, &q_rows), *out = r.address(7, q_size, kBf16, &q_rows);
    void *k_pool = r.address(5, pool, kBf16, &pool_rows), *v_pool = r.address(6, pool, kBf16, &pool_rows);
    auto lse = static_cast<float*>(r.address(8, T * d.num_heads, kFloat, &lse_rows));
    const double scale = PyFloat_AsDouble(args[9]);
    if (scale == -1.0 && PyErr_Occurred()) throw Refused{"softmax_scale is not a number"};
    void* workspace = r.address(10, 0, kBytes);
    const int64_t bytes = r.number(11, 10, true);
    auto stream = static_cast<wf_stream_t>(r.address(12, 0, kBytes));
    return without_gil([&] {
      return g_attn(&d, plan, table, prefix, q, k_pool, v_pool, out, lse, float(scale), workspace,
                    bytes < 0 ? 0 : size_t(bytes), stream);
    });
  });
}

// Addresses of the three functions in the libwf.so that wf.py has loaded.
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  if (nargs != 3) {
    PyErr_SetString(PyExc_TypeError, "3 arguments");
    return nullptr;
  }
  void* p[3];
  for (int i = 0; i < 3; ++i) {
    p[i] = PyLong_AsVoidPtr(args[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  g_tables = reinterpret_cast<decltype(g_tables)>(p[0]);
  g_append = reinterpret_cast<decltype(g_append)>(p[1]);
  g_attn = reinterpret_cast<decltype(g_attn)>(p[2]);
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyCFunction fast() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(F));
}

PyMethodDef g_methods[] = {
    {"bind", fast<bind>(), METH_FASTCALL, nullptr},
    {"tables", fast<tables>(), METH_FASTCALL, nullptr},
    {"append", fast<append>(), METH_FASTCALL, nullptr},
    {"attn", fast<attn>(), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_wf_torch", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__wf_torch() { return PyModule_Create(&g_module); }
