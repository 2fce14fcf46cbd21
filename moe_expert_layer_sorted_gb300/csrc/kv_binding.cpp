// Python binding of the key/value cache's calls (see KVCache in kv.py): checks
// the tensors and passes their addresses to the C ABI.  A decode step's calls
// are a few microseconds of GPU work each, and asking tensors for their types,
// shapes and strides from Python costs as much again per call.  One row written
// and read back, called from Python among other work: 22.8 us a pass, 33.9 with
// the same checks in Python; pages chosen and attended to at 6,000 tokens: 27.0, 42.7.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <string>

#include "moe.h"

namespace {

PyObject* g_error = nullptr;  // MoeError(status, text)

struct Failed {};  // a Python exception is set
struct Bad {
  std::string text;
};

[[noreturn]] void raise(int status, const char* text) {
  PyObject* e = PyObject_CallFunction(g_error, "is", status, text);
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Failed();
}
void check(bool ok, const char* text) {
  if (!ok) throw Bad{text};
}

struct Cache {
  PyObject_HEAD moe_kv_cache* h;
  int device;
  int running;  // calls inside the library (counted under the interpreter's lock)
  at::ScalarType type;
  int64_t kv_heads, head_dim;
};

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) throw Bad{std::string(name) + ": a tensor is wanted"};
  return THPVariable_Unpack(o);
}
int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Failed();
  return v;
}
int small(PyObject* o, const char* name) {
  const int64_t v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) throw Bad{std::string(name) + " is out of range"};
  return (int)v;
}
// None (the current stream), an address, or a stream object.
void* stream_of(const Cache* c, PyObject* o) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)c->device).stream();
  PyObject* address = PyLong_Check(o) ? Py_NewRef(o) : PyObject_GetAttrString(o, "cuda_stream");
  if (!address) throw Failed();
  void* p = PyLong_AsVoidPtr(address);
  Py_DECREF(address);
  if (!p && PyErr_Occurred()) throw Failed();
  return p;
}

const int32_t* indices(const Cache* c, PyObject* o, const char* name, int dim, const at::Tensor** out) {
  const at::Tensor& t = tensor(o, name);
  if (!(t.is_cuda() && t.get_device() == c->device && t.scalar_type() == at::kInt && t.dim() == dim))
    throw Bad{std::string(name) + ": int32 tensor of " + std::to_string(dim) + " axes on the cache's device"};
  if (t.size(dim - 1) > 1 && t.stride(dim - 1) != 1) throw Bad{std::string(name) + ": its last axis must be contiguous"};
  if (out) *out = &t;
  return static_cast<const int32_t*>(t.const_data_ptr());
}

// shape: that of the call's row tensors
moe_kv_batch batch_of(const Cache* c, at::IntArrayRef shape, PyObject* table_o, PyObject* lens_o, PyObject* starts_o,
                      PyObject* max_new_o) {
  moe_kv_batch b{};
  b.struct_size = sizeof b;
  const at::Tensor *table, *lens, *starts;
  b.table = indices(c, table_o, "table", 2, &table);
  b.lens = indices(c, lens_o, "lens", 1, &lens);
  const int64_t n = lens->size(0), cols = table->size(1);
  check(table->size(0) == n, "table and lens name different numbers of sequences");
  int64_t max_new;
  if (starts_o == Py_None) {
    check(shape.size() == 4 && shape[0] == n, "row tensors without starts: [sequences, rows, heads, head_dim]");
    max_new = shape[1];
    check(max_new_o == Py_None || integer(max_new_o) == max_new, "max_new belongs to starts");
    b.rows = n * max_new;
  } else {
    check(shape.size() == 3, "row tensors with starts: [rows, heads, head_dim]");
    b.starts = indices(c, starts_o, "starts", 1, &starts);
    check(starts->size(0) == n + 1, "starts: one entry more than sequences");
    b.rows = shape[0];
    max_new = max_new_o == Py_None ? b.rows : integer(max_new_o);
  }
  check(max_new >= 0 && max_new <= INT32_MAX && n <= INT32_MAX && cols <= INT32_MAX,
        "max_new, the sequences or the table's pages are out of range");
  b.batch = (int32_t)n;
  b.max_new = (int32_t)max_new;
  b.table_pages = (int32_t)cols;
  b.table_stride = n > 1 ? table->stride(0) : cols;
  return b;
}

moe_kv_tensor rows_of(const Cache* c, const at::Tensor& t, const char* name, at::IntArrayRef shape, bool written) {
  if (!(t.is_cuda() && t.get_device() == c->device && t.scalar_type() == c->type && t.sizes() == shape))
    throw Bad{std::string(name) + ": the cache's type and device, and the shape of the call's other row tensor"};
  const int64_t n = t.dim();
  check(t.stride(n - 1) == 1, "the channels of a row tensor must be contiguous");
  for (int64_t i = 0; written && i < n; ++i)
    check(t.size(i) < 2 || t.stride(i) != 0, "an expanded tensor cannot be written to");
  auto stride = [&](int64_t i) { return t.size(i) > 1 ? t.stride(i) : 0; };  // of an axis that is more than one long
  moe_kv_tensor x;
  x.data = const_cast<void*>(t.const_data_ptr());
  x.head_stride = stride(n - 2);
  x.row_stride = stride(n - 3);
  x.batch_stride = n == 4 ? stride(0) : 0;
  return x;
}
// The first row tensor of a call gives its shape.
const at::Tensor& leading(const Cache* c, PyObject* o, const char* name, bool kv) {
  const at::Tensor& t = tensor(o, name);
  const int64_t n = t.dim();
  if (!((n == 3 || n == 4) && t.size(n - 1) == c->head_dim && (!kv || t.size(n - 2) == c->kv_heads)))
    throw Bad{std::string(name) + ": [..., heads, head_dim] with 3 or 4 axes, the cache's head_dim" +
              (kv ? " and kv_heads" : "")};
  return t;
}
int32_t* choice_of(const Cache* c, PyObject* o, int64_t rows, int* budget) {
  const at::Tensor& t = tensor(o, "pages");
  const int64_t n = t.dim();
  check(t.is_cuda() && t.get_device() == c->device && t.scalar_type() == at::kInt && t.is_contiguous() && n >= 3 &&
            t.size(n - 2) == c->kv_heads && t.size(n - 1) <= INT32_MAX && t.numel() == rows * c->kv_heads * t.size(n - 1),
        "pages: contiguous int32 [rows, kv_heads, budget]");
  *budget = (int)t.size(n - 1);
  return static_cast<int32_t*>(const_cast<void*>(t.const_data_ptr()));
}

constexpr char kInUse[] = "the cache is in use by another thread";

// Runs f, a call of the C ABI, without the interpreter's lock: a launch can wait
// for room in the stream's queue.
template <typename F>
void run(Cache* c, F&& f) {
  ++c->running;
  PyThreadState* state = PyEval_SaveThread();
  const moe_status rc = f();
  PyEval_RestoreThread(state);
  --c->running;
  if (rc == MOE_OK) return;
  // a busy handle's text is the running call's
  raise(rc, rc == MOE_ERR_STATE ? kInUse : moe_kv_last_error(c->h));
}

// Runs a call's body; what it throws becomes a Python exception.
template <typename F>
PyObject* call(PyObject* self, Py_ssize_t given, Py_ssize_t wanted, F&& f) {
  try {
    if (given != wanted) {
      PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
      return nullptr;
    }
    Cache* c = reinterpret_cast<Cache*>(self);
    check(c->h != nullptr, "the cache is closed");
    f(c);
    Py_RETURN_NONE;
  } catch (const Failed&) {
  } catch (const Bad& e) {
    try {
      raise(MOE_ERR_INVALID, e.text.c_str());
    } catch (const Failed&) {
    }
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// append / read (k, v, table, lens, starts, max_new, layer, stream)
template <bool Write>
PyObject* rows_call(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  return call(self, n, 8, [&](Cache* c) {
    const at::Tensor &k = leading(c, a[0], "k", true), &v = tensor(a[1], "v");
    const moe_kv_batch b = batch_of(c, k.sizes(), a[2], a[3], a[4], a[5]);
    const moe_kv_tensor kt = rows_of(c, k, "k", k.sizes(), !Write), vt = rows_of(c, v, "v", k.sizes(), !Write);
    const int layer = small(a[6], "layer");
    void* s = stream_of(c, a[7]);
    run(c, [&, h = c->h] { return Write ? moe_kv_append(h, layer, &b, &kt, &vt, s) : moe_kv_read(h, layer, &b, &kt, &vt, s); });
  });
}

// attention (q, out, table, lens, starts, max_new, layer, stream, scale, causal, lse, pages)
PyObject* attention(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  return call(self, n, 12, [&](Cache* c) {
    const at::Tensor &q = leading(c, a[0], "q", false), &out = tensor(a[1], "out");
    const moe_kv_batch b = batch_of(c, q.sizes(), a[2], a[3], a[4], a[5]);
    const moe_kv_tensor qt = rows_of(c, q, "q", q.sizes(), false), ot = rows_of(c, out, "out", q.sizes(), true);
    const int64_t heads = q.size(q.dim() - 2);
    check(heads <= INT32_MAX, "too many heads");
    const double scale = a[8] == Py_None ? 1.0 / std::sqrt((double)c->head_dim) : PyFloat_AsDouble(a[8]);
    if (PyErr_Occurred()) throw Failed();
    const int causal = PyObject_IsTrue(a[9]);
    if (causal < 0) throw Failed();
    float* lse = nullptr;
    if (a[10] != Py_None) {
      const at::Tensor& t = tensor(a[10], "lse");
      check(t.is_cuda() && t.get_device() == c->device && t.scalar_type() == at::kFloat && t.is_contiguous() &&
                t.numel() == b.rows * heads,
            "lse: contiguous float32, one value per row and query head");
      lse = static_cast<float*>(const_cast<void*>(t.const_data_ptr()));
    }
    int budget = 0;
    const int32_t* pages = a[11] == Py_None ? nullptr : choice_of(c, a[11], b.rows, &budget);
    const int layer = small(a[6], "layer");
    void* s = stream_of(c, a[7]);
    run(c, [&, h = c->h] {
      return moe_kv_attention(h, layer, &b, &qt, (int)heads, (float)scale, causal, &ot, lse, pages, budget, s);
    });
  });
}

// select (q, pages, table, lens, starts, max_new, layer, stream, keep_first, keep_last)
PyObject* select(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  return call(self, n, 10, [&](Cache* c) {
    const at::Tensor& q = leading(c, a[0], "q", false);
    const moe_kv_batch b = batch_of(c, q.sizes(), a[2], a[3], a[4], a[5]);
    const moe_kv_tensor qt = rows_of(c, q, "q", q.sizes(), false);
    const int64_t heads = q.size(q.dim() - 2);
    check(heads <= INT32_MAX, "too many heads");
    int budget = 0;
    int32_t* pages = choice_of(c, a[1], b.rows, &budget);
    const int layer = small(a[6], "layer"), first = small(a[8], "keep_first"), last = small(a[9], "keep_last");
    void* s = stream_of(c, a[7]);
    run(c, [&, h = c->h] { return moe_kv_select(h, layer, &b, &qt, (int)heads, budget, first, last, pages, s); });
  });
}

PyObject* status(PyObject* self, PyObject*) {
  return call(self, 0, 0, [&](Cache* c) { run(c, [h = c->h] { return moe_kv_status(h); }); });
}
PyObject* fail_next(PyObject* self, PyObject*) {
  return call(self, 0, 0, [&](Cache* c) { run(c, [h = c->h] { return moe_kv_debug_fail_next_attention(h); }); });
}

// Destroys the handle; not while a call is inside the library (which may not have reached the
// handle's own guard yet): the cache then stays as it is.
PyObject* close(PyObject* self, PyObject*) {
  if (!reinterpret_cast<Cache*>(self)->h) Py_RETURN_NONE;
  return call(self, 0, 0, [&](Cache* c) {
    if (c->running) raise(MOE_ERR_STATE, kInUse);
    moe_kv_cache* h = c->h;
    c->h = nullptr;  // no call begins from here on
    PyThreadState* state = PyEval_SaveThread();
    const moe_status rc = moe_kv_destroy(h);
    PyEval_RestoreThread(state);
    if (rc == MOE_ERR_STATE) c->h = h;  // in use through the C ABI
    if (rc != MOE_OK) raise(rc, rc == MOE_ERR_STATE ? kInUse : moe_kv_last_error(nullptr));
  });
}

// Cache(MoeError, handle, device, bfloat16, kv_heads, head_dim)
int cache_init(PyObject* self, PyObject* args, PyObject*) {
  PyObject *error, *handle;
  int device, bf16;
  long long kv_heads, head_dim;
  if (!PyArg_ParseTuple(args, "OOipLL", &error, &handle, &device, &bf16, &kv_heads, &head_dim)) return -1;
  void* h = PyLong_AsVoidPtr(handle);
  if (!h) return -1;
  Py_INCREF(error);
  Py_XSETREF(g_error, error);
  Cache* c = reinterpret_cast<Cache*>(self);
  c->h = static_cast<moe_kv_cache*>(h);
  c->device = device;
  c->running = 0;
  c->type = bf16 ? at::kBFloat16 : at::kHalf;
  c->kv_heads = kv_heads;
  c->head_dim = head_dim;
  return 0;
}

// A function of METH_FASTCALL's signature as the table holds it.
template <typename F>
PyCFunction fast(F* f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef cache_methods[] = {
    {"append", fast(&rows_call<true>), METH_FASTCALL, nullptr},
    {"read", fast(&rows_call<false>), METH_FASTCALL, nullptr},
    {"attention", fast(&attention), METH_FASTCALL, nullptr},
    {"select", fast(&select), METH_FASTCALL, nullptr},
    {"check", status, METH_NOARGS, nullptr},
    {"debug_fail_next_attention", fail_next, METH_NOARGS, nullptr},
    {"close", close, METH_NOARGS, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyType_Slot cache_slots[] = {{Py_tp_init, reinterpret_cast<void*>(&cache_init)},
                             {Py_tp_new, reinterpret_cast<void*>(&PyType_GenericNew)},
                             {Py_tp_methods, cache_methods},
                             {0, nullptr}};
PyType_Spec cache_spec = {"moe_expert_layer_sorted_gb300._kv_binding.Cache", sizeof(Cache), 0, Py_TPFLAGS_DEFAULT, cache_slots};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kv_binding", nullptr, -1, nullptr, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kv_binding() {
  PyObject* m = PyModule_Create(&module);
  if (!m) return nullptr;
  PyObject* type = PyType_FromSpec(&cache_spec);
  if (!type || PyModule_AddObject(m, "Cache", type) < 0) {
    Py_XDECREF(type);
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
