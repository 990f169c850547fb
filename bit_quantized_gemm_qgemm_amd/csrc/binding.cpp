// The short way into the key-value cache calls: argument checks and the call
// itself in native code, for arguments as a serving loop passes them (tensors
// of one device, outputs and workspace given).  Such a call is made for every
// layer of every step, and its checks in Python take longer than the kernels
// run.  Each function returns the call's status, or None for anything that it
// does not take; the Python function of the same name then checks the
// arguments one by one, says what is wrong or makes the call.
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>

#include "qgemm.h"

namespace {

PyObject* stream_of = nullptr;   // torch's device number -> current stream

// Conditions that the Python side spells out: thrown over, never shown.
struct NotPlain {};

void need(bool ok) {
  if (!ok) throw NotPlain{};
}

const at::Tensor& tensor(PyObject* o, int64_t ndim) {
  need(THPVariable_CheckExact(o));
  const at::Tensor& t = THPVariable_Unpack(o);
  need(t.defined() && t.layout() == at::kStrided && t.is_cuda() && t.dim() == ndim);
  return t;
}

// The last axis dense; strides of the others as stride() gives them.
const at::Tensor& view(PyObject* o, int64_t ndim) {
  const at::Tensor& t = tensor(o, ndim);
  need(t.stride(-1) == 1 || t.size(-1) <= 1);
  return t;
}

// 0 where an axis has one entry or none: torch leaves that stride arbitrary.
int64_t stride(const at::Tensor& t, int64_t axis) { return t.size(axis) > 1 ? t.stride(axis) : 0; }

void* dense(PyObject* o, at::ScalarType type, int64_t ndim, int64_t n, const at::Tensor& first) {
  const at::Tensor& t = tensor(o, ndim);
  need(t.scalar_type() == type && t.is_contiguous() && t.get_device() == first.get_device() &&
       (n < 0 || t.size(0) == n));
  return t.data_ptr();
}

int64_t integer(PyObject* o) {
  need(PyLong_CheckExact(o));
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    throw NotPlain{};
  }
  return v;
}

int half_type(const at::Tensor& t) {
  const auto s = t.scalar_type();
  need(s == at::kHalf || s == at::kBFloat16);
  return s == at::kHalf ? QGEMM_F16 : QGEMM_BF16;
}

void* stream(const at::Tensor& t) {
  PyObject* device = PyLong_FromLong(t.get_device());
  need(device != nullptr);
  PyObject* handle = PyObject_CallOneArg(stream_of, device);
  Py_DECREF(device);
  need(handle != nullptr);
  void* p = PyLong_AsVoidPtr(handle);
  Py_DECREF(handle);
  need(!PyErr_Occurred());
  return p;
}

struct Pools {
  int type;
  void *k, *v;
  const float *k_scale = nullptr, *v_scale = nullptr;
  int64_t pages, kv_heads, page_size, dim, page_stride, head_stride, token_stride;

  Pools(PyObject* k_cache, PyObject* v_cache, PyObject* ks, PyObject* vs, const at::Tensor& first,
        int first_type) {
    const at::Tensor &a = view(k_cache, 4), &b = view(v_cache, 4);
    const auto s = a.scalar_type();
    need(a.get_device() == first.get_device() && b.get_device() == first.get_device());
    need(b.scalar_type() == s && b.sizes() == a.sizes());
    pages = a.size(0), kv_heads = a.size(1), page_size = a.size(2), dim = a.size(3);
    page_stride = stride(a, 0), head_stride = stride(a, 1), token_stride = stride(a, 2);
    need(stride(b, 0) == page_stride && stride(b, 1) == head_stride && stride(b, 2) == token_stride);
    need(page_size >= 1);
    if (s == at::kFloat8_e4m3fn || s == at::kByte) {
      type = QGEMM_E4M3;
      k_scale = static_cast<const float*>(dense(ks, at::kFloat, 1, kv_heads, first));
      v_scale = static_cast<const float*>(dense(vs, at::kFloat, 1, kv_heads, first));
    } else {
      type = half_type(a);
      need(type == first_type && ks == Py_None && vs == Py_None);
    }
    k = a.data_ptr();
    v = b.data_ptr();
  }
};

template <class Call>
PyObject* status_of(Call&& call) {
  PyThreadState* state = PyEval_SaveThread();
  const int status = call();
  PyEval_RestoreThread(state);
  return PyLong_FromLong(status);
}

template <class Body>
PyObject* guarded(Body&& body) {
  try {
    return body();
  } catch (...) {   // also what a tensor method throws: the Python side meets it again
    PyErr_Clear();
    Py_RETURN_NONE;
  }
}

// (table, cached, added, free_pages, page_size, tokens, out)
PyObject* kv_plan(PyObject*, PyObject* const* arg, Py_ssize_t nargs) {
  return guarded([&]() -> PyObject* {
    need(nargs == 7 && PyTuple_CheckExact(arg[6]) && PyTuple_GET_SIZE(arg[6]) == 4);
    const at::Tensor& table = view(arg[0], 2);
    need(table.scalar_type() == at::kInt);
    const int64_t batch = table.size(0), page_size = integer(arg[4]), tokens = integer(arg[5]);
    need(page_size >= 1 && tokens >= 0);
    auto i32 = [&](PyObject* o, int64_t n) {
      return static_cast<int32_t*>(dense(o, at::kInt, 1, n, table));
    };
    const int32_t *cached = i32(arg[1], batch), *added = i32(arg[2], batch), *free = i32(arg[3], -1);
    const int64_t num_free = THPVariable_Unpack(arg[3]).size(0);
    PyObject* const* out = &PyTuple_GET_ITEM(arg[6], 0);
    int32_t *lens = i32(out[0], batch), *cu_tokens = i32(out[1], batch + 1),
            *cu_pages = i32(out[2], batch + 1);
    int64_t* slots = static_cast<int64_t*>(dense(out[3], at::kLong, 1, tokens, table));
    int32_t* entries = static_cast<int32_t*>(table.data_ptr());
    void* s = stream(table);
    return status_of([&] {
      return qgemm_kv_plan(entries, cached, added, free, lens, cu_tokens, cu_pages, slots, batch,
                           table.size(1), stride(table, 0), num_free, page_size, tokens, s);
    });
  });
}

// (k, v, slots, k_cache, v_cache, k_scale, v_scale)
PyObject* kv_append(PyObject*, PyObject* const* arg, Py_ssize_t nargs) {
  return guarded([&]() -> PyObject* {
    need(nargs == 7);
    const at::Tensor &k = view(arg[0], 3), &v = view(arg[1], 3);
    const int type = half_type(k);
    need(v.scalar_type() == k.scalar_type() && v.get_device() == k.get_device());
    const Pools p(arg[3], arg[4], arg[5], arg[6], k, type);
    const int64_t tokens = k.size(0);
    const int64_t* slots = static_cast<int64_t*>(dense(arg[2], at::kLong, 1, tokens, k));
    need(k.size(1) == p.kv_heads && k.size(2) == p.dim && v.sizes() == k.sizes());
    const void *kx = k.data_ptr(), *vx = v.data_ptr();
    void* s = stream(k);
    return status_of([&] {
      return qgemm_kv_append(type, p.type, kx, vx, slots, p.k, p.v, p.k_scale, p.v_scale, tokens,
                             p.kv_heads, p.dim, stride(k, 0), stride(k, 1), stride(v, 0),
                             stride(v, 1), p.pages, p.page_size, p.page_stride, p.head_stride,
                             p.token_stride, s);
    });
  });
}

// (q, k_cache, v_cache, table, lens, k_scale, v_scale, window, max_len, scale, out, workspace)
PyObject* paged_attention(PyObject*, PyObject* const* arg, Py_ssize_t nargs) {
  return guarded([&]() -> PyObject* {
    need(nargs == 12);
    const at::Tensor& q = view(arg[0], 3);
    const int type = half_type(q);
    const Pools p(arg[1], arg[2], arg[5], arg[6], q, type);
    const int64_t batch = q.size(0), heads = q.size(1), dim = q.size(2);
    need(dim == p.dim && p.kv_heads >= 1 && heads % p.kv_heads == 0);
    const at::Tensor& table = view(arg[3], 2);
    need(table.scalar_type() == at::kInt && table.get_device() == q.get_device() &&
         table.size(0) == batch);
    const int32_t* lens = static_cast<int32_t*>(dense(arg[4], at::kInt, 1, batch, q));
    const int64_t window = integer(arg[7]), max_len = integer(arg[8]);
    float scale = (float)(1.0 / std::sqrt((double)dim));
    if (arg[9] != Py_None) {
      need(PyFloat_CheckExact(arg[9]));
      scale = (float)PyFloat_AS_DOUBLE(arg[9]);
    }
    void* out = dense(arg[10], q.scalar_type(), 3, batch, q);
    need(THPVariable_Unpack(arg[10]).sizes() == q.sizes());
    void* workspace = dense(arg[11], at::kByte, 1, -1, q);
    const int64_t bytes = qgemm_paged_attention_workspace_bytes(batch, heads, p.kv_heads, dim,
                                                                max_len, window);
    need(bytes >= 0 && THPVariable_Unpack(arg[11]).size(0) >= bytes);
    const void* qx = q.data_ptr();
    const int32_t* entries = static_cast<int32_t*>(table.data_ptr());
    void* s = stream(q);
    return status_of([&] {
      return qgemm_paged_attention(type, p.type, qx, p.k, p.v, entries, lens, p.k_scale, p.v_scale,
                                   out, workspace, batch, heads, p.kv_heads, dim, stride(q, 0),
                                   stride(q, 1), p.pages, p.page_size, p.page_stride,
                                   p.head_stride, p.token_stride, table.size(1), stride(table, 0),
                                   max_len, window, scale, s);
    });
  });
}

PyMethodDef methods[] = {
    {"kv_plan", (PyCFunction)(void (*)())kv_plan, METH_FASTCALL, nullptr},
    {"kv_append", (PyCFunction)(void (*)())kv_append, METH_FASTCALL, nullptr},
    {"paged_attention", (PyCFunction)(void (*)())paged_attention, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
  PyObject* torch_c = PyImport_ImportModule("torch._C");
  if (!torch_c) return nullptr;
  stream_of = PyObject_GetAttrString(torch_c, "_cuda_getCurrentRawStream");
  Py_DECREF(torch_c);
  if (!stream_of) return nullptr;
  return PyModule_Create(&module);
}
