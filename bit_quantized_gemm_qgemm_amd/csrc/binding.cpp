// The short way into the calls of a serving loop, those of the key-value cache and
// of int8 and expert layers: argument checks and the call itself in native code, for
// arguments as such a loop passes them (tensors of one device, outputs and workspace
// given).  Such a call is made for every
// layer of every step, and its checks in Python take longer than the kernels
// run.  Each function returns the call's status, or None for anything that it
// does not take; the Python function of the same name then checks the
// arguments one by one, says what is wrong or makes the call.
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <utility>

#include "qgemm.h"

namespace {

PyObject* stream_of = nullptr;   // torch's device number -> current stream
PyObject* device_of = nullptr;   // torch's current device number

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

// ---- int8 x int8 products, dense and by expert ---------------------------------

// The tensor's device is the current one: the calls launch there.
void need_current(const at::Tensor& t) {
  PyObject* now = PyObject_CallNoArgs(device_of);
  need(now != nullptr);
  const long device = PyLong_AsLong(now);
  Py_DECREF(now);
  need(!PyErr_Occurred() && device == t.get_device());
}

int flag(PyObject* o) {
  need(PyBool_Check(o));
  return o == Py_True;
}

// (x, out)
PyObject* quantize_int8(PyObject*, PyObject* const* arg, Py_ssize_t nargs) {
  return guarded([&]() -> PyObject* {
    need(nargs == 2 && PyTuple_CheckExact(arg[1]) && PyTuple_GET_SIZE(arg[1]) == 2);
    const at::Tensor& x = view(arg[0], 2);
    const auto s = x.scalar_type();
    need(s == at::kHalf || s == at::kBFloat16 || s == at::kFloat);
    const int type = s == at::kHalf ? QGEMM_F16 : s == at::kBFloat16 ? QGEMM_BF16 : QGEMM_F32;
    const int64_t rows = x.size(0), K = x.size(1);
    PyObject* const* out = &PyTuple_GET_ITEM(arg[1], 0);
    int8_t* codes = static_cast<int8_t*>(dense(out[0], at::kChar, 2, rows, x));
    need(THPVariable_Unpack(out[0]).size(1) == K);
    float* scale = static_cast<float*>(dense(out[1], at::kFloat, 1, rows, x));
    need_current(x);
    const void* p = x.data_ptr();
    const int64_t step = stride(x, 0);
    void* st = stream(x);
    return status_of([&] { return qgemm_quantize_int8(type, p, codes, scale, rows, K, step, st); });
  });
}

// Operands of both products.
struct W8a8Operands {
  const int8_t* a;
  const float* a_scale;
  const void* packed;
  int64_t rows, K;

  W8a8Operands(const at::Tensor& first, PyObject* a_, PyObject* scale, PyObject* w, int64_t experts,
               int64_t N, int gated) {
    a = static_cast<const int8_t*>(dense(a_, at::kChar, 2, -1, first));
    rows = first.size(0), K = first.size(1);
    a_scale = static_cast<const float*>(dense(scale, at::kFloat, 1, rows, first));
    packed = dense(w, at::kByte, 1, -1, first);
    const int64_t bytes = qgemm_prepack_w8a8_bytes(experts, K, N, gated);
    need(bytes >= 0 && THPVariable_Unpack(w).size(0) >= bytes);
  }
};

// The output given: its type and address.
std::pair<int, void*> product_out(PyObject* o, int64_t M, int64_t cols, const at::Tensor& first) {
  const at::Tensor& t = tensor(o, 2);
  const int type = half_type(t);
  void* p = dense(o, t.scalar_type(), 2, M, first);
  need(t.size(1) == cols);
  return {type, p};
}

// (a, a_scale, w_packed, w_scale, N, gated, out)
PyObject* w8a8(PyObject*, PyObject* const* arg, Py_ssize_t nargs) {
  return guarded([&]() -> PyObject* {
    need(nargs == 7);
    const at::Tensor& a = tensor(arg[0], 2);
    const int64_t N = integer(arg[4]);
    const int gated = flag(arg[5]);
    const W8a8Operands x(a, arg[0], arg[1], arg[2], 1, N, gated);
    const float* w_scale = static_cast<const float*>(dense(arg[3], at::kFloat, 1, N, a));
    const auto out = product_out(arg[6], x.rows, gated ? N / 2 : N, a);
    need_current(a);
    void* st = stream(a);
    return status_of([&] {
      return qgemm_w8a8(out.first, x.a, x.a_scale, x.packed, w_scale, out.second, x.rows, N, x.K, gated,
                        st);
    });
  });
}

// (a, a_scale, w_packed, w_scale, offsets, N, rows, gated, out)
PyObject* w8a8_experts(PyObject*, PyObject* const* arg, Py_ssize_t nargs) {
  return guarded([&]() -> PyObject* {
    need(nargs == 9);
    const at::Tensor& a = tensor(arg[0], 2);
    const int64_t N = integer(arg[5]);
    const int gated = flag(arg[7]);
    const int32_t* offsets = static_cast<const int32_t*>(dense(arg[4], at::kInt, 1, -1, a));
    const int64_t experts = THPVariable_Unpack(arg[4]).size(0) - 1;
    need(experts >= 1);
    const W8a8Operands x(a, arg[0], arg[1], arg[2], experts, N, gated);
    const float* w_scale = static_cast<const float*>(dense(arg[3], at::kFloat, 2, experts, a));
    need(THPVariable_Unpack(arg[3]).size(1) == N);
    int64_t M = x.rows;
    const int32_t* rows = nullptr;
    if (arg[6] != Py_None) {
      rows = static_cast<const int32_t*>(dense(arg[6], at::kInt, 1, -1, a));
      M = THPVariable_Unpack(arg[6]).size(0);
    }
    const auto out = product_out(arg[8], M, gated ? N / 2 : N, a);
    need_current(a);
    void* st = stream(a);
    return status_of([&] {
      return qgemm_w8a8_experts(out.first, x.a, x.a_scale, x.packed, w_scale, offsets, rows, out.second,
                                x.rows, M, N, x.K, experts, gated, st);
    });
  });
}

// (ids, experts, out, workspace)
PyObject* expert_plan(PyObject*, PyObject* const* arg, Py_ssize_t nargs) {
  return guarded([&]() -> PyObject* {
    need(nargs == 4 && PyTuple_CheckExact(arg[2]) && PyTuple_GET_SIZE(arg[2]) == 3);
    const at::Tensor& ids = tensor(arg[0], 2);
    const auto s = ids.scalar_type();
    need((s == at::kInt || s == at::kLong) && ids.is_contiguous());
    const int64_t tokens = ids.size(0), top = ids.size(1), experts = integer(arg[1]);
    const int64_t bytes = qgemm_expert_plan_workspace_bytes(tokens * top, experts);
    need(bytes >= 0);
    PyObject* const* out = &PyTuple_GET_ITEM(arg[2], 0);
    int32_t* offsets = static_cast<int32_t*>(dense(out[0], at::kInt, 1, experts + 1, ids));
    int32_t* rows = static_cast<int32_t*>(dense(out[1], at::kInt, 1, tokens * top, ids));
    int32_t* places = static_cast<int32_t*>(dense(out[2], at::kInt, 2, tokens, ids));
    need(THPVariable_Unpack(out[2]).size(1) == top);
    void* workspace = dense(arg[3], at::kByte, 1, -1, ids);
    need(THPVariable_Unpack(arg[3]).size(0) >= bytes);
    need_current(ids);
    const void* p = ids.data_ptr();
    void* st = stream(ids);
    return status_of([&] {
      return qgemm_expert_plan(s == at::kInt ? 4 : 8, p, offsets, rows, places, workspace, tokens, top,
                               experts, st);
    });
  });
}

// (y, places, gates, out)
PyObject* expert_combine(PyObject*, PyObject* const* arg, Py_ssize_t nargs) {
  return guarded([&]() -> PyObject* {
    need(nargs == 4);
    const at::Tensor& y = tensor(arg[0], 2);
    const int type = half_type(y);
    need(y.is_contiguous());
    const int32_t* places = static_cast<const int32_t*>(dense(arg[1], at::kInt, 2, -1, y));
    const int64_t tokens = THPVariable_Unpack(arg[1]).size(0), top = THPVariable_Unpack(arg[1]).size(1);
    const float* gates = static_cast<const float*>(dense(arg[2], at::kFloat, 2, tokens, y));
    need(THPVariable_Unpack(arg[2]).size(1) == top);
    void* out = dense(arg[3], y.scalar_type(), 2, tokens, y);
    need(THPVariable_Unpack(arg[3]).size(1) == y.size(1));
    need_current(y);
    const void* p = y.data_ptr();
    const int64_t rows = y.size(0), N = y.size(1);
    void* st = stream(y);
    return status_of([&] { return qgemm_expert_combine(type, p, places, gates, out, rows, tokens, top, N, st); });
  });
}

PyMethodDef methods[] = {
    {"kv_plan", (PyCFunction)(void (*)())kv_plan, METH_FASTCALL, nullptr},
    {"kv_append", (PyCFunction)(void (*)())kv_append, METH_FASTCALL, nullptr},
    {"paged_attention", (PyCFunction)(void (*)())paged_attention, METH_FASTCALL, nullptr},
    {"quantize_int8", (PyCFunction)(void (*)())quantize_int8, METH_FASTCALL, nullptr},
    {"w8a8", (PyCFunction)(void (*)())w8a8, METH_FASTCALL, nullptr},
    {"w8a8_experts", (PyCFunction)(void (*)())w8a8_experts, METH_FASTCALL, nullptr},
    {"expert_plan", (PyCFunction)(void (*)())expert_plan, METH_FASTCALL, nullptr},
    {"expert_combine", (PyCFunction)(void (*)())expert_combine, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
  PyObject* torch_c = PyImport_ImportModule("torch._C");
  if (!torch_c) return nullptr;
  stream_of = PyObject_GetAttrString(torch_c, "_cuda_getCurrentRawStream");
  device_of = PyObject_GetAttrString(torch_c, "_cuda_getDevice");
  Py_DECREF(torch_c);
  if (!stream_of || !device_of) return nullptr;
  return PyModule_Create(&module);
}
