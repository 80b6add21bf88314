// Argument marshalling of the calls that a decoder makes for every token and
// layer (qk_norm_rope, paged_kv_append, paged_attention), as a CPython module: it
// reads the tensors' sizes, strides and pointers, fills the descriptors of
// include/w8lin.h and calls the library.  What it does not take as it is (an output to be
// allocated, another stream, anything that is to be refused) it leaves to the
// binding's Python, which says what is wrong.  In Python the same takes 6 to 8 us a call,
// about three times the launch: one call among others 9.2 -> 2.9 us (one token's heads, without a cache),
// 12.0 -> 3.2 (an append of eight tokens), 11.1 -> 8.6 (attention of one token).  With outputs and
// workspace to allocate the three take 15.6, 17.4 and 15.9.
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <cmath>

#include "../../include/w8lin.h"

namespace {

decltype(&::qk_norm_rope) g_rope;
decltype(&::paged_kv_append) g_append;
decltype(&::paged_attention) g_attention;
decltype(&::paged_attention_workspace) g_workspace;

// The tensors of one call: of one 16-bit type, on one device.
struct Call {
  bool ok = true;
  at::ScalarType type = at::kBFloat16;
  c10::Device device{c10::kCPU};

  const at::Tensor* tensor(PyObject* o) {
    if (!THPVariable_CheckExact(o)) {
      ok = false;
      return nullptr;
    }
    const at::Tensor* t = &THPVariable_Unpack(o);
    if (t->layout() != at::kStrided) ok = false;
    return ok ? t : nullptr;
  }
  // The first tensor, which says the type and the device.
  const at::Tensor* first(PyObject* o) {
    const at::Tensor* t = tensor(o);
    if (!t) return nullptr;
    type = t->scalar_type();
    device = t->device();
    ok = (type == at::kBFloat16 || type == at::kHalf) && device.is_cuda() && t->dim() == 3;
    return ok ? t : nullptr;
  }
  int32_t dtype() const { return type == at::kBFloat16 ? W8_DTYPE_BF16 : W8_DTYPE_F16; }

  // [M, H, D] with dense D, of `type` or, where codes are allowed, bytes.
  void* rows(PyObject* o, int64_t M, int64_t H, int64_t D, int64_t* stride, bool codes = false) {
    const at::Tensor* t = tensor(o);
    if (!t) return nullptr;
    const at::ScalarType s = t->scalar_type();
    ok = t->dim() == 3 && t->size(0) == M && t->size(1) == H && t->size(2) == D && t->device() == device &&
         (codes ? s == at::kByte || s == at::kFloat8_e4m3fn : s == type) && (t->stride(2) == 1 || D <= 1);
    if (!ok) return nullptr;
    stride[0] = t->stride(0);
    stride[1] = t->stride(1);
    return t->data_ptr();
  }
  // n dense values of a type (n < 0: any number, and how many there are); null for None.
  void* dense(PyObject* o, at::ScalarType s, int64_t n, int64_t* count = nullptr) {
    if (o == Py_None || !ok) return nullptr;
    const at::Tensor* t = tensor(o);
    if (!t) return nullptr;
    ok = t->scalar_type() == s && (n < 0 || t->numel() == n) && t->is_contiguous() && t->device() == device;
    if (count) *count = t->numel();
    return ok ? t->data_ptr() : nullptr;
  }
  void* weight(PyObject* o, int64_t D) {
    void* p = dense(o, type, D);
    if (p && THPVariable_Unpack(o).dim() != 1) ok = false;
    return p;
  }
  float number(PyObject* o) {
    if (!PyFloat_Check(o) && !PyLong_Check(o)) ok = false;
    const double v = ok ? PyFloat_AsDouble(o) : 0.0;
    if (PyErr_Occurred()) {
      PyErr_Clear();
      ok = false;
    }
    return (float)v;
  }
  // What has no truth value raises in the binding's Python.
  bool truth(PyObject* o) {
    const int v = ok ? PyObject_IsTrue(o) : 0;
    if (v < 0) {
      PyErr_Clear();
      ok = false;
    }
    return v == 1;
  }
  // The current stream of the tensors' device, which has to be the current one.
  void* stream() {
    if (c10::cuda::current_device() != device.index()) ok = false;
    return ok ? (void*)c10::cuda::getCurrentCUDAStream(device.index()).stream() : nullptr;
  }
};

// The rotation's part of the descriptor, and its pointers.
void rotation(Call& c, w8_rope_desc& d, PyObject* turns, PyObject* positions, PyObject* axes, const uint64_t** p_turns,
              const int32_t** p_pos) {
  d.axes = 1;
  if (turns == Py_None) {
    if (positions != Py_None || axes != Py_None) c.ok = false;
    return;
  }
  int64_t pairs = 0;
  *p_turns = static_cast<const uint64_t*>(c.dense(turns, at::kLong, -1, &pairs));
  if (!c.ok || THPVariable_Unpack(turns).dim() != 1) {
    c.ok = false;
    return;
  }
  d.rot = (int32_t)(2 * pairs);
  d.axis_pairs[0] = (int32_t)pairs;
  if (axes != Py_None) {
    if (!PyTuple_Check(axes) || PyTuple_GET_SIZE(axes) < 1 || PyTuple_GET_SIZE(axes) > 3) {
      c.ok = false;
      return;
    }
    d.axes = (int32_t)PyTuple_GET_SIZE(axes);
    for (int i = 0; i < d.axes; ++i) {
      const long v = PyLong_AsLong(PyTuple_GET_ITEM(axes, i));
      if (v < 0 || v > 4096) {   // an error is -1
        PyErr_Clear();
        c.ok = false;
        return;
      }
      d.axis_pairs[i] = (int32_t)v;
    }
  }
  if (positions == Py_None) return;
  const at::Tensor* t = c.tensor(positions);
  if (!t) return;
  const int64_t dim = t->dim();
  c.ok = t->scalar_type() == at::kInt && t->device() == c.device && dim >= 1 && dim <= 2 && (dim == 2 || d.axes == 1) &&
         t->size(dim - 1) == d.M && (dim == 1 || t->size(0) == d.axes) && (t->stride(dim - 1) == 1 || d.M < 2);
  if (!c.ok) return;
  d.pos_stride = dim == 2 ? t->stride(0) : 0;
  *p_pos = static_cast<const int32_t*>(t->data_ptr());
}

// The cache's descriptor, and its pointers.
void paged(Call& c, w8_paged_desc& d, PyObject* k_cache, PyObject* v_cache, PyObject* table, int64_t D, void** p_k, void** p_v,
           const int32_t** p_table) {
  const at::Tensor* k = c.tensor(k_cache);
  const at::Tensor* v = c.ok ? c.tensor(v_cache) : nullptr;
  const at::Tensor* t = c.ok ? c.tensor(table) : nullptr;
  if (!c.ok) return;
  const auto codes = [](const at::Tensor* x) { return x->scalar_type() == at::kByte || x->scalar_type() == at::kFloat8_e4m3fn; };
  const bool e4m3 = codes(k);
  c.ok = k->dim() == 4 && k->sizes() == v->sizes() && k->device() == c.device && v->device() == c.device &&
         (e4m3 ? codes(v) : k->scalar_type() == c.type && v->scalar_type() == c.type) && k->size(3) == D &&
         ((k->stride(3) == 1 && v->stride(3) == 1) || D <= 1) && t->dim() == 2 && t->scalar_type() == at::kInt &&
         t->device() == c.device && (t->stride(1) == 1 || t->size(1) <= 1);
  if (!c.ok) return;
  d.B = t->size(0);
  d.table_cols = t->size(1);
  d.table_stride = t->stride(0);
  d.pages = k->size(0);
  d.page_size = k->size(1);
  d.Hkv = k->size(2);
  d.D = D;
  for (int i = 0; i < 3; ++i) {
    d.k_stride[i] = k->stride(i);
    d.v_stride[i] = v->stride(i);
  }
  d.dtype = e4m3 ? W8_DTYPE_E4M3 : c.dtype();
  *p_k = k->data_ptr();
  *p_v = v->data_ptr();
  *p_table = static_cast<const int32_t*>(t->data_ptr());
}

// The library's call, which may wait for room in the launch queue, without the interpreter's lock.
template <typename F>
PyObject* status_of(F&& call) {
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = (int)call();
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(status);
}

PyObject* left() { return PyLong_FromLong(-1); }   // to the binding's Python

// (q, k, positions, turns, q_weight, k_weight, eps, interleaved, axes, amplitude, q_out, k_out)
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) try {
  Call c;
  w8_rope_desc d{};
  if (n != 12) return left();
  const at::Tensor* q = c.first(a[0]);
  if (!q || a[10] == Py_None || (a[1] == Py_None) != (a[11] == Py_None)) return left();
  d.M = q->size(0);
  d.Hq = q->size(1);
  d.D = q->size(2);
  const void* p_q = c.rows(a[0], d.M, d.Hq, d.D, d.q_stride);
  void* p_qo = c.ok ? c.rows(a[10], d.M, d.Hq, d.D, d.q_out_stride) : nullptr;
  const void* p_k = nullptr;
  void* p_ko = nullptr;
  if (c.ok && a[1] != Py_None) {
    const at::Tensor* k = c.tensor(a[1]);
    if (!k || k->dim() != 3) return left();
    d.Hkv = k->size(1);
    p_k = c.rows(a[1], d.M, d.Hkv, d.D, d.k_stride);
    if (c.ok) p_ko = c.rows(a[11], d.M, d.Hkv, d.D, d.k_out_stride);
  }
  const uint64_t* p_turns = nullptr;
  const int32_t* p_pos = nullptr;
  if (c.ok) rotation(c, d, a[3], a[2], a[8], &p_turns, &p_pos);
  const void *p_wq = c.weight(a[4], d.D), *p_wk = c.weight(a[5], d.D);
  if (!p_k && a[5] != Py_None) return left();
  if (c.ok && p_turns && !p_pos) return left();
  d.dtype = c.dtype();
  d.eps = c.number(a[6]);
  d.interleaved = c.truth(a[7]);
  d.amplitude = c.number(a[9]);
  void* stream = c.stream();
  if (!c.ok) return left();
  return status_of([&] { return g_rope(&d, p_q, p_k, p_pos, p_turns, p_wq, p_wk, p_qo, p_ko, stream); });
} catch (...) {
  return left();
}

// (k, v, k_cache, v_cache, page_table, q_start, kv_len, turns, q, q_weight, k_weight, eps, interleaved, positions, axes,
//  amplitude, k_scale, v_scale, q_out)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) try {
  Call c;
  w8_rope_desc d{};
  w8_paged_desc p{};
  if (n != 19) return left();
  const at::Tensor* k = c.first(a[0]);
  if (!k || (a[8] == Py_None) != (a[18] == Py_None) || (a[8] == Py_None && a[9] != Py_None)) return left();
  d.M = k->size(0);
  d.Hkv = k->size(1);
  d.D = k->size(2);
  const void* p_k = c.rows(a[0], d.M, d.Hkv, d.D, d.k_stride);
  const void* p_v = c.ok ? c.rows(a[1], d.M, d.Hkv, d.D, d.v_stride) : nullptr;
  const void* p_q = nullptr;
  void* p_qo = nullptr;
  if (c.ok && a[8] != Py_None) {
    const at::Tensor* q = c.tensor(a[8]);
    if (!q || q->dim() != 3) return left();
    d.Hq = q->size(1);
    p_q = c.rows(a[8], d.M, d.Hq, d.D, d.q_stride);
    if (c.ok) p_qo = c.rows(a[18], d.M, d.Hq, d.D, d.q_out_stride);
  }
  void *p_kc = nullptr, *p_vc = nullptr;
  const int32_t* p_table = nullptr;
  if (c.ok) paged(c, p, a[2], a[3], a[4], d.D, &p_kc, &p_vc, &p_table);
  const int32_t* p_start = static_cast<const int32_t*>(c.dense(a[5], at::kInt, p.B + 1));
  const int32_t* p_len = static_cast<const int32_t*>(c.dense(a[6], at::kInt, p.B));
  const uint64_t* p_turns = nullptr;
  const int32_t* p_pos = nullptr;
  if (c.ok) rotation(c, d, a[7], a[13], a[14], &p_turns, &p_pos);
  const void *p_wq = c.weight(a[9], d.D), *p_wk = c.weight(a[10], d.D);
  const float* p_ks = static_cast<const float*>(c.dense(a[16], at::kFloat, 1));
  const float* p_vs = static_cast<const float*>(c.dense(a[17], at::kFloat, 1));
  d.dtype = c.dtype();
  d.eps = c.number(a[11]);
  d.interleaved = c.truth(a[12]);
  d.amplitude = c.number(a[15]);
  void* stream = c.stream();
  if (!c.ok || a[6] == Py_None) return left();
  return status_of([&] { return g_append(&d, &p, p_q, p_k, p_v, p_pos, p_turns, p_wq, p_wk, p_kc, p_vc, p_table, p_start, p_len, p_ks,
                                  p_vs, p_qo, stream); });
} catch (...) {
  return left();
}

// (q, k_cache, v_cache, page_table, q_start, kv_len, max_q, causal, scale, k_scale, v_scale, s_out, out, ws)
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) try {
  Call c;
  w8_paged_attention_desc d{};
  w8_paged_desc p{};
  if (n != 14) return left();
  const at::Tensor* q = c.first(a[0]);
  if (!q || a[5] == Py_None || a[12] == Py_None) return left();
  d.T = q->size(0);
  d.Hq = q->size(1);
  const int64_t D = q->size(2);
  const void* p_q = c.rows(a[0], d.T, d.Hq, D, d.q_stride);
  void *p_kc = nullptr, *p_vc = nullptr;
  const int32_t* p_table = nullptr;
  if (c.ok) paged(c, p, a[1], a[2], a[3], D, &p_kc, &p_vc, &p_table);
  void* p_out = c.ok ? c.rows(a[12], d.T, d.Hq, D, d.o_stride, a[11] != Py_None) : nullptr;
  const int32_t* p_start = static_cast<const int32_t*>(c.dense(a[4], at::kInt, p.B + 1));
  const int32_t* p_len = static_cast<const int32_t*>(c.dense(a[5], at::kInt, p.B));
  const float* p_ks = static_cast<const float*>(c.dense(a[9], at::kFloat, 1));
  const float* p_vs = static_cast<const float*>(c.dense(a[10], at::kFloat, 1));
  const float* p_so = static_cast<const float*>(c.dense(a[11], at::kFloat, 1));
  int64_t floats = 0;
  float* p_ws = static_cast<float*>(c.dense(a[13], at::kFloat, -1, &floats));
  d.max_q = d.T > 0 ? d.T : 1;
  if (a[6] != Py_None) {
    d.max_q = PyLong_AsLongLong(a[6]);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      return left();
    }
  }
  d.dtype = c.dtype();
  d.causal = c.truth(a[7]);
  d.scale = a[8] == Py_None ? (float)std::pow((double)D, -0.5) : c.number(a[8]);
  void* stream = c.stream();
  if (!c.ok) return left();
  if (a[13] == Py_None) {
    int64_t need = 0;
    if (g_workspace(&d, &p, &need) != W8_OK || need > 0) return left();
  }
  return status_of([&] { return g_attention(&d, &p, p_q, p_kc, p_vc, p_table, p_start, p_len, p_ks, p_vs, p_so, p_out, p_ws, floats,
                                     stream); });
} catch (...) {
  return left();
}

// The library's four entries, as addresses.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 4) return left();
  void* p[4];
  for (int i = 0; i < 4; ++i) p[i] = PyLong_AsVoidPtr(a[i]);
  if (PyErr_Occurred()) return nullptr;
  g_rope = reinterpret_cast<decltype(g_rope)>(p[0]);
  g_append = reinterpret_cast<decltype(g_append)>(p[1]);
  g_attention = reinterpret_cast<decltype(g_attention)>(p[2]);
  g_workspace = reinterpret_cast<decltype(g_workspace)>(p[3]);
  return PyLong_FromLong(0);
}

template <PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)>
PyCFunction fast() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef g_methods[] = {{"bind", fast<bind>(), METH_FASTCALL, nullptr},
                           {"rope", fast<rope>(), METH_FASTCALL, nullptr},
                           {"append", fast<append>(), METH_FASTCALL, nullptr},
                           {"attention", fast<attention>(), METH_FASTCALL, nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// The module reads tensors as they are laid out in the PyTorch, and calls the interpreter of the Python, that
// it was compiled with: `built_for` names them, and the binding takes it with no others.
PyMODINIT_FUNC PyInit__marshal(void) {
  PyObject* m = PyModule_Create(&g_module);
  if (m && PyModule_AddStringConstant(m, "built_for", W8_BUILT_FOR) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
