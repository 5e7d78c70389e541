// Native form of the decoder-layer binding (decode.py): checks the tensors of
// a call, allocates its outputs and makes the C call, in about a microsecond
// besides the launch.  A decode step makes these calls for every layer, with
// kernels of a few microseconds, so that the interpreter's part of a call
// (10 to 20 us for its dozens of attribute reads) would set their rate.
//
// Every function returns None for arguments that it does not take as they are;
// decode.py then makes the call itself, or says what is wrong with it.  The C
// entry points are handed over by address (bind), so this module does not link
// against libbq.so.
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdint>
#include <exception>

#include "bq_decode.h"

namespace {

decltype(&bq_gemm_f16xi4_group) f_gemm = nullptr;
decltype(&bq_qk_norm_rope_kv4) f_write = nullptr;
decltype(&bq_attn_kv4) f_attn = nullptr;
decltype(&bq_attn_kv4_workspace) f_workspace = nullptr;

// A CUDA tensor argument, or null.
inline const at::Tensor* tensor(PyObject* o) {
  if (!THPVariable_Check(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  return t.is_cuda() ? &t : nullptr;
}

inline bool whole(const at::Tensor* t, at::ScalarType type, int64_t dim, int dev) {
  return t && t->scalar_type() == type && t->dim() == dim && t->get_device() == dev && t->is_contiguous();
}

// Contiguous and of the given shape
template <class... S>
inline bool shaped(const at::Tensor* t, at::ScalarType type, int dev, S... want) {
  if (!whole(t, type, sizeof...(S), dev)) return false;
  const int64_t w[] = {(int64_t)want...};
  for (size_t i = 0; i < sizeof...(S); ++i)
    if (t->size(i) != w[i]) return false;
  return true;
}

// Elements from one token to the next of (tokens, heads, dims), or -1
inline int64_t row_stride(const at::Tensor& t) {
  const int64_t width = t.size(1) * t.size(2);
  if (t.is_contiguous()) return width;
  if (t.size(1) < 1 || t.stride(2) != 1 || (t.size(1) > 1 && t.stride(1) != t.size(2)) || t.size(0) < 2 ||
      t.stride(0) < width)
    return -1;
  return t.stride(0);
}

inline bool integer(PyObject* o, int64_t& v) {
  if (!PyLong_CheckExact(o)) return false;
  int over = 0;
  v = PyLong_AsLongLongAndOverflow(o, &over);
  return over == 0;
}

inline at::Tensor fresh(at::IntArrayRef shape, const at::Tensor& like, at::ScalarType type) {
  return at::detail::empty_cuda(shape, type, like.device(), std::nullopt);   // (at::empty past its dispatcher)
}

inline void* raw_stream(int dev) { return c10::cuda::getCurrentCUDAStream(dev).stream(); }

inline const uint16_t* u16(const at::Tensor* t) { return t ? static_cast<const uint16_t*>(t->data_ptr()) : nullptr; }
inline const int32_t* i32(const at::Tensor* t) { return t ? static_cast<const int32_t*>(t->data_ptr()) : nullptr; }
inline const float* f32(const at::Tensor* t) { return t ? static_cast<const float*>(t->data_ptr()) : nullptr; }

struct Pool {
  const at::Tensor *codes, *params;
  int64_t pages, heads, page, group;
};

inline bool pool(PyObject* codes, PyObject* params, int64_t D, int dev, Pool& p) {
  p.codes = tensor(codes);
  p.params = tensor(params);
  if (!whole(p.codes, at::kByte, 5, dev) || !whole(p.params, at::kHalf, 6, dev)) return false;
  p.pages = p.codes->size(0);
  p.heads = p.codes->size(2);
  p.page = p.codes->size(3);
  const int64_t groups = p.params->size(4);
  if (p.codes->size(1) != 2 || 2 * p.codes->size(4) != D || groups < 1 || D % groups != 0) return false;
  p.group = D / groups;
  return p.params->size(0) == p.pages && p.params->size(1) == 2 && p.params->size(2) == p.heads &&
         p.params->size(3) == p.page && p.params->size(5) == 2;
}

// The result of a call: its value, or its status as an integer.
inline PyObject* done(bq_status st, PyObject* value) {
  if (st == BQ_OK) return value;
  Py_XDECREF(value);
  return PyLong_FromLong(st);
}

// (as torch's own errors: memory that there is not is torch.OutOfMemoryError)
#define CATCH_ALL                                                    \
  catch (...) {                                                      \
    torch::translate_exception_to_python(std::current_exception());  \
    return nullptr;                                                  \
  }

// (X, Wp, scale, group, zero_point or None, layout, activation)
PyObject* py_gemm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  try {
    if (n != 7 || !f_gemm) Py_RETURN_NONE;
    const at::Tensor *x = tensor(a[0]), *w = tensor(a[1]), *s = tensor(a[2]);
    int64_t group, layout, act;
    if (!x || x->dim() != 2 || !integer(a[3], group) || !integer(a[5], layout) || !integer(a[6], act))
      Py_RETURN_NONE;
    const int dev = x->get_device();
    if (x->scalar_type() != at::kHalf || !x->is_contiguous() || !whole(w, at::kByte, 2, dev)) Py_RETURN_NONE;
    const int64_t M = x->size(0), K = x->size(1), N = w->size(0);
    if ((group != 32 && group != 64 && group != 128) || K % group != 0 || w->size(1) * 2 != K ||
        !shaped(s, at::kHalf, dev, N, K / group))
      Py_RETURN_NONE;
    const at::Tensor* z = nullptr;
    if (a[4] != Py_None) {
      z = tensor(a[4]);
      if (!shaped(z, at::kHalf, dev, N, K / group)) Py_RETURN_NONE;
    }
    const c10::cuda::CUDAGuard on(static_cast<c10::DeviceIndex>(dev));   // the C calls look at the current device
    at::Tensor out = fresh({M, N}, *x, at::kHalf);
    const bq_status st = f_gemm(u16(x), K, static_cast<const uint8_t*>(w->data_ptr()), (int)layout, M, N, K, (int)group,
                                u16(s), u16(z), (int)act, static_cast<uint16_t*>(out.data_ptr()), raw_stream(dev));
    return done(st, THPVariable_Wrap(std::move(out)));
  }
  CATCH_ALL
}

// (q, k, v, codes, params, slots, positions, cos, sin, q_weight, k_weight, eps, pairs, values); None where absent
PyObject* py_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
  try {
    if (n != 14 || !f_write) Py_RETURN_NONE;
    const at::Tensor *q = tensor(a[0]), *k = tensor(a[1]), *v = tensor(a[2]);
    if (!q || q->dim() != 3 || q->scalar_type() != at::kHalf) Py_RETURN_NONE;
    const int dev = q->get_device();
    const int64_t T = q->size(0), hq = q->size(1), D = q->size(2);
    Pool p;
    if (!pool(a[3], a[4], D, dev, p)) Py_RETURN_NONE;
    for (const at::Tensor* t : {k, v})
      if (!t || t->dim() != 3 || t->scalar_type() != at::kHalf || t->get_device() != dev || t->size(0) != T ||
          t->size(1) != p.heads || t->size(2) != D)
        Py_RETURN_NONE;
    const int64_t ldq = row_stride(*q), ldk = row_stride(*k), ldv = row_stride(*v);
    const at::Tensor* slots = tensor(a[5]);
    if (ldq < 0 || ldk < 0 || ldv < 0 || !shaped(slots, at::kInt, dev, T)) Py_RETURN_NONE;
    const at::Tensor *pos = nullptr, *cos = nullptr, *sin = nullptr, *qw = nullptr, *kw = nullptr;
    int64_t max_pos = 0, half = 0;
    if (a[7] != Py_None) {
      pos = tensor(a[6]);
      cos = tensor(a[7]);
      sin = tensor(a[8]);
      if (!whole(cos, at::kFloat, 2, dev) || !shaped(pos, at::kInt, dev, T)) Py_RETURN_NONE;
      max_pos = cos->size(0);
      half = cos->size(1);
      if (half == 0 || !shaped(sin, at::kFloat, dev, max_pos, half)) Py_RETURN_NONE;
    } else if (a[8] != Py_None) {
      Py_RETURN_NONE;
    }
    if (a[9] != Py_None && !shaped(qw = tensor(a[9]), at::kHalf, dev, D)) Py_RETURN_NONE;
    if (a[10] != Py_None && !shaped(kw = tensor(a[10]), at::kHalf, dev, D)) Py_RETURN_NONE;
    const double eps = PyFloat_Check(a[11]) ? PyFloat_AS_DOUBLE(a[11]) : -1.0;
    const int pairs = PyObject_IsTrue(a[12]), values = PyObject_IsTrue(a[13]);
    if (eps < 0.0 || pairs < 0 || values < 0) {
      PyErr_Clear();
      Py_RETURN_NONE;
    }
    const c10::cuda::CUDAGuard on(static_cast<c10::DeviceIndex>(dev));
    at::Tensor out = fresh({T, hq, D}, *q, at::kHalf), kval, vval;
    if (values) {
      kval = fresh({T, p.heads, D}, *q, at::kHalf);
      vval = fresh({T, p.heads, D}, *q, at::kHalf);
    }
    const bq_status st = f_write(
        u16(q), ldq, u16(k), ldk, u16(v), ldv, T, hq, p.heads, D, u16(qw), u16(kw), (float)eps, f32(cos), f32(sin),
        max_pos, 2 * half, pairs, i32(pos), i32(slots), static_cast<uint8_t*>(p.codes->data_ptr()),
        static_cast<uint16_t*>(p.params->data_ptr()), p.pages, p.page, p.group, static_cast<uint16_t*>(out.data_ptr()),
        values ? static_cast<uint16_t*>(kval.data_ptr()) : nullptr,
        values ? static_cast<uint16_t*>(vval.data_ptr()) : nullptr, raw_stream(dev));
    if (st != BQ_OK) return PyLong_FromLong(st);
    PyObject* r = PyTuple_New(3);
    if (!r) return nullptr;
    PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(std::move(out)));
    PyTuple_SET_ITEM(r, 1, values ? THPVariable_Wrap(std::move(kval)) : Py_NewRef(Py_None));
    PyTuple_SET_ITEM(r, 2, values ? THPVariable_Wrap(std::move(vval)) : Py_NewRef(Py_None));
    return r;
  }
  CATCH_ALL
}

// (q, codes, params, block_table, seq_lens, cu_q, max_q, max_len, scale, window, lse, workspace); None where absent
PyObject* py_attn(PyObject*, PyObject* const* a, Py_ssize_t n) {
  try {
    if (n != 12 || !f_attn || !f_workspace) Py_RETURN_NONE;
    const at::Tensor* q = tensor(a[0]);
    if (!q || q->dim() != 3 || q->scalar_type() != at::kHalf) Py_RETURN_NONE;
    const int dev = q->get_device();
    const int64_t T = q->size(0), hq = q->size(1), D = q->size(2);
    Pool p;
    const at::Tensor *table = tensor(a[3]), *lens = tensor(a[4]), *cu = nullptr;
    if (!pool(a[1], a[2], D, dev, p) || !whole(table, at::kInt, 2, dev)) Py_RETURN_NONE;
    const int64_t B = table->size(0), width = table->size(1);
    int64_t max_q = a[5] == Py_None || T < 1 ? 1 : T, max_len = width * p.page, window;
    if (!shaped(lens, at::kInt, dev, B) || !integer(a[9], window)) Py_RETURN_NONE;
    if (a[6] != Py_None && !integer(a[6], max_q)) Py_RETURN_NONE;
    if (a[5] != Py_None ? !shaped(cu = tensor(a[5]), at::kInt, dev, B + 1) : T != B) Py_RETURN_NONE;
    if (a[7] != Py_None && (!integer(a[7], max_len) || max_len > width * p.page)) Py_RETURN_NONE;
    double scale;
    if (a[8] == Py_None)
      scale = 1.0 / std::sqrt((double)D);
    else if (PyFloat_Check(a[8]))
      scale = PyFloat_AS_DOUBLE(a[8]);
    else
      Py_RETURN_NONE;
    const int64_t ldq = row_stride(*q);
    const int lse = PyObject_IsTrue(a[10]);
    if (ldq < 0 || lse < 0) {
      PyErr_Clear();
      Py_RETURN_NONE;
    }
    const c10::cuda::CUDAGuard on(static_cast<c10::DeviceIndex>(dev));
    at::Tensor out = fresh({T, hq, D}, *q, at::kHalf), logs, own;
    if (lse) logs = fresh({T, hq}, *q, at::kFloat);
    void* ws = nullptr;
    size_t bytes = 0;
    if (a[11] == Py_None) {
      bytes = f_workspace(B, hq, p.heads, D, max_q, max_len);
      if (bytes) {
        own = fresh({(int64_t)bytes}, *q, at::kByte);
        ws = own.data_ptr();
      }
    } else {
      const at::Tensor* w = tensor(a[11]);
      if (!whole(w, at::kByte, 1, dev)) Py_RETURN_NONE;
      ws = w->data_ptr();
      bytes = (size_t)w->numel();
    }
    const bq_status st =
        f_attn(u16(q), ldq, T, hq, p.heads, D, static_cast<const uint8_t*>(p.codes->data_ptr()), u16(p.params), p.pages,
               p.page, p.group, i32(table), width, i32(lens), i32(cu), B, max_q, max_len, (float)scale, window,
               static_cast<uint16_t*>(out.data_ptr()), lse ? static_cast<float*>(logs.data_ptr()) : nullptr, ws, bytes,
               raw_stream(dev));
    if (st != BQ_OK) return PyLong_FromLong(st);
    PyObject* r = PyTuple_New(2);
    if (!r) return nullptr;
    PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(std::move(out)));
    PyTuple_SET_ITEM(r, 1, lse ? THPVariable_Wrap(std::move(logs)) : Py_NewRef(Py_None));
    return r;
  }
  CATCH_ALL
}

// (addresses of bq_gemm_f16xi4_group, bq_qk_norm_rope_kv4, bq_attn_kv4, bq_attn_kv4_workspace)
PyObject* py_bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 4) {
    PyErr_SetString(PyExc_TypeError, "bind takes four addresses");
    return nullptr;
  }
  void* p[4];
  for (int i = 0; i < 4; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (!p[i] && PyErr_Occurred()) return nullptr;
  }
  f_gemm = reinterpret_cast<decltype(f_gemm)>(p[0]);
  f_write = reinterpret_cast<decltype(f_write)>(p[1]);
  f_attn = reinterpret_cast<decltype(f_attn)>(p[2]);
  f_workspace = reinterpret_cast<decltype(f_workspace)>(p[3]);
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"gemm", reinterpret_cast<PyCFunction>(py_gemm), METH_FASTCALL, nullptr},
    {"write", reinterpret_cast<PyCFunction>(py_write), METH_FASTCALL, nullptr},
    {"attn", reinterpret_cast<PyCFunction>(py_attn), METH_FASTCALL, nullptr},
    {"bind", reinterpret_cast<PyCFunction>(py_bind), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_decode_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__decode_binding() { return PyModule_Create(&module); }
