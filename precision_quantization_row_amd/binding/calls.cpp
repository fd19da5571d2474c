// calls.cpp -- the short way from torch tensors to the C ABI, for calls that a
// model makes for every layer and token (_calls.so).
//
// A kernel of a decode step runs 3 to 5 us; checking ten tensors in Python and
// converting two dozen arguments with ctypes takes 9 to 14. Each function here
// checks what its namesake in __init__.py checks and calls the library on the
// tensors' device and the stream given, or the device's current one. It returns
// the status, or None where anything is not as it should be: the caller then
// looks closer, in Python, and says what.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/core/DeviceGuard.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>

#include "nvfp4.h"

namespace {

enum : unsigned { BF16 = 1, F32 = 2, F8 = 4, I8 = 8, U8 = 16, I32 = 32, OUT = BF16 | F32, SCALE = U8 | F8 };

unsigned type_bit(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return BF16;
    case at::kFloat: return F32;
    case at::kFloat8_e4m3fn: return F8;
    case at::kChar: return I8;
    case at::kByte: return U8;
    case at::kInt: return I32;
    default: return 0;
  }
}
int dtype_code(unsigned bit) { return bit == BF16 ? NVFP4_BF16 : NVFP4_FP32; }

PyObject* current_stream_fn = nullptr;  // torch._C._cuda_getCurrentRawStream

// The arguments of one call. `ok` falls when one of them needs a closer look.
struct Args {
  PyObject* const* at;
  bool ok = true;
  int dev = -1;

  const at::Tensor* tensor(int i) {
    if (at[i] == Py_None) return nullptr;
    if (!THPVariable_Check(at[i])) {
      ok = false;
      return nullptr;
    }
    return &THPVariable_Unpack(at[i]);
  }
  // the tensor that decides the device and, by its dtype, those of others
  const at::Tensor* first(int i, unsigned types) {
    const at::Tensor* t = tensor(i);
    if (!t || !t->is_cuda() || !(type_bit(*t) & types)) {
      ok = false;
      return nullptr;
    }
    dev = t->get_device();
    return t;
  }
  bool here(const at::Tensor& t) const { return t.is_cuda() && t.get_device() == dev; }
  // the address of an optional contiguous tensor of n elements
  void* ptr(int i, unsigned types, int64_t n) {
    const at::Tensor* t = tensor(i);
    if (!t) return nullptr;
    if (!(type_bit(*t) & types) || !here(*t) || t->numel() != n || !t->is_contiguous()) {
      ok = false;
      return nullptr;
    }
    return t->data_ptr();
  }
  template <typename T>
  T* ptr_as(int i, unsigned types, int64_t n) {
    return static_cast<T*>(ptr(i, types, n));
  }
  unsigned bit(int i) {
    const at::Tensor* t = tensor(i);
    return t ? type_bit(*t) : 0u;
  }
  int64_t integer(int i) {
    const long long v = PyLong_Check(at[i]) ? PyLong_AsLongLong(at[i]) : -1;
    if (!PyLong_Check(at[i]) || (v == -1 && PyErr_Occurred())) {
      PyErr_Clear();
      ok = false;
      return 0;
    }
    return v;
  }
  float number(int i) {
    const double v = PyFloat_Check(at[i]) ? PyFloat_AS_DOUBLE(at[i]) : 0.0;
    if (!PyFloat_Check(at[i])) ok = false;
    return static_cast<float>(v);
  }
  int64_t times(int64_t a, int64_t b) {
    int64_t r;
    if (__builtin_mul_overflow(a, b, &r)) {
      ok = false;
      return -1;
    }
    return r;
  }
  void* stream(int i) {
    PyObject* v = nullptr;
    if (!ok) return nullptr;
    if (at[i] == Py_None) {
      PyObject* d = PyLong_FromLong(dev);
      if (d) v = PyObject_CallFunctionObjArgs(current_stream_fn, d, nullptr);
      Py_XDECREF(d);
    } else {
      v = PyObject_GetAttrString(at[i], "cuda_stream");
    }
    void* s = v ? PyLong_AsVoidPtr(v) : nullptr;
    Py_XDECREF(v);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      ok = false;
    }
    return s;
  }
  c10::Device device() const { return c10::Device(c10::DeviceType::CUDA, static_cast<c10::DeviceIndex>(dev)); }
};

// Runs `body`, which returns a status, with exactly n arguments; None where it
// could not. No C++ exception leaves.
template <typename F>
PyObject* run(PyObject* const* args, Py_ssize_t have, Py_ssize_t n, F body) {
  if (have != n) Py_RETURN_NONE;
  try {
    Args a{args};
    const int status = body(a);
    if (a.ok) return PyLong_FromLong(status);
  } catch (const std::exception&) {
  }
  if (PyErr_Occurred()) PyErr_Clear();
  Py_RETURN_NONE;
}

// x, row_amax, q, noop, stream
PyObject* int8_quantize(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return run(args, n, 5, [](Args& a) {
    const at::Tensor* x = a.first(0, OUT);
    if (!x || x->dim() != 2 || !x->is_contiguous()) return a.ok = false, 0;
    const int64_t M = x->size(0), K = x->size(1);
    float* amax = a.ptr_as<float>(1, F32, M);
    int8_t* q = a.ptr_as<int8_t>(2, I8, M * K);
    const float* noop = a.ptr_as<float>(3, F32, 1);
    void* s = a.stream(4);
    if (!a.ok) return 0;
    c10::DeviceGuard guard(a.device());
    return nvfp4_int8_quantize(x->data_ptr(), dtype_code(type_bit(*x)), M, K, amax, q, noop, s);
  });
}

// x, row_amax, col_amax, q_row, q_col, noop, stream
PyObject* int8_quantize_rowcol(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return run(args, n, 7, [](Args& a) {
    const at::Tensor* x = a.first(0, OUT);
    if (!x || x->dim() != 2 || !x->is_contiguous()) return a.ok = false, 0;
    const int64_t M = x->size(0), K = x->size(1);
    float *ra = a.ptr_as<float>(1, F32, M), *ca = a.ptr_as<float>(2, F32, K);
    int8_t *qr = a.ptr_as<int8_t>(3, I8, M * K), *qc = a.ptr_as<int8_t>(4, I8, M * K);
    const float* noop = a.ptr_as<float>(5, F32, 1);
    void* s = a.stream(6);
    if (!a.ok) return 0;
    c10::DeviceGuard guard(a.device());
    return nvfp4_int8_quantize_rowcol(x->data_ptr(), dtype_code(type_bit(*x)), M, K, ra, ca, qr, qc, noop, s);
  });
}

// a, a_mode, a_amax, b, b_mode, b_amax, M, N, K, y, bias, act, residual, z, noop, stream
PyObject* int8_gemm(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return run(args, n, 16, [](Args& a) {
    if (!a.first(0, I8)) return 0;
    const int64_t am = a.integer(1), bm = a.integer(4), M = a.integer(6), N = a.integer(7), K = a.integer(8), act = a.integer(11);
    const unsigned out = a.bit(9), bias_bit = a.bit(10);
    if (!a.ok || !(out & OUT) || act < NVFP4_ACT_NONE || act > NVFP4_ACT_SWIGLU || am < 0 || am > 2 || bm < 0 || bm > 2)
      return a.ok = false, 0;
    const int64_t NB = act == NVFP4_ACT_SWIGLU ? a.times(2, N) : N, MN = a.times(M, N);
    const auto* qa = a.ptr_as<int8_t>(0, I8, a.times(M, K));
    const auto* aa = a.ptr_as<float>(2, F32, am == NVFP4_AMAX_LINE ? M : 1);
    const auto* qb = a.ptr_as<int8_t>(3, I8, a.times(NB, K));
    const auto* ab = a.ptr_as<float>(5, F32, bm == NVFP4_AMAX_LINE ? NB : 1);
    void* y = a.ptr(9, out, MN);
    const void* bias = a.ptr(10, OUT, NB);
    const void* res = a.ptr(12, out, MN);
    void* z = a.ptr(13, out, a.times(M, NB));
    const float* noop = a.ptr_as<float>(14, F32, 1);
    void* s = a.stream(15);
    if (!a.ok) return 0;
    c10::DeviceGuard guard(a.device());
    return nvfp4_int8_gemm(qa, (int)am, aa, qb, (int)bm, ab, M, N, K, bias, bias ? dtype_code(bias_bit) : 0, (int)act, res, z, y,
                           dtype_code(out), noop, s);
  });
}

int line_format(unsigned bit) { return bit == F8 ? NVFP4_FMT_E4M3 : bit == I8 ? NVFP4_FMT_INT8 : bit == U8 ? NVFP4_FMT_NVFP4 : NVFP4_FMT_NONE; }

// x, weight, eps, bias, residual, h, y, mean, rstd, q, s, row_amax, bound, noop, stream
PyObject* layernorm(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return run(args, n, 15, [](Args& a) {
    const at::Tensor* x = a.first(0, OUT);
    if (!x || x->dim() != 2 || !x->is_contiguous()) return a.ok = false, 0;
    const int64_t M = x->size(0), K = x->size(1);
    const unsigned same = type_bit(*x), wbit = a.bit(1), ybit = a.bit(6), qbit = a.bit(9);
    const int fmt = line_format(qbit);
    if (!(wbit & OUT) || (qbit != 0) != (a.at[9] != Py_None) || (qbit && fmt == NVFP4_FMT_NONE))
      return a.ok = false, 0;
    const void* w = a.ptr(1, wbit, K);
    const float eps = a.number(2), bound = a.number(12);
    const void *b = a.ptr(3, wbit, K), *res = a.ptr(4, same, M * K);
    void *h = a.ptr(5, same, M * K), *y = a.ptr(6, OUT, M * K);
    float *mean = a.ptr_as<float>(7, F32, M), *rstd = a.ptr_as<float>(8, F32, M);
    auto* q = a.ptr_as<uint8_t>(9, F8 | I8 | U8, fmt == NVFP4_FMT_NVFP4 ? M * ((K + 1) / 2) : M * K);
    auto* sc = a.ptr_as<uint8_t>(10, SCALE, M * ((K + 15) / 16));
    float* amax = a.ptr_as<float>(11, F32, M);
    const float* noop = a.ptr_as<float>(13, F32, 1);
    void* s = a.stream(14);
    if (!a.ok) return 0;
    c10::DeviceGuard guard(a.device());
    return nvfp4_layernorm(x->data_ptr(), res, dtype_code(same), w, b, dtype_code(wbit), eps, M, K, h, y, y ? dtype_code(ybit) : 0,
                           mean, rstd, fmt, q, sc, amax, bound, noop, s);
  });
}

// dy, h, weight, mean, rstd, dx, dweight, dbias, dres, workspace, noop, stream
PyObject* layernorm_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return run(args, n, 12, [](Args& a) {
    const at::Tensor* dy = a.first(0, OUT);
    if (!dy || dy->dim() != 2 || !dy->is_contiguous()) return a.ok = false, 0;
    const int64_t M = dy->size(0), K = dy->size(1);
    const unsigned same = type_bit(*dy), wbit = a.bit(2);
    const void *h = a.ptr(1, same, M * K), *w = a.ptr(2, OUT, K);
    const float *mean = a.ptr_as<float>(3, F32, M), *rstd = a.ptr_as<float>(4, F32, M);
    void* dx = a.ptr(5, same, M * K);
    float *dw = a.ptr_as<float>(6, F32, K), *db = a.ptr_as<float>(7, F32, K);
    const void* dres = a.ptr(8, same, M * K);
    const at::Tensor* given = a.tensor(9);
    const float* noop = a.ptr_as<float>(10, F32, 1);
    void* s = a.stream(11);
    if (!a.ok || !w) return a.ok = false, 0;
    c10::DeviceGuard guard(a.device());
    at::Tensor ws;
    int64_t bytes = dw || db ? nvfp4_layernorm_backward_workspace(M, K) : 0;
    if (bytes > 0 && given) {
      if (!a.here(*given) || !given->is_contiguous() || (int64_t)given->nbytes() < bytes) return a.ok = false, 0;
      ws = *given;
    } else if (bytes > 0) {
      if (a.at[11] != Py_None) return a.ok = false, 0;  // (of that stream's pool)
      ws = at::empty({bytes}, at::TensorOptions().dtype(at::kByte).device(a.device()));
    }
    return nvfp4_layernorm_backward(dy->data_ptr(), h, dtype_code(same), w, dtype_code(wbit), mean, rstd, dres, M, K, dx, dw, db,
                                    bytes > 0 ? ws.data_ptr() : nullptr, bytes, noop, s);
  });
}

// rows [T, H, D] that may lie apart: address and elements from row to row
void* row_ptr(Args& a, int i, unsigned type, const at::Tensor& like, int64_t* stride) {
  const at::Tensor* t = a.tensor(i);
  *stride = 0;
  if (!t) return nullptr;
  const int64_t H = like.size(1), D = like.size(2);
  if (!(type_bit(*t) & type) || !a.here(*t) || t->sizes() != like.sizes() || (D > 1 && t->stride(2) != 1) ||
      (H > 1 && t->stride(1) != D)) {
    a.ok = false;
    return nullptr;
  }
  *stride = t->size(0) > 1 ? t->stride(0) : H * D;
  return t->data_ptr();
}

// k, v, k_q, k_s, k_amax, v_q, v_s, v_amax, table, starts, first, bound, noop, stream
template <bool WRITE>
PyObject* cache(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return run(args, n, 14, [](Args& a) {
    const at::Tensor* k = a.first(0, OUT);
    const at::Tensor *ka = a.tensor(4), *table = a.tensor(8);
    const int fmt = line_format(a.bit(2));
    if (!k || k->dim() != 3 || !ka || ka->dim() != 3 || !table || table->dim() != 2 || fmt == NVFP4_FMT_NONE ||
        a.at[9] == Py_None || (a.at[1] == Py_None) != (a.at[5] == Py_None) || (a.at[5] == Py_None) != (a.at[7] == Py_None) ||
        (a.at[3] != Py_None) != (fmt == NVFP4_FMT_NVFP4) ||
        (a.at[6] != Py_None) != (fmt == NVFP4_FMT_NVFP4 && a.at[5] != Py_None))
      return a.ok = false, 0;
    const int64_t T = k->size(0), H = k->size(1), D = k->size(2), B = table->size(0), cols = table->size(1);
    const int64_t pages = ka->size(0), size = ka->size(1), lines = ka->numel();
    const int64_t width = fmt == NVFP4_FMT_NVFP4 ? (D + 1) / 2 : D, blocks = (D + 15) / 16;
    if (ka->size(2) != H) return a.ok = false, 0;
    const unsigned type = type_bit(*k), qtype = a.bit(2);
    int64_t ks, vs;
    void *kp = row_ptr(a, 0, type, *k, &ks), *vp = row_ptr(a, 1, type, *k, &vs);
    void *kq = a.ptr(2, qtype, lines * width), *vq = a.ptr(5, qtype, lines * width);
    void *ksc = a.ptr(3, SCALE, lines * blocks), *vsc = a.ptr(6, SCALE, lines * blocks);
    float *kam = a.ptr_as<float>(4, F32, lines), *vam = a.ptr_as<float>(7, F32, lines);
    const auto* tb = a.ptr_as<int32_t>(8, I32, B * cols);
    const auto *st = a.ptr_as<int32_t>(9, I32, B + 1), *first = a.ptr_as<int32_t>(10, I32, B);
    const float bound = a.number(11);
    const float* noop = a.ptr_as<float>(12, F32, 1);
    void* s = a.stream(13);
    if (!a.ok) return 0;
    c10::DeviceGuard guard(a.device());
    if constexpr (WRITE)
      return nvfp4_cache_write(kp, ks, vp, vs, dtype_code(type), T, H, D, fmt, bound, pages, size, kq, ksc, kam, vq, vsc, vam, tb,
                               B, cols, st, first, noop, s);
    else
      return nvfp4_cache_read(kq, ksc, kam, vq, vsc, vam, fmt, bound, pages, size, tb, B, cols, st, first, T, H, D, kp, ks, vp, vs,
                              dtype_code(type), noop, s);
  });
}

using Fast = PyObject* (*)(PyObject*, PyObject* const*, Py_ssize_t);
PyCFunction as_method(Fast f) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)); }
PyMethodDef methods[] = {
    {"int8_quantize", as_method(int8_quantize), METH_FASTCALL, nullptr},
    {"int8_quantize_rowcol", as_method(int8_quantize_rowcol), METH_FASTCALL, nullptr},
    {"int8_gemm", as_method(int8_gemm), METH_FASTCALL, nullptr},
    {"layernorm", as_method(layernorm), METH_FASTCALL, nullptr},
    {"layernorm_backward", as_method(layernorm_backward), METH_FASTCALL, nullptr},
    {"cache_write", as_method(cache<true>), METH_FASTCALL, nullptr},
    {"cache_read", as_method(cache<false>), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() {
  PyObject* c = PyImport_ImportModule("torch._C");
  if (!c) return nullptr;
  current_stream_fn = PyObject_GetAttrString(c, "_cuda_getCurrentRawStream");
  Py_DECREF(c);
  return current_stream_fn ? PyModule_Create(&module) : nullptr;
}
