// marshal.cpp -- Python module _marshal: argument checks and marshalling of the operators around the
// block, from torch tensors straight to the C ABI (include/hs2.h).
//
// These calls are made for single tokens too, where the kernels take 2 to 5 us: reading five or six
// tensors' types, shapes, strides and devices through Python takes as long again (calls in a loop on a
// B200: norm of 8 x 4096 9.1 us that way, 3.9 this way; product of 1 x 256 x 4096 9.1 and 5.0).
// Nothing is computed here and nothing kept. Each function returns the hs2_status of its call; wrong
// types raise TypeError, wrong shapes, strides and devices ValueError.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/TensorBase.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <string>

#include "hs2.h"

namespace {

using Types = std::initializer_list<at::ScalarType>;
const Types kBf16 = {at::kBFloat16};
const Types kF32 = {at::kFloat};
const Types kWide = {at::kBFloat16, at::kFloat};
const Types kCodes = {at::kFloat8_e4m3fn, at::kByte};

// a failed check: the Python exception is set
struct Refused {};

std::string list(at::IntArrayRef v) {
  std::string s = "[";
  for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + std::to_string(v[i]);
  return s + "]";
}

[[noreturn]] void refuse(PyObject *kind, const std::string &what) {
  PyErr_SetString(kind, what.c_str());
  throw Refused();
}

const at::TensorBase &tensor(const char *name, PyObject *o) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

void on_device(const char *name, const at::TensorBase &t, int device) {
  if (t.get_device() == device) return;
  refuse(PyExc_ValueError, std::string(name) + " is on " + t.device().str() + ", the current device is cuda:" +
                               std::to_string(device));
}

void of_type(const char *name, const at::TensorBase &t, Types types) {
  for (at::ScalarType s : types)
    if (t.scalar_type() == s) return;
  refuse(PyExc_TypeError, std::string(name) + ": dtype " + c10::toString(t.scalar_type()));
}

void of_shape(const char *name, const at::TensorBase &t, at::IntArrayRef shape) {
  if (t.sizes() != shape)
    refuse(PyExc_ValueError, std::string(name) + " must be " + list(shape) + ", not " + list(t.sizes()));
}

struct Matrix {
  void *p = nullptr;
  int64_t rows = 0, cols = 0, ld = 0;
  int32_t type = HS2_OUT_BF16;   // hs2_out_dtype of a wide type
};

// a 2-D tensor with unit column stride; a single row's stride is its length rounded up to `pad`
Matrix matrix(const char *name, PyObject *o, Types types, int device, int64_t pad = 16) {
  const at::TensorBase &t = tensor(name, o);
  of_type(name, t, types);
  if (t.dim() != 2) refuse(PyExc_ValueError, std::string(name) + " must be 2-D, not " + list(t.sizes()));
  if (t.stride(1) != 1 && t.size(1) > 1) refuse(PyExc_ValueError, std::string(name) + " must have contiguous rows");
  on_device(name, t, device);
  Matrix m;
  m.p = t.mutable_data_ptr();
  m.rows = t.size(0);
  m.cols = t.size(1);
  m.ld = m.rows > 1 ? t.stride(0) : (m.cols + pad - 1) / pad * pad;
  m.type = t.scalar_type() == at::kFloat ? HS2_OUT_F32 : HS2_OUT_BF16;
  return m;
}

Matrix matrix(const char *name, PyObject *o, Types types, int64_t rows, int64_t cols, int device, int64_t pad = 16) {
  const at::TensorBase &t = tensor(name, o);
  of_type(name, t, types);
  of_shape(name, t, {rows, cols});
  return matrix(name, o, types, device, pad);
}

// a contiguous tensor of this shape
void *dense(const char *name, PyObject *o, Types types, at::IntArrayRef shape, int device) {
  const at::TensorBase &t = tensor(name, o);
  of_type(name, t, types);
  of_shape(name, t, shape);
  if (!t.is_contiguous()) refuse(PyExc_ValueError, std::string(name) + " must be contiguous");
  on_device(name, t, device);
  return t.mutable_data_ptr();
}

// device memory of any type: address and bytes
void *buffer(const char *name, PyObject *o, int device, size_t *bytes) {
  const at::TensorBase &t = tensor(name, o);
  on_device(name, t, device);
  if (!t.is_non_overlapping_and_dense()) refuse(PyExc_ValueError, std::string(name) + " must be one piece of memory");
  *bytes = t.nbytes();
  return t.mutable_data_ptr();
}

int64_t integer(PyObject *o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused();
  return v;
}

int32_t integer32(const char *name, PyObject *o) {
  const int64_t v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) refuse(PyExc_ValueError, std::string(name) + " out of range");
  return (int32_t)v;
}

float real(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused();
  return (float)v;
}

void *address(PyObject *o) {
  void *p = PyLong_AsVoidPtr(o);
  if (!p && PyErr_Occurred()) throw Refused();
  return p;
}

bool given(PyObject *o) { return o != Py_None; }

// other Python threads run while this lives: a launch waits when the stream's queue is full
struct Unlocked {
  PyThreadState *state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};

// runs `call` with the number of arguments checked, every C++ exception turned into a Python one
template <class F>
PyObject *guarded(Py_ssize_t n, Py_ssize_t want, F call) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments expected, not %zd", want, n);
    return nullptr;
  }
  try {
    return PyLong_FromLong((long)call());
  } catch (const Refused &) {
    return nullptr;
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// x, weight, eps, residual, residual_out, out, codes, scales, device, stream
PyObject *rms_norm(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 10, [&] {
    const int device = integer32("device", a[8]);
    const Matrix x = matrix("x", a[0], kBf16, device);
    const int64_t d = x.cols;
    const at::TensorBase &w = tensor("weight", a[1]);
    void *wp = dense("weight", a[1], kWide, {d}, device);
    Matrix res, res_out, out, codes, scales;
    if (given(a[3]) != given(a[4])) refuse(PyExc_ValueError, "residual and residual_out: both or neither");
    if (given(a[3])) {
      res = matrix("residual", a[3], kWide, x.rows, d, device);
      res_out = matrix("residual_out", a[4], {tensor("residual", a[3]).scalar_type()}, x.rows, d, device);
      if (res.ld != res_out.ld) refuse(PyExc_ValueError, "residual and residual_out must have one row stride");
    }
    if (given(a[5])) out = matrix("out", a[5], kWide, x.rows, d, device);
    if (given(a[6]) != given(a[7])) refuse(PyExc_ValueError, "codes and scales: both or neither");
    if (given(a[6])) {
      codes = matrix("codes", a[6], kCodes, x.rows, d, device);
      scales = matrix("scales", a[7], kF32, (d + 127) / 128, x.rows, device, 4);
    }
    if (d > INT32_MAX) refuse(PyExc_ValueError, "x has too many columns");
    const float eps = real(a[2]);
    void *stream = address(a[9]);
    Unlocked unlocked;
    return hs2_rms_norm(x.rows, (int32_t)d, x.p, x.ld, res.p, res_out.p, res.type, res.ld, wp,
                        w.scalar_type() == at::kFloat ? HS2_OUT_F32 : HS2_OUT_BF16, eps, out.p, out.type, out.ld,
                        codes.p, codes.ld, static_cast<float *>(scales.p), scales.ld, stream);
  });
}

// x, codes, scales, block_rows, device, stream
PyObject *fp8_quantize(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 6, [&] {
    const int device = integer32("device", a[4]);
    const int32_t block_rows = integer32("block_rows", a[3]);
    const Matrix x = matrix("x", a[0], kBf16, device);
    const Matrix codes = matrix("codes", a[1], kCodes, x.rows, x.cols, device);
    const int64_t br = block_rows > 0 ? block_rows : 1;
    const Matrix scales = matrix("scales", a[2], kF32, (x.cols + 127) / 128, (x.rows + br - 1) / br, device, 4);
    if (x.cols > INT32_MAX) refuse(PyExc_ValueError, "x has too many columns");
    void *stream = address(a[5]);
    Unlocked unlocked;
    return hs2_fp8_quantize(x.rows, (int32_t)x.cols, x.p, x.ld, block_rows, codes.p, codes.ld,
                            static_cast<float *>(scales.p), scales.ld, stream);
  });
}

// a, a_scale, w, w_scale, out, workspace, device, stream
PyObject *gemm_fp8(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 8, [&] {
    const int device = integer32("device", a[6]);
    const Matrix x = matrix("a", a[0], kCodes, device);
    const Matrix w = matrix("w", a[2], kCodes, device);
    if (w.cols != x.cols) refuse(PyExc_ValueError, "a and w must have the same number of columns");
    const int64_t kb = (x.cols + 127) / 128;
    const Matrix sa = matrix("a_scale", a[1], kF32, kb, x.rows, device, 4);
    const Matrix sw = matrix("w_scale", a[3], kF32, kb, (w.rows + 127) / 128, device, 4);
    const Matrix out = matrix("out", a[4], kWide, x.rows, w.rows, device, 1);
    size_t bytes = 0;
    void *ws = buffer("workspace", a[5], device, &bytes);
    if (x.cols > INT32_MAX || w.rows > INT32_MAX) refuse(PyExc_ValueError, "too many rows or columns");
    void *stream = address(a[7]);
    Unlocked unlocked;
    return hs2_gemm_fp8(x.rows, (int32_t)w.rows, (int32_t)x.cols, x.p, x.ld, static_cast<const float *>(sa.p), sa.ld, w.p,
                        w.ld, static_cast<const float *>(sw.p), sw.ld, out.p, out.type, out.ld, ws, bytes, stream);
  });
}

// view address, k, v, prefix_start, prefix_len, q, scale, out, lse, workspace, device, stream
PyObject *prefix_attn(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 12, [&] {
    const int device = integer32("device", a[10]);
    const hs2_kv_view *kv = static_cast<const hs2_kv_view *>(address(a[0]));
    on_device("k", tensor("k", a[1]), device);
    on_device("v", tensor("v", a[2]), device);
    const int64_t rows[4] = {kv->batch, kv->n_q, kv->n_heads, HS2_HEAD_DIM};
    void *q = dense("q", a[5], kBf16, at::IntArrayRef(rows, 4), device);
    void *out = dense("out", a[7], kWide, at::IntArrayRef(rows, 4), device);
    void *lse = given(a[8]) ? dense("lse", a[8], kF32, at::IntArrayRef(rows, 3), device) : nullptr;
    size_t bytes = 0;
    void *ws = buffer("workspace", a[9], device, &bytes);
    const int64_t start = integer(a[3]);
    const int32_t len = integer32("prefix_len", a[4]);
    const int32_t type = tensor("out", a[7]).scalar_type() == at::kFloat ? HS2_OUT_F32 : HS2_OUT_BF16;
    const float scale = real(a[6]);
    void *stream = address(a[11]);
    Unlocked unlocked;
    return hs2_prefix_attn(kv, start, len, q, scale, out, type, static_cast<float *>(lse), ws, bytes, stream);
  });
}

PyMethodDef methods[] = {
    {"rms_norm", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rms_norm)), METH_FASTCALL, "hs2_rms_norm"},
    {"fp8_quantize", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(fp8_quantize)), METH_FASTCALL, "hs2_fp8_quantize"},
    {"gemm_fp8", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(gemm_fp8)), METH_FASTCALL, "hs2_gemm_fp8"},
    {"prefix_attn", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(prefix_attn)), METH_FASTCALL, "hs2_prefix_attn"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", "The operators' calls from torch tensors.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
