// The short way from a Python call to the C ABI, for the operators whose calls last a few microseconds on
// the device (norm, MXFP4): checks, output allocation and the call in one step of native code.
//
// Each function takes the usual case only: tensors on the current device with unit stride along their rows,
// outputs allocated, work on the current stream.  For anything else, a refused argument among it, it
// returns None before anything is enqueued, and the binding's own checks take the call and say what is
// wrong.  A launch that failed is raised as AwqError: some of the call's work may be enqueued.  No exception
// passes: what torch throws (memory) is handed to Python.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "awq_serve.h"

namespace {

using at::Tensor;

// The device of the call, its current stream; what a call allocates.
struct Place {
  int dev = c10::hip::current_device();
  c10::Device device{c10::kCUDA, (c10::DeviceIndex)dev};
  void* stream() const { return (void*)c10::hip::getCurrentHIPStream((c10::DeviceIndex)dev).stream(); }
  Tensor empty(at::IntArrayRef size, at::ScalarType type) const {
    return at::detail::empty_cuda(size, type, device, std::nullopt);
  }
};

int type_of(at::ScalarType t) { return t == at::kHalf ? AWQ_FP16 : t == at::kBFloat16 ? AWQ_BF16 : -1; }

// Whether an argument is a tensor of a GPU: looked at before the current device, which there is none of on
// a machine without one.
bool on_gpu(PyObject* o) { return THPVariable_Check(o) && THPVariable_Unpack(o).is_cuda(); }

// The tensor that a Python object is, or NULL; it has to be on the call's device.
const Tensor* tensor(PyObject* o, const Place& p) {
  if (!THPVariable_Check(o)) return nullptr;
  const Tensor& t = THPVariable_Unpack(o);
  return t.defined() && t.is_cuda() && t.get_device() == p.dev && t.layout() == at::kStrided ? &t : nullptr;
}

// The same of a matrix with rows and columns; ld receives its row stride.
const Tensor* matrix(PyObject* o, const Place& p, int64_t* ld) {
  const Tensor* t = tensor(o, p);
  if (!t || t->dim() != 2 || t->size(0) == 0 || t->size(1) == 0) return nullptr;
  if (t->size(1) > 1 && t->stride(1) != 1) return nullptr;
  *ld = t->size(0) > 1 ? t->stride(0) : t->size(1);
  return *ld >= t->size(1) ? t : nullptr;
}

// The address of a contiguous vector of n elements (NULL for None, with ok kept).
const void* vector(PyObject* o, const Place& p, at::ScalarType type, int64_t n, bool* ok) {
  if (o == Py_None) return nullptr;
  const Tensor* t = tensor(o, p);
  if (!t || t->scalar_type() != type || t->dim() != 1 || t->size(0) != n || !t->is_contiguous()) {
    *ok = false;
    return nullptr;
  }
  return t->const_data_ptr();
}

int64_t round16(int64_t k) { return (k + 15) / 16 * 16; }
int64_t code_bytes(int64_t k) { return (k + 31) / 32 * 16; }
int64_t words(int64_t k) { return (k + 127) / 128; }
int64_t round4(int64_t r) { return (r + 3) / 4 * 4; }

PyObject* none() { Py_RETURN_NONE; }

// What a call that was not carried out returns: None where its arguments were refused.
PyObject* failed(int status, const char* where) {
  if (status != AWQ_E_HIP) return none();
  PyObject* m = PyImport_ImportModule("weight_only_quantization_act_amd._lib");
  PyObject* type = m ? PyObject_GetAttrString(m, "AwqError") : nullptr;
  PyObject* e = type ? PyObject_CallFunction(type, "is", status, where) : nullptr;
  if (e) PyErr_SetObject(type, e);
  Py_XDECREF(e);
  Py_XDECREF(type);
  Py_XDECREF(m);
  return nullptr;
}

// The interpreter is free for other threads while a call is enqueued.
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};
template <class F>
int enqueue(F call) {
  const Unlocked u;
  return call();
}

// dtype of an argument, or -1
int type_arg(PyObject* o, at::ScalarType* type) {
  if (!THPDtype_Check(o)) return -1;
  *type = ((THPDtype*)o)->scalar_type;
  return type_of(*type);
}

// MXFP4 codes and scales; ld and lds receive their strides.
struct Codes {
  const Tensor *codes = nullptr, *scales = nullptr;
  int64_t rows = 0, bytes = 0, ld = 0, lds = 0;
  Codes(PyObject* c, PyObject* s, const Place& p) {
    const Tensor* t = matrix(c, p, &ld);
    const Tensor* u = tensor(s, p);
    if (!t || !u || t->scalar_type() != at::kByte || u->scalar_type() != at::kByte || u->dim() != 3 ||
        !u->is_contiguous())
      return;
    rows = t->size(0);
    bytes = t->size(1);
    lds = u->size(1);
    if (bytes % 16 || u->size(0) != (bytes / 16 + 3) / 4 || u->size(2) != 4 || lds < rows || lds % 4) return;
    codes = t;
    scales = u;
  }
};

// ------------------------------------------------------------------------------------- norm
struct Norm {
  bool ok = false;
  const Tensor *x = nullptr, *r = nullptr;
  int64_t ldx = 0, ldr = 0, rows = 0, cols = 0;
  int type = 0, wtype = 0;
  const void* w = nullptr;
  double eps = 0;
  Tensor h;
  // (x, weight, eps, residual)
  Norm(PyObject* const* a, const Place& p) {
    x = matrix(a[0], p, &ldx);
    if (!x || (type = type_of(x->scalar_type())) < 0) return;
    rows = x->size(0);
    cols = x->size(1);
    if (!PyFloat_Check(a[2])) return;
    eps = PyFloat_AS_DOUBLE(a[2]);
    bool good = true;
    wtype = type;
    if (a[1] != Py_None) {
      const Tensor* t = tensor(a[1], p);
      if (!t) return;
      if (t->scalar_type() == at::kFloat) wtype = AWQ_FP32;
      w = vector(a[1], p, wtype == AWQ_FP32 ? at::kFloat : x->scalar_type(), cols, &good);
    }
    if (a[3] != Py_None) {
      r = matrix(a[3], p, &ldr);
      if (!r || r->scalar_type() != x->scalar_type() || r->sizes() != x->sizes()) return;
    }
    ok = good;
  }
  void* sum(const Place& p) {
    if (r) h = p.empty({rows, cols}, x->scalar_type());
    return r ? h.mutable_data_ptr() : nullptr;
  }
  PyObject* h_object(PyObject* x_object) {
    if (r) return THPVariable_Wrap(h);
    Py_INCREF(x_object);
    return x_object;
  }
};

PyObject* pair(PyObject* a, PyObject* b) {
  PyObject* t = a && b ? PyTuple_Pack(2, a, b) : nullptr;
  Py_XDECREF(a);
  Py_XDECREF(b);
  return t;
}
PyObject* triple(PyObject* a, PyObject* b, PyObject* c) {
  PyObject* t = a && b && c ? PyTuple_Pack(3, a, b, c) : nullptr;
  Py_XDECREF(a);
  Py_XDECREF(b);
  Py_XDECREF(c);
  return t;
}

PyObject* rmsnorm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 4 || !on_gpu(a[0])) return none();
  const Place p;
  Norm m(a, p);
  if (!m.ok) return none();
  void* h = m.sum(p);
  Tensor y = p.empty({m.rows, m.cols}, m.x->scalar_type());
  if (const int status = enqueue([&] {
        return awq_rmsnorm(m.x->const_data_ptr(), m.ldx, m.r ? m.r->const_data_ptr() : nullptr, m.ldr, m.rows, m.cols,
                      m.type, m.w, m.wtype, m.eps, h, m.cols, y.mutable_data_ptr(), m.cols, p.stream());
      }))
    return failed(status, "awq_rmsnorm");
  return pair(THPVariable_Wrap(y), m.h_object(a[0]));
  END_HANDLE_TH_ERRORS
}

PyObject* rmsnorm_int8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 4 || !on_gpu(a[0])) return none();
  const Place p;
  Norm m(a, p);
  if (!m.ok) return none();
  void* h = m.sum(p);
  const int64_t ld = round16(m.cols);
  Tensor codes = p.empty({m.rows, ld}, at::kChar), steps = p.empty({m.rows}, at::kFloat);
  if (const int status = enqueue([&] {
        return awq_rmsnorm_int8(m.x->const_data_ptr(), m.ldx, m.r ? m.r->const_data_ptr() : nullptr, m.ldr, m.rows,
                           m.cols, m.type, m.w, m.wtype, m.eps, h, m.cols, (int8_t*)codes.mutable_data_ptr(), ld,
                           (float*)steps.mutable_data_ptr(), p.stream());
      }))
    return failed(status, "awq_rmsnorm_int8");
  return triple(THPVariable_Wrap(codes), THPVariable_Wrap(steps), m.h_object(a[0]));
  END_HANDLE_TH_ERRORS
}

PyObject* rmsnorm_mxfp4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 4 || !on_gpu(a[0])) return none();
  const Place p;
  Norm m(a, p);
  if (!m.ok) return none();
  void* h = m.sum(p);
  const int64_t ld = code_bytes(m.cols), lds = round4(m.rows);
  Tensor codes = p.empty({m.rows, ld}, at::kByte), scales = p.empty({words(m.cols), lds, 4}, at::kByte);
  if (const int status = enqueue([&] {
        return awq_rmsnorm_mxfp4(m.x->const_data_ptr(), m.ldx, m.r ? m.r->const_data_ptr() : nullptr, m.ldr, m.rows,
                            m.cols, m.type, m.w, m.wtype, m.eps, h, m.cols, (uint8_t*)codes.mutable_data_ptr(), ld,
                            (uint8_t*)scales.mutable_data_ptr(), lds, p.stream());
      }))
    return failed(status, "awq_rmsnorm_mxfp4");
  return triple(THPVariable_Wrap(codes), THPVariable_Wrap(scales), m.h_object(a[0]));
  END_HANDLE_TH_ERRORS
}

// --------------------------------------------------------------------------- rows and values
// (codes, steps, cols, dtype)
PyObject* int8_dequantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 4 || !on_gpu(a[0]) || !PyLong_CheckExact(a[2])) return none();
  const Place p;
  int64_t ld;
  const Tensor* codes = matrix(a[0], p, &ld);
  const int64_t cols = PyLong_AsLongLong(a[2]);
  if (cols == -1 && PyErr_Occurred()) PyErr_Clear();
  at::ScalarType st;
  const int type = type_arg(a[3], &st);
  if (!codes || codes->scalar_type() != at::kChar || type < 0 || cols <= 0 || codes->size(1) != round16(cols))
    return none();
  bool ok = a[1] != Py_None;
  const int64_t rows = codes->size(0);
  const void* steps = vector(a[1], p, at::kFloat, rows, &ok);
  if (!ok) return none();
  Tensor y = p.empty({rows, cols}, st);
  if (const int status = enqueue([&] {
        return awq_int8_dequantize((const int8_t*)codes->const_data_ptr(), ld, (const float*)steps, rows, cols, type,
                              y.mutable_data_ptr(), cols, p.stream());
      }))
    return failed(status, "awq_int8_dequantize");
  return THPVariable_Wrap(y);
  END_HANDLE_TH_ERRORS
}

// (A, s, multiply)
PyObject* mxfp4_quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 3 || !on_gpu(a[0])) return none();
  const Place p;
  int64_t lda;
  const Tensor* A = matrix(a[0], p, &lda);
  if (!A || type_of(A->scalar_type()) < 0) return none();
  const int64_t rows = A->size(0), cols = A->size(1), ld = code_bytes(cols), lds = round4(rows);
  bool ok = true;
  const void* s = vector(a[1], p, at::kFloat, cols, &ok);
  if (!ok) return none();
  Tensor codes = p.empty({rows, ld}, at::kByte), scales = p.empty({words(cols), lds, 4}, at::kByte);
  if (const int status = enqueue([&] {
        return awq_mxfp4_quantize(A->const_data_ptr(), rows, cols, lda, type_of(A->scalar_type()), (const float*)s,
                             a[2] == Py_True ? AWQ_FOLD_MULTIPLY : AWQ_FOLD_DIVIDE, (uint8_t*)codes.mutable_data_ptr(),
                             ld, (uint8_t*)scales.mutable_data_ptr(), lds, p.stream());
      }))
    return failed(status, "awq_mxfp4_quantize");
  return pair(THPVariable_Wrap(codes), THPVariable_Wrap(scales));
  END_HANDLE_TH_ERRORS
}

// (codes, scales, cols, dtype)
PyObject* mxfp4_dequantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 4 || !on_gpu(a[0]) || !PyLong_CheckExact(a[2])) return none();
  const Place p;
  const Codes c(a[0], a[1], p);
  const int64_t cols = PyLong_AsLongLong(a[2]);
  if (cols == -1 && PyErr_Occurred()) PyErr_Clear();
  at::ScalarType st;
  const int type = type_arg(a[3], &st);
  if (!c.codes || type < 0 || cols <= 0 || c.bytes != code_bytes(cols)) return none();
  Tensor y = p.empty({c.rows, cols}, st);
  if (const int status = enqueue([&] {
        return awq_mxfp4_dequantize((const uint8_t*)c.codes->const_data_ptr(), c.ld,
                               (const uint8_t*)c.scales->const_data_ptr(), c.lds, c.rows, cols, type,
                               y.mutable_data_ptr(), cols, p.stream());
      }))
    return failed(status, "awq_mxfp4_dequantize");
  return THPVariable_Wrap(y);
  END_HANDLE_TH_ERRORS
}

// ----------------------------------------------------------------------------------- product
// (xc, xs, wc, ws, dtype, bias)
PyObject* mxfp4_matmul(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 6 || !on_gpu(a[0])) return none();
  const Place p;
  const Codes x(a[0], a[1], p), w(a[2], a[3], p);
  at::ScalarType st;
  const int type = type_arg(a[4], &st);
  if (!x.codes || !w.codes || x.bytes != w.bytes || type < 0) return none();
  bool ok = true;
  const void* bias = vector(a[5], p, st, w.rows, &ok);
  if (!ok) return none();
  Tensor y = p.empty({x.rows, w.rows}, st);
  if (const int status = enqueue([&] {
        return awq_mxfp4_matmul((const uint8_t*)x.codes->const_data_ptr(), x.ld,
                           (const uint8_t*)x.scales->const_data_ptr(), x.lds, x.rows,
                           (const uint8_t*)w.codes->const_data_ptr(), w.ld,
                           (const uint8_t*)w.scales->const_data_ptr(), w.lds, w.rows, 2 * x.bytes, bias, type,
                           y.mutable_data_ptr(), w.rows, p.stream());
      }))
    return failed(status, "awq_mxfp4_matmul");
  return THPVariable_Wrap(y);
  END_HANDLE_TH_ERRORS
}

// (x, wc, ws, s, bias)
PyObject* mxfp4_linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 5 || !on_gpu(a[0])) return none();
  const Place p;
  int64_t ldx;
  const Tensor* x = matrix(a[0], p, &ldx);
  const Codes w(a[1], a[2], p);
  if (!x || !w.codes || type_of(x->scalar_type()) < 0) return none();
  const int64_t T = x->size(0), K = x->size(1), M = w.rows;
  if (w.bytes != code_bytes(K)) return none();
  bool ok = true;
  const void* s = vector(a[3], p, at::kFloat, K, &ok);
  const void* bias = vector(a[4], p, x->scalar_type(), M, &ok);
  if (!ok) return none();
  Tensor y = p.empty({T, M}, x->scalar_type()), ws;
  const size_t need = awq_mxfp4_linear_workspace_bytes(T, M, K);
  if (need) ws = p.empty({(int64_t)need}, at::kByte);
  if (const int status = enqueue([&] {
        return awq_mxfp4_linear(x->const_data_ptr(), ldx, (const float*)s, T, (const uint8_t*)w.codes->const_data_ptr(),
                           w.ld, (const uint8_t*)w.scales->const_data_ptr(), w.lds, M, K, bias,
                           type_of(x->scalar_type()), y.mutable_data_ptr(), M,
                           need ? ws.mutable_data_ptr() : nullptr, need, p.stream());
      }))
    return failed(status, "awq_mxfp4_linear");
  return THPVariable_Wrap(y);
  END_HANDLE_TH_ERRORS
}

#define AWQ_CALL(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {AWQ_CALL(rmsnorm),        AWQ_CALL(rmsnorm_int8),     AWQ_CALL(rmsnorm_mxfp4),
                         AWQ_CALL(int8_dequantize), AWQ_CALL(mxfp4_quantize), AWQ_CALL(mxfp4_dequantize),
                         AWQ_CALL(mxfp4_matmul),   AWQ_CALL(mxfp4_linear),     {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls(void) { return PyModule_Create(&module); }
