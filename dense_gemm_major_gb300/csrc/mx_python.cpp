// The torch wrappers of the microscaled operators as a CPython extension around
// the C ABI (see py_call.h).  dense_gemm_major_gb300/__init__.py documents the
// functions and gives their defaults.
#include "py_call.h"

#include "dense_gemm_mx.h"

namespace {

PyObject *g_tensor_type;   // set by setup()
PyObject *n_codes, *n_scales, *n_buffer, *n_rows, *n_cols, *n_fmt, *n_ld, *n_mxfp4, *n_numel,
    *n_is_contiguous, *n_mx_device;

bool too_large() { return value_error("a size is above the formats' limit, 2^31 - 1024"); }

// An MXTensor's arrays, kept alive.  (Its _device is that of the arrays, None
// where they are not on a GPU.)
struct Quantized {
  int rows, cols, ld;
  gemm_mx_format_t fmt;
  char *codes, *scales;
  Ref device, owner, owner2;
  bool read(PyObject* q) {
    if (!PyObject_TypeCheck(q, (PyTypeObject*)g_tensor_type))
      return value_error("the operand must be an MXTensor");
    device.set(PyObject_GetAttr(q, n_mx_device));
    if (!device) return false;
    if (device.p == Py_None) return value_error("operands must be CUDA tensors");
    if (!attr_int(q, n_rows, &rows) || !attr_int(q, n_cols, &cols) || !attr_int(q, n_ld, &ld))
      return false;
    Ref f(PyObject_GetAttr(q, n_fmt));
    if (!f) return false;
    fmt = f.p == n_mxfp4 || PyUnicode_CompareWithASCIIString(f.p, "mxfp4") == 0 ? GEMM_MXFP4
                                                                               : GEMM_MXINT8;
    Ref buffer(PyObject_GetAttr(q, n_buffer));
    if (!buffer) return false;
    void* p;
    if (buffer.p != Py_None) {   // codes, then scales
      if (!address(buffer.p, &p)) return false;
      codes = (char*)p;
      scales = codes + (long long)rows * ld;
      owner.set(buffer.release());
      return true;
    }
    Ref c(PyObject_GetAttr(q, n_codes)), s(PyObject_GetAttr(q, n_scales));
    if (!c || !s) return false;
    if (!address(c.p, &p)) return false;
    codes = (char*)p;
    if (!address(s.p, &p)) return false;
    scales = (char*)p;
    owner.set(c.release());
    owner2.set(s.release());
    return true;
  }
};

// quantize(X, fmt, stream) -> (buffer, rows, cols, pitch of the codes, device)
PyObject* quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 3)) return nullptr;
  if (!PyUnicode_Check(a[1])) return value_error("fmt must be 'mxfp4' or 'mxint8'"), nullptr;
  const bool fp4 = PyUnicode_CompareWithASCIIString(a[1], "mxfp4") == 0;
  if (!fp4 && PyUnicode_CompareWithASCIIString(a[1], "mxint8") != 0)
    return value_error("fmt must be 'mxfp4' or 'mxint8'"), nullptr;
  const gemm_mx_format_t fmt = fp4 ? GEMM_MXFP4 : GEMM_MXINT8;
  Matrix x;
  if (!x.read(a[0])) return nullptr;
  gemm_op_t op = GEMM_OP_N;
  int ldx;
  if (x.s1 == 1 || x.cols <= 1) {
    ldx = x.rows > 1 ? x.s0 : (x.cols > 0 ? x.cols : 1);
  } else if (x.s0 == 1 || x.rows <= 1) {
    op = GEMM_OP_T;
    ldx = x.s1;
  } else {
    return value_error("operands must have a unit row or column stride"), nullptr;
  }
  cudaStream_t stream;
  if (!stream_of(a[2], x.device.p, &stream)) return nullptr;
  if (x.rows > GEMM_MX_MAX_SIZE || x.cols > GEMM_MX_MAX_SIZE) return too_large(), nullptr;
  const int ldq = gemm_mx_code_ld(fmt, x.cols);
  const long long codes = (long long)x.rows * ldq;
  Ref size(PyLong_FromLongLong(codes + gemm_mx_scale_bytes(x.rows, x.cols)));
  if (!size) return nullptr;
  Ref buffer(empty(size.p, g_uint8, x.device.p));
  void* p;
  if (!buffer || !address(buffer.p, &p)) return nullptr;
  const gemm_status_t st = without_gil([&] {
    return gemm_mx_quantize(fmt, x.code, op, x.rows, x.cols, x.ptr, ldx, p, ldq, (char*)p + codes,
                            stream);
  });
  if (st != GEMM_OK) return failed(st, "gemm_mx_quantize");
  return Py_BuildValue("NiiiN", buffer.release(), x.rows, x.cols, ldq, x.device.release());
}

// dequantize(q, dtype, out, stream)
PyObject* dequantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 4)) return nullptr;
  Quantized q;
  if (!q.read(a[0])) return nullptr;
  Ref dtype(result_dtype(a[1], a[2], g_dtype[2]));
  int code;
  Result y;
  cudaStream_t stream;
  if (!dtype || !dtype_code(dtype.p, &code) || !stream_of(a[3], q.device.p, &stream) ||
      !y.make(a[2], q.rows, q.cols, dtype.p, q.device.p, 0.0))
    return nullptr;
  const gemm_status_t st = without_gil([&] {
    return gemm_mx_dequantize(q.fmt, code, q.rows, q.cols, q.codes, q.ld, q.scales, y.ptr, y.ld,
                              stream);
  });
  if (st != GEMM_OK) return failed(st, "gemm_mx_dequantize");
  return y.tensor.release();
}

// matmul(A, B, out, dtype, alpha, beta, stream)
PyObject* matmul(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 7)) return nullptr;
  Quantized x, w;
  if (!x.read(a[0]) || !w.read(a[1])) return nullptr;
  if (x.fmt != GEMM_MXFP4 || w.fmt != GEMM_MXFP4)
    return value_error("mx_matmul takes mxfp4 operands"), nullptr;
  if (!one_device(x.device.p, w.device.p) || !same_inner(x.cols, w.cols)) return nullptr;
  Ref dtype(result_dtype(a[3], a[2], g_dtype[2]));
  int code;
  double alpha, beta;
  Result c;
  cudaStream_t stream;
  if (!dtype || !dtype_code(dtype.p, &code) || !two_doubles(a[4], a[5], &alpha, &beta) ||
      !stream_of(a[6], x.device.p, &stream) ||
      !c.make(a[2], x.rows, w.rows, dtype.p, x.device.p, beta))
    return nullptr;
  const gemm_status_t st = without_gil([&] {
    return gemm_mx4(code, x.rows, w.rows, x.cols, (float)alpha, x.codes, x.ld, x.scales, w.codes,
                    w.ld, w.scales, (float)beta, c.ptr, c.ld, stream);
  });
  if (st != GEMM_OK) return failed(st, "gemm_mx4");
  return c.tensor.release();
}

// linear(x, W, out, stream)
PyObject* linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 4)) return nullptr;
  Matrix x;
  Quantized w;
  if (!x.read(a[0]) || !w.read(a[1])) return nullptr;
  if (w.fmt != GEMM_MXFP4) return value_error("mx_linear takes mxfp4 weights"), nullptr;
  int ldx;
  Result y;
  cudaStream_t stream;
  if (!one_device(x.device.p, w.device.p) || !same_inner(x.cols, w.cols) || !x.row_major(&ldx) ||
      !stream_of(a[3], x.device.p, &stream) ||
      !y.make(a[2], x.rows, w.rows, x.dtype.p, x.device.p, 0.0))
    return nullptr;
  const gemm_status_t st = without_gil([&] {
    return gemm_mx4_linear(x.code, x.rows, w.rows, x.cols, x.ptr, ldx, w.codes, w.ld, w.scales,
                           y.ptr, y.ld, stream);
  });
  if (st != GEMM_OK) return failed(st, "gemm_mx4_linear");
  return y.tensor.release();
}

// grad(A, B, out, dtype, alpha, beta, stream)
PyObject* grad(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 7)) return nullptr;
  Matrix x;
  Quantized b;
  if (!x.read(a[0]) || !b.read(a[1])) return nullptr;
  if (x.code == 0) return value_error("mx_grad takes a float16 or bfloat16 A"), nullptr;
  if (!one_device(x.device.p, b.device.p) || !same_inner(x.cols, b.rows)) return nullptr;
  // The leading dimension of a single stored row is free: rounded up to a
  // multiple of 8, which is read where it is, or for an unaligned one its width.
  // A single column with unit stride is a single row stored transposed.
  const bool aligned = ((uintptr_t)x.ptr & 15u) == 0;
  auto single = [&](int width) { return aligned ? (int)(((long long)width + 7) / 8 * 8) : width; };
  gemm_op_t op = GEMM_OP_N;
  int lda;
  if ((x.s1 == 1 || x.cols <= 1) && !(x.cols == 1 && x.rows > 1 && x.s0 == 1)) {
    lda = x.rows > 1 ? x.s0 : single(x.cols);
  } else if (x.s0 == 1 || x.rows <= 1) {
    op = GEMM_OP_T;
    lda = x.cols > 1 ? x.s1 : single(x.rows);
  } else {
    return value_error("operands must have a unit row or column stride"), nullptr;
  }
  Ref dtype(result_dtype(a[3], a[2], x.dtype.p));
  int code;
  double alpha, beta;
  if (!dtype || !dtype_code(dtype.p, &code) || !two_doubles(a[4], a[5], &alpha, &beta))
    return nullptr;
  if (code != 0 && code != x.code)
    return value_error("the result is of A's dtype or float32"), nullptr;
  Result c;
  cudaStream_t stream;
  if (!stream_of(a[6], x.device.p, &stream) ||
      !c.make(a[2], x.rows, b.cols, dtype.p, x.device.p, beta))
    return nullptr;
  const gemm_status_t st = without_gil([&] {
    return gemm_mx_grad(b.fmt, x.code, op, code, x.rows, b.cols, x.cols, (float)alpha, x.ptr, lda,
                        b.codes, b.ld, b.scales, (float)beta, c.ptr, c.ld, stream);
  });
  if (st != GEMM_OK) return failed(st, "gemm_mx_grad");
  return c.tensor.release();
}

// describe(codes, scales, cols, fmt) -> (rows, pitch of the codes, device or
// None): the checks of an MXTensor's arrays.
PyObject* describe(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 4)) return nullptr;
  int cols, rows, width, ld, unit;
  if (!to_int(a[2], &cols)) return nullptr;
  gemm_mx_format_t fmt = GEMM_MXFP4;
  if (!PyUnicode_Check(a[3])) return value_error("fmt must be 'mxfp4' or 'mxint8'"), nullptr;
  if (PyUnicode_CompareWithASCIIString(a[3], "mxfp4") != 0) {
    if (PyUnicode_CompareWithASCIIString(a[3], "mxint8") != 0)
      return value_error("fmt must be 'mxfp4' or 'mxint8'"), nullptr;
    fmt = GEMM_MXINT8;
  }
  Ref type(PyObject_GetAttr(a[0], n_dtype)), shape(PyObject_GetAttr(a[0], n_shape));
  if (!type || !shape || !pair_of(shape.p, &rows, &width)) return nullptr;
  Ref stride(PyObject_CallMethodNoArgs(a[0], n_stride));
  if (!stride || !pair_of(stride.p, &ld, &unit)) return nullptr;
  if (type.p != g_uint8 || (long long)width * (fmt == GEMM_MXFP4 ? 2 : 1) < cols ||
      (unit != 1 && width > 1))
    return value_error("codes must be uint8 rows of at least the format's bytes for cols"),
           nullptr;
  if (rows > GEMM_MX_MAX_SIZE || cols > GEMM_MX_MAX_SIZE) return too_large(), nullptr;
  Ref stype(PyObject_GetAttr(a[1], n_dtype));
  Ref contiguous(PyObject_CallMethodNoArgs(a[1], n_is_contiguous));
  Ref count(PyObject_CallMethodNoArgs(a[1], n_numel));
  if (!stype || !contiguous || !count) return nullptr;
  const long long have = PyLong_AsLongLong(count.p);
  if (have == -1 && PyErr_Occurred()) return nullptr;
  if (stype.p != g_uint8 || contiguous.p != Py_True || have < gemm_mx_scale_bytes(rows, cols))
    return value_error("scales must be contiguous uint8, 512 bytes for each 128 x 128 tile"),
           nullptr;
  Ref device(PyObject_GetAttr(a[0], n_device)), sdevice(PyObject_GetAttr(a[1], n_device));
  if (!device || !sdevice || !one_device(device.p, sdevice.p)) return nullptr;
  // (The pitch of a single row is free: its padded width.)
  Ref cuda(PyObject_GetAttr(a[0], n_is_cuda));
  if (!cuda) return nullptr;
  return Py_BuildValue("iiO", rows, rows > 1 ? ld : (int)(((long long)width + 15) / 16 * 16),
                       cuda.p == Py_True ? device.p : Py_None);
}

// setup(torch, MXTensor, GemmError)
PyObject* setup(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 3) {
    PyErr_SetString(PyExc_TypeError, "setup(torch, MXTensor, GemmError)");
    return nullptr;
  }
  const Name names[] = {{&n_codes, "_codes"}, {&n_scales, "_scales"}, {&n_buffer, "_buffer"},
                        {&n_rows, "rows"},    {&n_cols, "cols"},      {&n_fmt, "fmt"},
                        {&n_ld, "_ld"},       {&n_mxfp4, "mxfp4"},    {&n_numel, "numel"},
                        {&n_is_contiguous, "is_contiguous"},
                        {&n_mx_device, "_device"}, {nullptr, nullptr}};
  Py_INCREF(a[1]);
  g_tensor_type = a[1];
  if (!setup_common(a[0], a[2], names)) return nullptr;
  Py_RETURN_NONE;
}

#define METHOD(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {METHOD(setup), METHOD(quantize), METHOD(dequantize), METHOD(matmul),
                           METHOD(linear), METHOD(grad),
                           METHOD(describe), {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_mxcall", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mxcall(void) { return PyModule_Create(&g_module); }
