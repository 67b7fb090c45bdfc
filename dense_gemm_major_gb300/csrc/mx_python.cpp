// The torch wrappers of the microscaled operators as a CPython extension: it
// reads the tensors' properties, allocates the result and calls the C ABI.
// In Python, with ctypes, that took 3 to 4 us more per call, for a layer that
// takes 5 us on the GPU.  dense_gemm_major_gb300/__init__.py documents the
// functions and gives their defaults.
//
// torch itself is only used through its Python objects, handed over once by
// setup(); nothing of it is linked or included.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <climits>
#include <cstdint>

#include "dense_gemm_mx.h"

namespace {

PyObject *g_empty, *g_raw_stream, *g_current_device, *g_error, *g_tensor_type;   // set by setup()
PyObject *g_dtype[3], *g_uint8;                               // float32, float16, bfloat16
PyObject *g_empty_names;                                      // ("dtype", "device")
PyObject *n_is_cuda, *n_dtype, *n_shape, *n_stride, *n_data_ptr, *n_device, *n_index, *n_codes,
    *n_scales, *n_buffer, *n_rows, *n_cols, *n_fmt, *n_ld, *n_mxfp4, *n_numel, *n_is_contiguous,
    *n_mx_device;

// An owned reference.
struct Ref {
  PyObject* p;
  explicit Ref(PyObject* o = nullptr) : p(o) {}
  Ref(const Ref&) = delete;
  Ref& operator=(const Ref&) = delete;
  ~Ref() { Py_XDECREF(p); }
  void set(PyObject* o) {
    Py_XDECREF(p);
    p = o;
  }
  PyObject* release() {
    PyObject* o = p;
    p = nullptr;
    return o;
  }
  explicit operator bool() const { return p != nullptr; }
};

// A call of the library, which may wait (for a workspace, or for room in a full
// stream): other Python threads run meanwhile, the callbacks among them that the
// stream may be waiting for.
template <typename F>
gemm_status_t without_gil(F call) {
  PyThreadState* state = PyEval_SaveThread();
  const gemm_status_t st = call();
  PyEval_RestoreThread(state);
  return st;
}

bool value_error(const char* text) {
  PyErr_SetString(PyExc_ValueError, text);
  return false;
}

bool too_large() { return value_error("a size is above the formats' limit, 2^31 - 1024"); }

PyObject* failed(gemm_status_t st, const char* what) {
  Ref e(PyObject_CallFunction(g_error, "is", (int)st, what));
  if (e) PyErr_SetObject(g_error, e.p);
  return nullptr;
}

bool to_int(PyObject* o, int* out) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) return false;
  if (v < 0 || v > INT_MAX) return value_error("a size or stride is negative or above 2^31 - 1");
  *out = (int)v;
  return true;
}

bool attr_int(PyObject* o, PyObject* name, int* out) {
  Ref a(PyObject_GetAttr(o, name));
  return a && to_int(a.p, out);
}

bool address(PyObject* t, void** out) {
  Ref a(PyObject_CallMethodNoArgs(t, n_data_ptr));
  if (!a) return false;
  *out = PyLong_AsVoidPtr(a.p);
  return *out != nullptr || !PyErr_Occurred();
}

bool dtype_code(PyObject* dtype, int* code) {
  for (int i = 0; i < 3; ++i)
    if (dtype == g_dtype[i]) {
      *code = i;
      return true;
    }
  PyErr_Format(PyExc_ValueError, "unsupported dtype %S: float32, float16 or bfloat16", dtype);
  return false;
}

// Two ints of a tuple-like (torch.Size and strides are tuples).
bool pair_of(PyObject* t, int* a, int* b) {
  if (!PyTuple_Check(t) || PyTuple_GET_SIZE(t) != 2) return value_error("operands must be 2-D");
  return to_int(PyTuple_GET_ITEM(t, 0), a) && to_int(PyTuple_GET_ITEM(t, 1), b);
}

// A 2-D CUDA tensor.
struct Matrix {
  int code, rows, cols, s0, s1;
  void* ptr;
  Ref dtype, device;
  bool read(PyObject* t) {
    Ref cuda(PyObject_GetAttr(t, n_is_cuda));
    if (!cuda) return false;
    if (cuda.p != Py_True) return value_error("operands must be CUDA tensors");
    dtype.set(PyObject_GetAttr(t, n_dtype));
    if (!dtype || !dtype_code(dtype.p, &code)) return false;
    Ref shape(PyObject_GetAttr(t, n_shape));
    if (!shape || !pair_of(shape.p, &rows, &cols)) return false;
    Ref stride(PyObject_CallMethodNoArgs(t, n_stride));
    if (!stride || !pair_of(stride.p, &s0, &s1)) return false;
    device.set(PyObject_GetAttr(t, n_device));
    return device && address(t, &ptr);
  }
  // Leading dimension as a row-major array.
  bool row_major(int* ld) const {
    if (s1 != 1 && cols > 1)
      return value_error("operands must be 2-D row-major (unit column stride)");
    *ld = rows > 1 ? s0 : (cols > 0 ? cols : 1);
    return true;
  }
};

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

// Whether two operands' devices are the same.
bool one_device(PyObject* a, PyObject* b) {
  const int same = PyObject_RichCompareBool(a, b, Py_EQ);
  if (same == 0) return value_error("operands must be on one device");
  return same == 1;
}

// The given cudaStream_t, or torch's current stream on `device`, which must be
// the current one: the library's kernels run there.
bool stream_of(PyObject* stream, PyObject* device, cudaStream_t* out) {
  Ref s;
  Ref index(PyObject_GetAttr(device, n_index));
  if (!index) return false;
  Ref current(PyObject_CallNoArgs(g_current_device));
  if (!current) return false;
  const int same = PyObject_RichCompareBool(index.p, current.p, Py_EQ);
  if (same < 0) return false;
  if (!same) return value_error("operands must be on the current CUDA device");
  if (stream == Py_None) {
    s.set(PyObject_CallOneArg(g_raw_stream, index.p));
    if (!s) return false;
  } else {
    Py_INCREF(stream);
    s.set(stream);
  }
  *out = (cudaStream_t)PyLong_AsVoidPtr(s.p);
  return *out != nullptr || !PyErr_Occurred();
}

PyObject* empty(PyObject* size, PyObject* dtype, PyObject* device) {
  PyObject* args[3] = {size, dtype, device};
  return PyObject_Vectorcall(g_empty, args, 1, g_empty_names);
}

// `out`, checked, or a new rows x cols tensor.
struct Result {
  Ref tensor;
  int ld;
  void* ptr;
  bool make(PyObject* out, int rows, int cols, PyObject* dtype, PyObject* device, double beta) {
    if (out == Py_None) {
      if (beta != 0.0) return value_error("beta != 0 needs an existing out");
      Ref size(Py_BuildValue("(ii)", rows, cols));
      if (!size) return false;
      tensor.set(empty(size.p, dtype, device));
      ld = cols > 0 ? cols : 1;
      return tensor && address(tensor.p, &ptr);
    }
    Matrix m;
    if (!m.read(out)) return false;
    const int same = PyObject_RichCompareBool(m.device.p, device, Py_EQ);
    if (same < 0) return false;
    if (m.rows != rows || m.cols != cols || m.dtype.p != dtype || !same)
      return value_error("out has the wrong shape, dtype or device");
    Py_INCREF(out);
    tensor.set(out);
    ptr = m.ptr;
    return m.row_major(&ld);
  }
};

// The dtype asked for, that of `out`, or `otherwise` (a new reference).
PyObject* result_dtype(PyObject* dtype, PyObject* out, PyObject* otherwise) {
  if (dtype == Py_None && out != Py_None) return PyObject_GetAttr(out, n_dtype);
  PyObject* d = dtype == Py_None ? otherwise : dtype;
  Py_INCREF(d);
  return d;
}

bool same_inner(int a, int b) {
  if (a == b) return true;
  PyErr_Format(PyExc_ValueError, "inner dimensions differ: %d vs %d", a, b);
  return false;
}

bool two_doubles(PyObject* a, PyObject* b, double* x, double* y) {
  *x = PyFloat_AsDouble(a);
  if (*x == -1.0 && PyErr_Occurred()) return false;
  *y = PyFloat_AsDouble(b);
  return *y != -1.0 || !PyErr_Occurred();
}

bool arity(Py_ssize_t n, Py_ssize_t want) {
  if (n == want && g_empty != nullptr) return true;
  PyErr_SetString(PyExc_TypeError, "wrong number of arguments, or setup() was not called");
  return false;
}

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
  struct {
    PyObject** to;
    const char* name;
  } names[] = {{&n_is_cuda, "is_cuda"}, {&n_dtype, "dtype"},   {&n_shape, "shape"},
               {&n_stride, "stride"},   {&n_data_ptr, "data_ptr"}, {&n_device, "device"},
               {&n_index, "index"},     {&n_codes, "_codes"},  {&n_scales, "_scales"},
               {&n_buffer, "_buffer"},  {&n_rows, "rows"},     {&n_cols, "cols"},
               {&n_fmt, "fmt"},         {&n_ld, "_ld"},        {&n_mxfp4, "mxfp4"},
               {&n_numel, "numel"},     {&n_is_contiguous, "is_contiguous"},
               {&n_mx_device, "_device"}};
  for (auto& x : names)
    if (*x.to == nullptr && (*x.to = PyUnicode_InternFromString(x.name)) == nullptr)
      return nullptr;
  const char* types[3] = {"float32", "float16", "bfloat16"};
  for (int i = 0; i < 3; ++i)
    if ((g_dtype[i] = PyObject_GetAttrString(a[0], types[i])) == nullptr) return nullptr;
  if ((g_uint8 = PyObject_GetAttrString(a[0], "uint8")) == nullptr) return nullptr;
  Ref c(PyObject_GetAttrString(a[0], "_C"));
  if (!c || (g_raw_stream = PyObject_GetAttrString(c.p, "_cuda_getCurrentRawStream")) == nullptr ||
      (g_current_device = PyObject_GetAttrString(c.p, "_cuda_getDevice")) == nullptr)
    return nullptr;
  if ((g_empty_names = Py_BuildValue("(OO)", n_dtype, n_device)) == nullptr) return nullptr;
  Py_INCREF(a[1]);
  g_tensor_type = a[1];
  Py_INCREF(a[2]);
  g_error = a[2];
  if ((g_empty = PyObject_GetAttrString(a[0], "empty")) == nullptr) return nullptr;
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
