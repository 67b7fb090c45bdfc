// The torch wrappers of the grouped products and of those with 4-bit weights as a
// CPython extension around the C ABI (see py_call.h).  dense_gemm_major_gb300/__init__.py
// documents the functions and gives their defaults.
#include "py_call.h"

#include "dense_gemm_group.h"
#include "dense_gemm_q4.h"

namespace {

PyObject *g_int32, *g_q4_type;   // set by setup()
PyObject *n_codes, *n_scales, *n_zeros, *n_experts, *n_rows, *n_cols, *n_group, *n_ld;

// A 3-D CUDA tensor: matrices of rows x cols.
struct Matrices {
  int code, count, rows, cols, s1, s2;
  long long s0;
  void* ptr;
  Ref dtype, device;
  bool read(PyObject* t) {
    Ref cuda(PyObject_GetAttr(t, n_is_cuda));
    if (!cuda) return false;
    if (cuda.p != Py_True) return value_error("operands must be CUDA tensors");
    dtype.set(PyObject_GetAttr(t, n_dtype));
    if (!dtype || !dtype_code(dtype.p, &code)) return false;
    Ref shape(PyObject_GetAttr(t, n_shape));
    Ref stride(PyObject_CallMethodNoArgs(t, n_stride));
    if (!shape || !stride) return false;
    if (!PyTuple_Check(shape.p) || PyTuple_GET_SIZE(shape.p) != 3 || !PyTuple_Check(stride.p) ||
        PyTuple_GET_SIZE(stride.p) != 3)
      return value_error("the groups' matrices must be one 3-D tensor");
    s0 = PyLong_AsLongLong(PyTuple_GET_ITEM(stride.p, 0));
    if (s0 == -1 && PyErr_Occurred()) return false;
    if (!to_int(PyTuple_GET_ITEM(shape.p, 0), &count) ||
        !to_int(PyTuple_GET_ITEM(shape.p, 1), &rows) ||
        !to_int(PyTuple_GET_ITEM(shape.p, 2), &cols) ||
        !to_int(PyTuple_GET_ITEM(stride.p, 1), &s1) || !to_int(PyTuple_GET_ITEM(stride.p, 2), &s2))
      return false;
    device.set(PyObject_GetAttr(t, n_device));
    return device && address(t, &ptr);
  }
};

inline int round8(int n) {
  const long long r = ((long long)n + 7) / 8 * 8;
  return r > INT_MAX ? n : (int)r;
}

// Leading dimension of a single stored row: free, so a multiple of 8 where the
// rest is aligned (it is then read where it is).
inline int single(int width, const void* p) {
  return ((uintptr_t)p & 15u) == 0 ? round8(width) : width;
}

bool row_major16(const Matrix& m, int* ld) {
  if (m.code == 0) return value_error("grouped products take float16 or bfloat16 operands");
  if (!m.row_major(ld)) return false;
  if (m.rows <= 1) *ld = single(m.cols > 0 ? m.cols : 1, m.ptr);
  return true;
}

// The groups' offsets: their address and number.
struct Offsets {
  int groups;
  void* ptr;
  bool read(PyObject* t, PyObject* device_of_operands) {
    Ref cuda(PyObject_GetAttr(t, n_is_cuda)), type(PyObject_GetAttr(t, n_dtype)),
        shape(PyObject_GetAttr(t, n_shape)), stride(PyObject_CallMethodNoArgs(t, n_stride)),
        device(PyObject_GetAttr(t, n_device));
    if (!cuda || !type || !shape || !stride || !device) return false;
    int n, step;
    if (cuda.p != Py_True || type.p != g_int32 || !PyTuple_Check(shape.p) ||
        PyTuple_GET_SIZE(shape.p) != 1)
      return value_error("offsets must be a 1-D int32 CUDA tensor");
    if (!to_int(PyTuple_GET_ITEM(shape.p, 0), &n) || !to_int(PyTuple_GET_ITEM(stride.p, 0), &step))
      return false;
    if (n < 1) return value_error("offsets must have one element more than there are groups");
    if (step != 1 && n > 1) return value_error("offsets must be contiguous");
    if (n - 1 > GEMM_GROUP_MAX_GROUPS) return value_error("more than 1024 groups");
    groups = n - 1;
    return one_device(device.p, device_of_operands) && address(t, &ptr);
  }
};

// grouped_matmul(A, B, offsets, out, dtype, alpha, beta, stream)
PyObject* grouped_matmul(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 8)) return nullptr;
  Matrix x;
  Matrices b;
  Offsets off;
  int lda;
  if (!x.read(a[0]) || !b.read(a[1]) || !row_major16(x, &lda) || !off.read(a[2], x.device.p))
    return nullptr;
  if (b.code != x.code) return value_error("A and B must have the same dtype"), nullptr;
  if (off.groups != b.count)
    return value_error("offsets must have one element more than B has matrices"), nullptr;
  if (!one_device(x.device.p, b.device.p) || !same_inner(x.cols, b.rows)) return nullptr;
  gemm_op_t op = GEMM_OP_N;
  int ldb, outer = b.rows, inner = b.cols;
  // (A single column with unit stride is a single row stored transposed.)
  if ((b.s2 == 1 || b.cols <= 1) && !(b.cols == 1 && b.rows > 1 && b.s1 == 1)) {
    ldb = b.s1;
  } else if (b.s1 == 1 || b.rows <= 1) {
    op = GEMM_OP_T;
    ldb = b.s2;
    outer = b.cols, inner = b.rows;
  } else {
    return value_error("B's matrices must have a unit row or column stride"), nullptr;
  }
  const long long stride_b = b.count > 1 ? b.s0 : 0;
  if (outer <= 1) ldb = stride_b % 8 == 0 ? single(inner, b.ptr) : inner;
  if (inner == 0) ldb = 1;
  Ref dtype(result_dtype(a[4], a[3], x.dtype.p));
  int code;
  double alpha, beta;
  if (!dtype || !dtype_code(dtype.p, &code) || !two_doubles(a[5], a[6], &alpha, &beta))
    return nullptr;
  if (code != 0 && code != x.code)
    return value_error("the result is of the operands' dtype or float32"), nullptr;
  Result c;
  cudaStream_t stream;
  if (!stream_of(a[7], x.device.p, &stream) ||
      !c.make(a[3], x.rows, b.cols, dtype.p, x.device.p, beta))
    return nullptr;
  const gemm_status_t st = without_gil([&] {
    return gemm_grouped(x.code, op, code, x.rows, b.cols, x.cols, off.groups, (float)alpha, x.ptr,
                        lda, b.ptr, ldb, stride_b, (const int*)off.ptr, (float)beta, c.ptr, c.ld,
                        stream);
  });
  if (st != GEMM_OK) return failed(st, "gemm_grouped");
  return c.tensor.release();
}

// grouped_grad(A, X, offsets, out, dtype, alpha, beta, stream)
PyObject* grouped_grad(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 8)) return nullptr;
  Matrix x, y;
  Offsets off;
  int lda, ldx;
  if (!y.read(a[0]) || !x.read(a[1]) || !row_major16(y, &lda) || !row_major16(x, &ldx) ||
      !off.read(a[2], x.device.p))
    return nullptr;
  if (y.code != x.code) return value_error("A and X must have the same dtype"), nullptr;
  if (!one_device(x.device.p, y.device.p)) return nullptr;
  if (y.rows != x.rows) {
    PyErr_Format(PyExc_ValueError, "rows differ: %d vs %d", y.rows, x.rows);
    return nullptr;
  }
  Ref dtype(result_dtype(a[4], a[3], x.dtype.p));
  int code;
  double alpha, beta;
  if (!dtype || !dtype_code(dtype.p, &code) || !two_doubles(a[5], a[6], &alpha, &beta))
    return nullptr;
  if (code != 0 && code != x.code)
    return value_error("the result is of the operands' dtype or float32"), nullptr;
  cudaStream_t stream;
  if (!stream_of(a[7], x.device.p, &stream)) return nullptr;
  Ref out;
  void* ptr;
  int ldc = x.cols > 0 ? x.cols : 1;
  long long stride_c = (long long)y.cols * ldc;
  if (a[3] == Py_None) {
    if (beta != 0.0) return value_error("beta != 0 needs an existing out"), nullptr;
    Ref size(Py_BuildValue("(iii)", off.groups, y.cols, x.cols));
    if (!size) return nullptr;
    out.set(empty(size.p, dtype.p, x.device.p));
    if (!out || !address(out.p, &ptr)) return nullptr;
  } else {
    Matrices m;
    if (!m.read(a[3])) return nullptr;
    const int same = PyObject_RichCompareBool(m.device.p, x.device.p, Py_EQ);
    if (same < 0) return nullptr;
    if (m.count != off.groups || m.rows != y.cols || m.cols != x.cols || m.dtype.p != dtype.p ||
        !same)
      return value_error("out has the wrong shape, dtype or device"), nullptr;
    if (m.s2 != 1 && m.cols > 1)
      return value_error("out's matrices must be row-major (unit column stride)"), nullptr;
    if (m.rows > 1) ldc = m.s1;
    stride_c = m.s0;
    ptr = m.ptr;
    Py_INCREF(a[3]);
    out.set(a[3]);
  }
  const gemm_status_t st = without_gil([&] {
    return gemm_grouped_grad(x.code, code, x.rows, y.cols, x.cols, off.groups, (float)alpha, y.ptr,
                             lda, x.ptr, ldx, (const int*)off.ptr, (float)beta, ptr, ldc, stride_c,
                             stream);
  });
  if (st != GEMM_OK) return failed(st, "gemm_grouped_grad");
  return out.release();
}

// q4_linear(x, W, offsets, out, stream)
PyObject* q4_linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 5)) return nullptr;
  Matrix x;
  int ldx, experts, rows, cols, group, ldq;
  if (!x.read(a[0]) || !row_major16(x, &ldx)) return nullptr;
  PyObject* const w = a[1];
  if (!PyObject_TypeCheck(w, (PyTypeObject*)g_q4_type))
    return value_error("the weights must be a Q4Tensor"), nullptr;
  if (!attr_int(w, n_experts, &experts) || !attr_int(w, n_rows, &rows) ||
      !attr_int(w, n_cols, &cols) || !attr_int(w, n_group, &group) || !attr_int(w, n_ld, &ldq))
    return nullptr;
  Ref codes(PyObject_GetAttr(w, n_codes)), scales(PyObject_GetAttr(w, n_scales)),
      zeros(PyObject_GetAttr(w, n_zeros));
  if (!codes || !scales || !zeros) return nullptr;
  Ref device(PyObject_GetAttr(codes.p, n_device)), type(PyObject_GetAttr(scales.p, n_dtype));
  if (!device || !type) return nullptr;
  if (type.p != x.dtype.p) return value_error("x and the scales must have the same dtype"), nullptr;
  if (!one_device(x.device.p, device.p) || !same_inner(x.cols, cols)) return nullptr;
  Offsets off{0, nullptr};
  if (experts > 0) {
    if (a[2] == Py_None) return value_error("weights of experts need offsets"), nullptr;
    if (!off.read(a[2], x.device.p)) return nullptr;
    if (off.groups != experts)
      return value_error("offsets must have one element more than there are experts"), nullptr;
  } else if (a[2] != Py_None) {
    return value_error("offsets are for weights of experts (3-D codes)"), nullptr;
  }
  void *qp, *sp, *zp = nullptr;
  if (!address(codes.p, &qp) || !address(scales.p, &sp) ||
      (zeros.p != Py_None && !address(zeros.p, &zp)))
    return nullptr;
  Result y;
  cudaStream_t stream;
  if (!stream_of(a[4], x.device.p, &stream) ||
      !y.make(a[3], x.rows, rows, x.dtype.p, x.device.p, 0.0))
    return nullptr;
  const gemm_status_t st = without_gil([&] {
    return gemm_q4_linear(x.code, group, x.rows, rows, x.cols, experts, x.ptr, ldx, qp, ldq, sp,
                          zp, (const int*)off.ptr, y.ptr, y.ld, stream);
  });
  if (st != GEMM_OK) return failed(st, "gemm_q4_linear");
  return y.tensor.release();
}

// setup(torch, Q4Tensor, GemmError)
PyObject* setup(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 3) {
    PyErr_SetString(PyExc_TypeError, "setup(torch, Q4Tensor, GemmError)");
    return nullptr;
  }
  const Name names[] = {{&n_codes, "codes"}, {&n_scales, "_scales"}, {&n_zeros, "_zeros"},
                        {&n_experts, "experts"}, {&n_rows, "rows"}, {&n_cols, "cols"},
                        {&n_group, "group"}, {&n_ld, "_ld"}, {nullptr, nullptr}};
  Py_INCREF(a[1]);
  g_q4_type = a[1];
  if ((g_int32 = PyObject_GetAttrString(a[0], "int32")) == nullptr ||
      !setup_common(a[0], a[2], names))
    return nullptr;
  Py_RETURN_NONE;
}

#define METHOD(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {METHOD(setup), METHOD(grouped_matmul), METHOD(grouped_grad),
                           METHOD(q4_linear),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_groupcall", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__groupcall(void) { return PyModule_Create(&g_module); }
