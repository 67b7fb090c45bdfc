// What the CPython extensions around the C ABI share: they read the tensors'
// properties, allocate the results and call the library.  In Python, with
// ctypes, that took 3 to 4 us more per call, for layers that take 5 us on the GPU.
//
// torch itself is only used through its Python objects, handed over once by
// each extension's setup(); nothing of it is linked or included.
#pragma once

#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <climits>
#include <cstdint>

#include "dense_gemm.h"

namespace {

PyObject *g_empty, *g_raw_stream, *g_current_device, *g_error;   // set by setup_common()
PyObject *g_dtype[3], *g_uint8;                               // float32, float16, bfloat16
PyObject *g_empty_names;                                      // ("dtype", "device")
PyObject *n_is_cuda, *n_dtype, *n_shape, *n_stride, *n_data_ptr, *n_device, *n_index;

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

[[maybe_unused]] bool attr_int(PyObject* o, PyObject* name, int* out) {
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

// The names and objects of torch that every extension needs; `names` ends with a null.
struct Name {
  PyObject** to;
  const char* name;
};
bool setup_common(PyObject* torch, PyObject* error, const Name* names) {
  const Name common[] = {{&n_is_cuda, "is_cuda"}, {&n_dtype, "dtype"},       {&n_shape, "shape"},
                         {&n_stride, "stride"},   {&n_data_ptr, "data_ptr"}, {&n_device, "device"},
                         {&n_index, "index"},     {nullptr, nullptr}};
  for (const Name* list : {common, names})
    for (const Name* x = list; x->to != nullptr; ++x)
      if (*x->to == nullptr && (*x->to = PyUnicode_InternFromString(x->name)) == nullptr)
        return false;
  const char* types[3] = {"float32", "float16", "bfloat16"};
  for (int i = 0; i < 3; ++i)
    if ((g_dtype[i] = PyObject_GetAttrString(torch, types[i])) == nullptr) return false;
  if ((g_uint8 = PyObject_GetAttrString(torch, "uint8")) == nullptr) return false;
  Ref c(PyObject_GetAttrString(torch, "_C"));
  if (!c || (g_raw_stream = PyObject_GetAttrString(c.p, "_cuda_getCurrentRawStream")) == nullptr ||
      (g_current_device = PyObject_GetAttrString(c.p, "_cuda_getDevice")) == nullptr)
    return false;
  if ((g_empty_names = Py_BuildValue("(OO)", n_dtype, n_device)) == nullptr) return false;
  Py_INCREF(error);
  g_error = error;
  return (g_empty = PyObject_GetAttrString(torch, "empty")) != nullptr;
}

}  // namespace
