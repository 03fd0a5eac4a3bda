/* pycall.c -- Python calls of the 8-bit linear layer's entry points and of the products
 * by group (include/mcg.h) without ctypes: the small operators take 2.7 us to launch, and
 * marshalling a dozen arguments through ctypes and Python took as long again.  Arguments
 * come by position, in the C order; a tensor gives its address, None a null pointer, an
 * integer itself.  Each function returns the mcg_status; the stream's None is torch's
 * current stream.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <stdint.h>

#include "../../include/mcg.h"

static PyObject *dtypes, *layouts; /* names of the enums: dicts */
static PyObject *to_stream;        /* stream(object) -> handle */
static PyObject *raw_stream, *raw_device; /* the current stream's handle; None: by to_stream */
static PyObject *s_data_ptr, *s_nbytes;
static int stream_up; /* to_stream has initialised torch's device */

/* The converters do nothing once one of them has raised; CALL then returns NULL. */
static int64_t as_int(PyObject *o) {
  if (PyErr_Occurred()) return -1;
  if (PyLong_Check(o)) return PyLong_AsLongLong(o);
  PyObject *i = PyNumber_Index(o);
  if (!i) return -1;
  const int64_t v = PyLong_AsLongLong(i);
  Py_DECREF(i);
  return v;
}
static int as_enum(PyObject *o, PyObject *names) {
  if (PyErr_Occurred()) return -1;
  if (!PyUnicode_Check(o)) return (int)as_int(o);
  PyObject *v = PyDict_GetItemWithError(names, o);
  if (!v) {
    if (!PyErr_Occurred()) PyErr_SetObject(PyExc_KeyError, o);
    return -1;
  }
  return (int)PyLong_AsLong(v);
}
static void *as_ptr(PyObject *o) {
  if (o == Py_None || PyErr_Occurred()) return NULL;
  if (PyLong_Check(o)) return PyLong_AsVoidPtr(o);
  PyObject *v = PyObject_CallMethodNoArgs(o, s_data_ptr);
  if (!v) return NULL;
  void *p = PyLong_AsVoidPtr(v);
  Py_DECREF(v);
  return p;
}
static void *as_stream(PyObject *o) {
  if (PyErr_Occurred()) return NULL;
  if (PyLong_Check(o)) return PyLong_AsVoidPtr(o);
  PyObject *v;
  if (o == Py_None && stream_up && raw_stream != Py_None && raw_device != Py_None) {
    PyObject *dev = PyObject_CallNoArgs(raw_device);
    if (!dev) return NULL;
    v = PyObject_CallOneArg(raw_stream, dev);
    Py_DECREF(dev);
  } else {
    v = PyObject_CallOneArg(to_stream, o);
    if (v) stream_up = 1;
  }
  if (!v) return NULL;
  void *p = PyLong_AsVoidPtr(v);
  Py_DECREF(v);
  return p;
}
/* Bytes of a workspace: a tensor's own when none are given. */
static int64_t as_bytes(PyObject *bytes, PyObject *ws) {
  const int64_t n = as_int(bytes); /* (-1 if it raised) */
  if (n != 0 || ws == Py_None || PyLong_Check(ws)) return n;
  PyObject *v = PyObject_GetAttr(ws, s_nbytes);
  if (!v) return -1;
  const int64_t m = as_int(v);
  Py_DECREF(v);
  return m;
}

static int count_ok(const char *name, Py_ssize_t got, Py_ssize_t want) {
  if (got == want) return 1;
  PyErr_Format(PyExc_TypeError, "%s takes %zd arguments (%zd given)", name, want, got);
  return 0;
}

/* Converts the arguments, calls without the interpreter's lock, returns the status. */
#define CALL(expr)                     \
  do {                                 \
    int st_;                           \
    if (PyErr_Occurred()) return NULL; \
    Py_BEGIN_ALLOW_THREADS st_ = expr; \
    Py_END_ALLOW_THREADS               \
    return PyLong_FromLong(st_);       \
  } while (0)
#define INT(i) const int64_t a##i = as_int(v[i])
#define PTR(i) void *const a##i = as_ptr(v[i])
#define DT(i) const int a##i = as_enum(v[i], dtypes)
#define LAY(i) const int a##i = as_enum(v[i], layouts)
/* A block's extent as an int, which no long integer wraps into. */
static int block(int64_t n) { return n == 1 || n == 128 ? (int)n : 0; }
#define DBL(i) const double a##i = PyErr_Occurred() ? 0.0 : PyFloat_AsDouble(v[i])

static PyObject *py_rmsnorm_quant(PyObject *self, PyObject *const *v, Py_ssize_t n) {
  if (!count_ok("rmsnorm_quant", n, 16)) return NULL;
  DT(0); INT(1); INT(2); PTR(3); INT(4); PTR(5); INT(6); PTR(7); DBL(8); PTR(9); INT(10); PTR(11); INT(12); PTR(13); PTR(14);
  void *const stream = as_stream(v[15]);
  CALL(rmsnorm_quant(a0, a1, a2, a3, a4, a5, a6, a7, a8, a9, a10, a11, a12, a13, a14, stream));
}
static PyObject *py_rmsnorm_backward(PyObject *self, PyObject *const *v, Py_ssize_t n) {
  if (!count_ok("rmsnorm_backward", n, 19)) return NULL;
  DT(0); DT(1); INT(2); INT(3); PTR(4); INT(5); PTR(6); INT(7); PTR(8); PTR(9); PTR(10); PTR(11); INT(12); PTR(13); INT(14);
  PTR(15); PTR(16);
  const int64_t bytes = as_bytes(v[17], v[16]);
  void *const stream = as_stream(v[18]);
  CALL(rmsnorm_backward(a0, a1, a2, a3, a4, a5, a6, a7, a8, a9, a10, a11, a12, a13, a14, a15, a16, bytes, stream));
}
static PyObject *py_quantize_rows(PyObject *self, PyObject *const *v, Py_ssize_t n) {
  if (!count_ok("quantize_rows", n, 9)) return NULL;
  DT(0); INT(1); INT(2); PTR(3); INT(4); PTR(5); INT(6); PTR(7);
  void *const stream = as_stream(v[8]);
  CALL(quantize_rows(a0, a1, a2, a3, a4, a5, a6, a7, stream));
}
static PyObject *py_dequantize_rows(PyObject *self, PyObject *const *v, Py_ssize_t n) {
  if (!count_ok("dequantize_rows", n, 9)) return NULL;
  DT(0); INT(1); INT(2); PTR(3); INT(4); PTR(5); PTR(6); INT(7);
  void *const stream = as_stream(v[8]);
  CALL(dequantize_rows(a0, a1, a2, a3, a4, a5, a6, a7, stream));
}
static PyObject *py_gemm_i8_scaled(PyObject *self, PyObject *const *v, Py_ssize_t n) {
  if (!count_ok("gemm_i8_scaled", n, 17)) return NULL;
  LAY(0); INT(1); INT(2); INT(3); PTR(4); INT(5); PTR(6); PTR(7); INT(8); PTR(9); PTR(10); PTR(11); INT(12); DT(13); PTR(14);
  const int64_t bytes = as_bytes(v[15], v[14]);
  void *const stream = as_stream(v[16]);
  CALL(gemm_i8_scaled(a0, a1, a2, a3, a4, a5, a6, a7, a8, a9, a10, a11, a12, a13, a14, bytes, stream));
}
static PyObject *py_gemm_grad_i8(PyObject *self, PyObject *const *v, Py_ssize_t n) {
  if (!count_ok("gemm_grad_i8", n, 18)) return NULL;
  DT(0); LAY(1); INT(2); INT(3); INT(4); PTR(5); INT(6); PTR(7); INT(8); PTR(9); PTR(10); PTR(11); INT(12); DT(13); DBL(14);
  PTR(15);
  const int64_t bytes = as_bytes(v[16], v[15]);
  void *const stream = as_stream(v[17]);
  CALL(gemm_grad_i8(a0, a1, a2, a3, a4, a5, a6, a7, a8, a9, a10, a11, a12, a13, a14, a15, bytes, stream));
}

static PyObject *py_quantize_blocks(PyObject *self, PyObject *const *v, Py_ssize_t n) {
  if (!count_ok("quantize_blocks", n, 13)) return NULL;
  DT(0); DT(1); INT(2); INT(3); INT(4); INT(5); PTR(6); INT(7); PTR(8); INT(9); PTR(10); INT(11);
  void *const stream = as_stream(v[12]);
  CALL(quantize_blocks(a0, a1, block(a2), block(a3), a4, a5, a6, a7, a8, a9, a10, a11, stream));
}
static PyObject *py_dequantize_blocks(PyObject *self, PyObject *const *v, Py_ssize_t n) {
  if (!count_ok("dequantize_blocks", n, 13)) return NULL;
  DT(0); DT(1); INT(2); INT(3); INT(4); INT(5); PTR(6); INT(7); PTR(8); INT(9); PTR(10); INT(11);
  void *const stream = as_stream(v[12]);
  CALL(dequantize_blocks(a0, a1, block(a2), block(a3), a4, a5, a6, a7, a8, a9, a10, a11, stream));
}
static PyObject *py_gemm_f8_blocks(PyObject *self, PyObject *const *v, Py_ssize_t n) {
  if (!count_ok("gemm_f8_blocks", n, 22)) return NULL;
  DT(0); DT(1); LAY(2); LAY(3); INT(4); INT(5); INT(6); INT(7); PTR(8); INT(9); PTR(10); INT(11); PTR(12); INT(13); PTR(14);
  INT(15); PTR(16); PTR(17); INT(18); DT(19); DBL(20);
  void *const stream = as_stream(v[21]);
  CALL(gemm_f8_blocks(a0, a1, a2, a3, block(a4), a5, a6, a7, a8, a9, a10, a11, a12, a13, a14, a15, a16, a17, a18, a19, a20,
                      stream));
}
static PyObject *py_gemm_grouped(PyObject *self, PyObject *const *v, Py_ssize_t n) {
  if (!count_ok("gemm_grouped", n, 16)) return NULL;
  DT(0); LAY(1); INT(2); INT(3); INT(4); INT(5); PTR(6); PTR(7); INT(8); PTR(9); INT(10); INT(11); PTR(12); INT(13); DT(14);
  void *const stream = as_stream(v[15]);
  CALL(gemm_grouped(a0, a1, a2, a3, a4, a5, a6, a7, a8, a9, a10, a11, a12, a13, a14, stream));
}
static PyObject *py_gemm_grouped_grad(PyObject *self, PyObject *const *v, Py_ssize_t n) {
  if (!count_ok("gemm_grouped_grad", n, 17)) return NULL;
  DT(0); INT(1); INT(2); INT(3); INT(4); PTR(5); PTR(6); INT(7); PTR(8); INT(9); PTR(10); PTR(11); INT(12); INT(13); DT(14);
  DBL(15);
  void *const stream = as_stream(v[16]);
  CALL(gemm_grouped_grad(a0, a1, a2, a3, a4, a5, a6, a7, a8, a9, a10, a11, a12, a13, a14, a15, stream));
}
static PyObject *py_gemm_grouped_f8_blocks(PyObject *self, PyObject *const *v, Py_ssize_t n) {
  if (!count_ok("gemm_grouped_f8_blocks", n, 22)) return NULL;
  DT(0); DT(1); LAY(2); INT(3); INT(4); INT(5); INT(6); PTR(7); PTR(8); INT(9); PTR(10); INT(11); PTR(12); INT(13); INT(14);
  PTR(15); INT(16); INT(17); PTR(18); INT(19); DT(20);
  void *const stream = as_stream(v[21]);
  CALL(gemm_grouped_f8_blocks(a0, a1, a2, a3, a4, a5, a6, a7, a8, a9, a10, a11, a12, a13, a14, a15, a16, a17, a18, a19, a20,
                              stream));
}

/* setup(dtypes, layouts, to_stream, raw_stream, raw_device), once, by the package. */
static PyObject *py_setup(PyObject *self, PyObject *args) {
  if (!PyArg_ParseTuple(args, "O!O!OOO", &PyDict_Type, &dtypes, &PyDict_Type, &layouts, &to_stream, &raw_stream, &raw_device))
    return NULL;
  Py_INCREF(dtypes);
  Py_INCREF(layouts);
  Py_INCREF(to_stream);
  Py_INCREF(raw_stream);
  Py_INCREF(raw_device);
  Py_RETURN_NONE;
}

#define ENTRY(f) {#f, (PyCFunction)(void (*)(void))py_##f, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {ENTRY(rmsnorm_quant), ENTRY(rmsnorm_backward), ENTRY(quantize_rows), ENTRY(dequantize_rows),
                                ENTRY(gemm_i8_scaled), ENTRY(gemm_grad_i8),
                                ENTRY(quantize_blocks), ENTRY(dequantize_blocks), ENTRY(gemm_f8_blocks), ENTRY(gemm_grouped),
                                ENTRY(gemm_grouped_grad), ENTRY(gemm_grouped_f8_blocks), {"setup", py_setup, METH_VARARGS, NULL}, {NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_mcgcall", NULL, -1, methods};

PyMODINIT_FUNC PyInit__mcgcall(void) {
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  s_nbytes = PyUnicode_InternFromString("nbytes");
  if (!s_data_ptr || !s_nbytes) return NULL;
  return PyModule_Create(&module);
}
