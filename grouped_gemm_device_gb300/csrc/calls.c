/* Python entry to the operators around the layer. Their smallest calls are bound by the host: a
 * foreign-function call of 14 arguments measured 1.3 us beside a kernel launch of 2.0 us, the
 * calls below a tenth of that. They take addresses and sizes as integers (None: NULL) and return
 * the status; bind() takes the library's functions, so that this module holds none itself. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "moegmm.h"

static void *ptr(PyObject *o) { return o == Py_None ? NULL : PyLong_AsVoidPtr(o); }
static int64_t i64(PyObject *o) { return PyLong_AsLongLong(o); }
static int32_t i32(PyObject *o) {
  const long long v = PyLong_AsLongLong(o);
  if (v < INT32_MIN || v > INT32_MAX) PyErr_SetString(PyExc_OverflowError, "not a 32-bit number");
  return (int32_t)v;
}
static size_t size(PyObject *o) { return PyLong_AsSize_t(o); }
static float f32(PyObject *o) { return (float)PyFloat_AsDouble(o); }

/* The library is called without the interpreter's lock: a launch waits when the GPU's queue is
 * full. */
#define RETURN_CALL(name, ...)                          \
  do {                                                  \
    moe_status_t st;                                    \
    if (PyErr_Occurred()) return NULL;                  \
    Py_BEGIN_ALLOW_THREADS st = name(__VA_ARGS__);      \
    Py_END_ALLOW_THREADS return PyLong_FromLong(st);    \
  } while (0)
#define ARGUMENTS(name, count)                                                        \
  if (!p_##name || n != count)                                                        \
    return PyErr_Format(PyExc_TypeError, #name ": not bound, or not %d arguments", count)

static __typeof__(&moe_router_loss_fwd) p_moe_router_loss_fwd;
static PyObject *py_moe_router_loss_fwd(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  ARGUMENTS(moe_router_loss_fwd, 15);
  void *v0 = ptr(a[0]); int64_t v1 = i64(a[1]); void *v2 = ptr(a[2]); void *v3 = ptr(a[3]);
  int32_t v4 = i32(a[4]); int32_t v5 = i32(a[5]); int32_t v6 = i32(a[6]); float v7 = f32(a[7]);
  void *v8 = ptr(a[8]); void *v9 = ptr(a[9]); void *v10 = ptr(a[10]); void *v11 = ptr(a[11]);
  void *v12 = ptr(a[12]); size_t v13 = size(a[13]); void *v14 = ptr(a[14]);
  RETURN_CALL(p_moe_router_loss_fwd, v0, v1, v2, v3, v4, v5, v6, v7, v8, v9, v10, v11, v12, v13,
               v14);
}
static __typeof__(&moe_router_loss_bwd) p_moe_router_loss_bwd;
static PyObject *py_moe_router_loss_bwd(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  ARGUMENTS(moe_router_loss_bwd, 16);
  void *v0 = ptr(a[0]); int64_t v1 = i64(a[1]); void *v2 = ptr(a[2]); void *v3 = ptr(a[3]);
  void *v4 = ptr(a[4]); void *v5 = ptr(a[5]); int32_t v6 = i32(a[6]); int32_t v7 = i32(a[7]);
  int32_t v8 = i32(a[8]); float v9 = f32(a[9]); void *v10 = ptr(a[10]); void *v11 = ptr(a[11]);
  void *v12 = ptr(a[12]); void *v13 = ptr(a[13]); int64_t v14 = i64(a[14]);
  void *v15 = ptr(a[15]);
  RETURN_CALL(p_moe_router_loss_bwd, v0, v1, v2, v3, v4, v5, v6, v7, v8, v9, v10, v11, v12, v13,
               v14, v15);
}
static __typeof__(&moe_layernorm_fwd) p_moe_layernorm_fwd;
static PyObject *py_moe_layernorm_fwd(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  ARGUMENTS(moe_layernorm_fwd, 14);
  void *v0 = ptr(a[0]); int64_t v1 = i64(a[1]); void *v2 = ptr(a[2]); void *v3 = ptr(a[3]);
  void *v4 = ptr(a[4]); int64_t v5 = i64(a[5]); void *v6 = ptr(a[6]); void *v7 = ptr(a[7]);
  int64_t v8 = i64(a[8]); int64_t v9 = i64(a[9]); float v10 = f32(a[10]);
  int32_t v11 = i32(a[11]); int32_t v12 = i32(a[12]); void *v13 = ptr(a[13]);
  RETURN_CALL(p_moe_layernorm_fwd, v0, v1, v2, v3, v4, v5, v6, v7, v8, v9, v10, v11, v12, v13);
}
static __typeof__(&moe_layernorm_bwd) p_moe_layernorm_bwd;
static PyObject *py_moe_layernorm_bwd(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  ARGUMENTS(moe_layernorm_bwd, 18);
  void *v0 = ptr(a[0]); int64_t v1 = i64(a[1]); void *v2 = ptr(a[2]); int64_t v3 = i64(a[3]);
  void *v4 = ptr(a[4]); void *v5 = ptr(a[5]); void *v6 = ptr(a[6]); void *v7 = ptr(a[7]);
  int64_t v8 = i64(a[8]); void *v9 = ptr(a[9]); void *v10 = ptr(a[10]); int64_t v11 = i64(a[11]);
  int64_t v12 = i64(a[12]); int32_t v13 = i32(a[13]); int32_t v14 = i32(a[14]);
  void *v15 = ptr(a[15]); size_t v16 = size(a[16]); void *v17 = ptr(a[17]);
  RETURN_CALL(p_moe_layernorm_bwd, v0, v1, v2, v3, v4, v5, v6, v7, v8, v9, v10, v11, v12, v13,
               v14, v15, v16, v17);
}
static __typeof__(&moe_grad_clip) p_moe_grad_clip;
static PyObject *py_moe_grad_clip(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  ARGUMENTS(moe_grad_clip, 10);
  int32_t v0 = i32(a[0]); void *v1 = ptr(a[1]); void *v2 = ptr(a[2]); void *v3 = ptr(a[3]);
  void *v4 = ptr(a[4]); float v5 = f32(a[5]); void *v6 = ptr(a[6]); void *v7 = ptr(a[7]);
  size_t v8 = size(a[8]); void *v9 = ptr(a[9]);
  RETURN_CALL(p_moe_grad_clip, v0, v1, v2, v3, v4, v5, v6, v7, v8, v9);
}
static __typeof__(&fp8_block_quantize_rows) p_fp8_block_quantize_rows;
static PyObject *py_fp8_block_quantize_rows(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  ARGUMENTS(fp8_block_quantize_rows, 13);
  void *v0 = ptr(a[0]); int64_t v1 = i64(a[1]); int64_t v2 = i64(a[2]); int64_t v3 = i64(a[3]);
  void *v4 = ptr(a[4]); int64_t v5 = i64(a[5]); void *v6 = ptr(a[6]); int64_t v7 = i64(a[7]);
  void *v8 = ptr(a[8]); int64_t v9 = i64(a[9]); void *v10 = ptr(a[10]); int64_t v11 = i64(a[11]);
  void *v12 = ptr(a[12]);
  RETURN_CALL(p_fp8_block_quantize_rows, v0, v1, v2, v3, v4, v5, v6, v7, v8, v9, v10, v11, v12);
}
static __typeof__(&fp8_block_quantize_weight) p_fp8_block_quantize_weight;
static PyObject *py_fp8_block_quantize_weight(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  ARGUMENTS(fp8_block_quantize_weight, 11);
  void *v0 = ptr(a[0]); int64_t v1 = i64(a[1]); int64_t v2 = i64(a[2]); int64_t v3 = i64(a[3]);
  void *v4 = ptr(a[4]); int64_t v5 = i64(a[5]); void *v6 = ptr(a[6]); void *v7 = ptr(a[7]);
  int64_t v8 = i64(a[8]); void *v9 = ptr(a[9]); void *v10 = ptr(a[10]);
  RETURN_CALL(p_fp8_block_quantize_weight, v0, v1, v2, v3, v4, v5, v6, v7, v8, v9, v10);
}
static __typeof__(&fp8_block_gemm) p_fp8_block_gemm;
static PyObject *py_fp8_block_gemm(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  ARGUMENTS(fp8_block_gemm, 17);
  void *v0 = ptr(a[0]); int64_t v1 = i64(a[1]); void *v2 = ptr(a[2]); int64_t v3 = i64(a[3]);
  void *v4 = ptr(a[4]); int64_t v5 = i64(a[5]); void *v6 = ptr(a[6]); int64_t v7 = i64(a[7]);
  int32_t v8 = i32(a[8]); void *v9 = ptr(a[9]); int64_t v10 = i64(a[10]);
  int32_t v11 = i32(a[11]); int64_t v12 = i64(a[12]); int64_t v13 = i64(a[13]);
  int64_t v14 = i64(a[14]); void *v15 = ptr(a[15]); void *v16 = ptr(a[16]);
  RETURN_CALL(p_fp8_block_gemm, v0, v1, v2, v3, v4, v5, v6, v7, v8, v9, v10, v11, v12, v13, v14,
               v15, v16);
}

/* bind(address, ...): the functions' addresses in the order of the table below. */
static PyObject *bind(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  if (n != 8) return PyErr_Format(PyExc_TypeError, "bind: 8 addresses");
  p_moe_router_loss_fwd = (__typeof__(p_moe_router_loss_fwd))ptr(a[0]);
  p_moe_router_loss_bwd = (__typeof__(p_moe_router_loss_bwd))ptr(a[1]);
  p_moe_layernorm_fwd = (__typeof__(p_moe_layernorm_fwd))ptr(a[2]);
  p_moe_layernorm_bwd = (__typeof__(p_moe_layernorm_bwd))ptr(a[3]);
  p_moe_grad_clip = (__typeof__(p_moe_grad_clip))ptr(a[4]);
  p_fp8_block_quantize_rows = (__typeof__(p_fp8_block_quantize_rows))ptr(a[5]);
  p_fp8_block_quantize_weight = (__typeof__(p_fp8_block_quantize_weight))ptr(a[6]);
  p_fp8_block_gemm = (__typeof__(p_fp8_block_gemm))ptr(a[7]);
  if (PyErr_Occurred()) return NULL;
  Py_RETURN_NONE;
}

#define METHOD(name) {#name, (PyCFunction)(void (*)(void))py_##name, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {
    METHOD(moe_router_loss_fwd),
    METHOD(moe_router_loss_bwd),
    METHOD(moe_layernorm_fwd),
    METHOD(moe_layernorm_bwd),
    METHOD(moe_grad_clip),
    METHOD(fp8_block_quantize_rows),
    METHOD(fp8_block_quantize_weight),
    METHOD(fp8_block_gemm),
    {"bind", (PyCFunction)(void (*)(void))bind, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_moecalls", NULL, -1, methods,
                                    NULL, NULL, NULL, NULL};
PyMODINIT_FUNC PyInit__moecalls(void) { return PyModule_Create(&module); }
