/* mp_call.c — argument marshalling of the block operators for Python.
 *
 * A one-token norm takes 2.3 us on the GPU and 2.1 to launch; its arguments
 * checked in Python and converted by ctypes took 4.4 more, here 2.2.  The
 * functions make the same checks, through the tensors' own methods, and call the
 * library without the GIL.  They raise nothing: arguments that do not pass give
 * None, and the Python function of the same name says what is wrong.
 *
 *   bind(entry point addresses, (float32, float16, bfloat16), current_device, current_stream)
 *   <entry point>(its Python function's arguments, in order) -> mp_status | None
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "mpnum.h"

static mp_status (*norm_fp8)(const void*, const void*, mp_dtype, int64_t, int64_t, const void*, mp_dtype, float, void*,
                             void*, mp_dtype, int32_t, void*, float*, void*, float*, void*);
static mp_status (*norm_backward)(const void*, const void*, mp_dtype, int64_t, int64_t, const void*, const void*,
                                  const float*, const void*, mp_dtype, const float*, void*, void*, mp_dtype, void*,
                                  size_t, void*);
static mp_status (*glu_fp8)(const void*, const void*, int64_t, mp_dtype, int64_t, int64_t, void*, mp_dtype, int32_t,
                            void*, void*, float*, void*);
static mp_status (*glu_backward)(const void*, mp_dtype, int64_t, int64_t, const void*, const void*, int64_t,
                                 const void*, const float*, void*, void*, int64_t, void*);
static PyObject *dtypes[3], *current_device, *current_stream; /* dtypes by mp_dtype */
static PyObject *s_data_ptr, *s_get_device, *s_is_contiguous, *s_nbytes, *s_dtype, *s_shape, *s_stride, *s_cuda_stream;

static PyObject* method(PyObject* self, PyObject* name) {
  return PyObject_VectorcallMethod(name, &self, 1, NULL);
}
/* The integer in a new reference, which it releases; false if there is none. */
static int integer(PyObject* r, long long* out) {
  if (!r) return 0;
  *out = PyLong_Check(r) ? PyLong_AsLongLong(r) : -1;
  const int ok = PyLong_Check(r) && !PyErr_Occurred();
  Py_DECREF(r);
  return ok;
}
static int element_size(int dt) { return dt == MP_F32 ? 4 : 2; }

/* mp_dtype of a tensor, or -1. */
static int dtype_of(PyObject* t) {
  PyObject* d = PyObject_GetAttr(t, s_dtype);
  if (!d) return -1;
  int k = 0;
  while (k < 3 && d != dtypes[k]) ++k;
  Py_DECREF(d);
  return k < 3 ? k : -1;
}
/* What the arguments of a call have in common. */
typedef struct {
  long long dev, rows, cols, n, tile_bytes;
  int dt;
  void* stream;
} Call;

/* Fills it from the call's first tensor and its stream argument. */
static int begin(Call* c, PyObject* x, PyObject* stream) {
  long long dev;
  if (!integer(method(x, s_get_device), &c->dev) || c->dev < 0) return 0;
  if (!integer(PyObject_CallNoArgs(current_device), &dev) || dev != c->dev) return 0;
  PyObject* shape = PyObject_GetAttr(x, s_shape);
  if (!shape) return 0;
  int ok = PyTuple_Check(shape) && PyTuple_GET_SIZE(shape) == 2;
  if (ok) {
    c->rows = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, 0));
    c->cols = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, 1));
    ok = !PyErr_Occurred();
  }
  Py_DECREF(shape);
  if (!ok || (c->dt = dtype_of(x)) < 0) return 0;
  c->n = c->rows * c->cols;
  c->tile_bytes = 4 * c->rows * ((c->cols + 127) / 128);
  long long s;
  if (stream == Py_None) {
    PyObject* index = PyLong_FromLongLong(dev);
    if (!index) return 0;
    ok = integer(PyObject_CallOneArg(current_stream, index), &s);
    Py_DECREF(index);
  } else if (PyLong_Check(stream)) {
    s = PyLong_AsLongLong(stream);
    ok = !PyErr_Occurred();
  } else {
    ok = integer(PyObject_GetAttr(stream, s_cuda_stream), &s);
  }
  c->stream = (void*)(intptr_t)s;
  return ok;
}
/* Pointer of a contiguous tensor of at least `nbytes` on the call's device, of
 * type `dt` unless that is negative; NULL for None. */
static int pointer(const Call* c, PyObject* t, long long nbytes, int dt, void** out) {
  long long p, dev, have;
  *out = NULL;
  if (t == Py_None) return 1;
  if (!integer(method(t, s_data_ptr), &p) || !integer(method(t, s_get_device), &dev) || dev != c->dev) return 0;
  PyObject* dense = method(t, s_is_contiguous);
  if (!dense) return 0;
  const int ok = dense == Py_True;
  Py_DECREF(dense);
  if (!ok || !integer(PyObject_GetAttr(t, s_nbytes), &have) || have < nbytes) return 0;
  if (dt >= 0 && dtype_of(t) != dt) return 0;
  *out = (void*)(intptr_t)p;
  return 1;
}
/* Pointer and row distance of a [rows, cols] matrix of the call's type whose
 * rows are contiguous. */
static int matrix(const Call* c, PyObject* t, void** out, long long* ld) {
  long long p, dev, rows, cols, one;
  if (!integer(method(t, s_data_ptr), &p) || !integer(method(t, s_get_device), &dev) || dev != c->dev) return 0;
  if (dtype_of(t) != c->dt) return 0;
  PyObject *shape = PyObject_GetAttr(t, s_shape), *stride = shape ? method(t, s_stride) : NULL;
  int ok = stride && PyTuple_Check(shape) && PyTuple_Check(stride) && PyTuple_GET_SIZE(shape) == 2 &&
           PyTuple_GET_SIZE(stride) == 2;
  if (ok) {
    rows = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, 0));
    cols = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, 1));
    *ld = PyLong_AsLongLong(PyTuple_GET_ITEM(stride, 0));
    one = PyLong_AsLongLong(PyTuple_GET_ITEM(stride, 1));
    ok = !PyErr_Occurred() && rows == c->rows && cols == c->cols && (one == 1 || cols <= 1);
    if (rows <= 1) *ld = cols;
  }
  Py_XDECREF(shape);
  Py_XDECREF(stride);
  *out = (void*)(intptr_t)p;
  return ok;
}
static int pair(const Call* c, PyObject* a, PyObject* b, void** pa, void** pb, long long* ld) {
  long long ld_b;
  return matrix(c, a, pa, ld) && matrix(c, b, pb, &ld_b) && ld_b == *ld;
}
static int whole(PyObject* v, long* out) {
  *out = PyLong_Check(v) ? PyLong_AsLong(v) : -1;
  return PyLong_Check(v) && !PyErr_Occurred() && *out >= INT32_MIN && *out <= INT32_MAX;
}
static PyObject* pass(void) { /* the Python function says what is wrong */
  PyErr_Clear();
  Py_RETURN_NONE;
}

/* x, weight, y, y_scales, residual, h, rstd, ckpt, ckpt_scales, eps, fp8_dtype, scale_block, stream */
static PyObject* rmsnorm_residual_fp8_py(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  Call c;
  void *x, *w, *y, *ys, *r, *h, *rstd, *ck, *cs;
  long fp8, block;
  int wt;
  if (!norm_fp8 || n != 13 || !begin(&c, a[0], a[12]) || !whole(a[10], &fp8) || !whole(a[11], &block)) return pass();
  const double eps = PyFloat_AsDouble(a[9]);
  if (PyErr_Occurred() || (wt = dtype_of(a[1])) < 0) return pass();
  const long long bytes = c.n * element_size(c.dt);
  if (!pointer(&c, a[0], bytes, c.dt, &x) || !pointer(&c, a[1], c.cols * element_size(wt), wt, &w) ||
      !pointer(&c, a[2], c.n, -1, &y) || !pointer(&c, a[3], block == 32 ? c.n / 32 : c.tile_bytes, -1, &ys) ||
      !pointer(&c, a[4], bytes, c.dt, &r) || !pointer(&c, a[5], bytes, c.dt, &h) ||
      !pointer(&c, a[6], 4 * c.rows, MP_F32, &rstd) || !pointer(&c, a[7], c.n, -1, &ck) ||
      !pointer(&c, a[8], c.tile_bytes, MP_F32, &cs))
    return pass();
  mp_status st;
  Py_BEGIN_ALLOW_THREADS;
  st = norm_fp8(x, r, c.dt, c.rows, c.cols, w, wt, (float)eps, h, y, (mp_dtype)fp8, (int32_t)block, ys, rstd, ck, cs,
                c.stream);
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(st);
}

/* dy, weight, rstd, dx, dweight, workspace, h, ckpt, ckpt_scales, dh, stream */
static PyObject* rmsnorm_residual_backward_py(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  Call c;
  void *dy, *w, *rstd, *dx, *dw, *ws, *h, *ck, *cs, *dh;
  long long ws_bytes = 0;
  int wt, dwt;
  if (!norm_backward || n != 11 || !begin(&c, a[0], a[10]) || (wt = dtype_of(a[1])) < 0 || (dwt = dtype_of(a[4])) < 0)
    return pass();
  const long long bytes = c.n * element_size(c.dt);
  if (!pointer(&c, a[0], bytes, c.dt, &dy) || !pointer(&c, a[1], c.cols * element_size(wt), wt, &w) ||
      !pointer(&c, a[2], 4 * c.rows, MP_F32, &rstd) || !pointer(&c, a[3], bytes, c.dt, &dx) ||
      !pointer(&c, a[4], c.cols * element_size(dwt), dwt, &dw) || !pointer(&c, a[5], 0, -1, &ws) ||
      (ws && !integer(PyObject_GetAttr(a[5], s_nbytes), &ws_bytes)) || !pointer(&c, a[6], bytes, c.dt, &h) ||
      !pointer(&c, a[7], c.n, -1, &ck) || !pointer(&c, a[8], c.tile_bytes, MP_F32, &cs) ||
      !pointer(&c, a[9], bytes, c.dt, &dh))
    return pass();
  mp_status st;
  Py_BEGIN_ALLOW_THREADS;
  st = norm_backward(dy, dh, c.dt, c.rows, c.cols, h, ck, cs, w, wt, rstd, dx, dw, dwt, ws, (size_t)ws_bytes, c.stream);
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(st);
}

/* gate, up, y, y_scales, ckpt, ckpt_scales, fp8_dtype, scale_block, stream */
static PyObject* swiglu_fp8_py(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  Call c;
  void *g, *u, *y, *ys, *ck, *cs;
  long long ld;
  long fp8, block;
  if (!glu_fp8 || n != 9 || !begin(&c, a[0], a[8]) || !whole(a[6], &fp8) || !whole(a[7], &block) ||
      !pair(&c, a[0], a[1], &g, &u, &ld) || !pointer(&c, a[2], c.n, -1, &y) ||
      !pointer(&c, a[3], block == 32 ? c.n / 32 : c.tile_bytes, -1, &ys) || !pointer(&c, a[4], 2 * c.n, -1, &ck) ||
      !pointer(&c, a[5], 2 * c.tile_bytes, MP_F32, &cs))
    return pass();
  mp_status st;
  Py_BEGIN_ALLOW_THREADS;
  st = glu_fp8(g, u, ld, c.dt, c.rows, c.cols, y, (mp_dtype)fp8, (int32_t)block, ys, ck, cs, c.stream);
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(st);
}

/* dp, dgate, dup, gate, up, ckpt, ckpt_scales, stream */
static PyObject* swiglu_backward_py(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  Call c;
  void *dp, *dg, *du, *g = NULL, *u = NULL, *ck, *cs;
  long long ld, d_ld;
  if (!glu_backward || n != 8 || !begin(&c, a[0], a[7])) return pass();
  ld = c.cols;
  if ((a[3] == Py_None) != (a[4] == Py_None) || (a[3] != Py_None && !pair(&c, a[3], a[4], &g, &u, &ld)) ||
      !pair(&c, a[1], a[2], &dg, &du, &d_ld) || !pointer(&c, a[0], c.n * element_size(c.dt), c.dt, &dp) ||
      !pointer(&c, a[5], 2 * c.n, -1, &ck) || !pointer(&c, a[6], 2 * c.tile_bytes, MP_F32, &cs))
    return pass();
  mp_status st;
  Py_BEGIN_ALLOW_THREADS;
  st = glu_backward(dp, c.dt, c.rows, c.cols, g, u, ld, ck, cs, dg, du, d_ld, c.stream);
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(st);
}

static PyObject* bind(PyObject* self, PyObject* args) {
  (void)self;
  PyObject *t[3], *dev, *stream;
  unsigned long long f[4];
  if (!PyArg_ParseTuple(args, "(KKKK)(OOO)OO", &f[0], &f[1], &f[2], &f[3], &t[0], &t[1], &t[2], &dev, &stream))
    return NULL;
  for (int k = 0; k < 3; ++k) Py_XSETREF(dtypes[k], Py_NewRef(t[k]));
  Py_XSETREF(current_device, Py_NewRef(dev));
  Py_XSETREF(current_stream, Py_NewRef(stream));
  *(void**)&norm_fp8 = (void*)(uintptr_t)f[0];
  *(void**)&norm_backward = (void*)(uintptr_t)f[1];
  *(void**)&glu_fp8 = (void*)(uintptr_t)f[2];
  *(void**)&glu_backward = (void*)(uintptr_t)f[3];
  Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"bind", bind, METH_VARARGS, NULL},
    {"rmsnorm_residual_fp8", (PyCFunction)(void (*)(void))rmsnorm_residual_fp8_py, METH_FASTCALL, NULL},
    {"rmsnorm_residual_backward", (PyCFunction)(void (*)(void))rmsnorm_residual_backward_py, METH_FASTCALL, NULL},
    {"swiglu_fp8", (PyCFunction)(void (*)(void))swiglu_fp8_py, METH_FASTCALL, NULL},
    {"swiglu_backward", (PyCFunction)(void (*)(void))swiglu_backward_py, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_mpcall", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__mpcall(void) {
  struct {
    PyObject** at;
    const char* name;
  } names[] = {{&s_data_ptr, "data_ptr"}, {&s_get_device, "get_device"}, {&s_is_contiguous, "is_contiguous"},
               {&s_nbytes, "nbytes"},     {&s_dtype, "dtype"},           {&s_shape, "shape"},
               {&s_stride, "stride"},     {&s_cuda_stream, "cuda_stream"}};
  for (size_t k = 0; k < sizeof(names) / sizeof(names[0]); ++k)
    if (!(*names[k].at = PyUnicode_InternFromString(names[k].name))) return NULL;
  return PyModule_Create(&module);
}
