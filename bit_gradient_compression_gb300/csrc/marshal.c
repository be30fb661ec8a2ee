/*
 * Argument marshalling of the layer entry points for Python: what loco.py does
 * tensor by tensor, in C, because on small layers that took longer than the
 * kernels (a norm of one token of 4096: 10.1 us a call in Python, 6.4 us here).
 *
 * Every function takes tensors (or None) and integers, reads their shapes,
 * strides, types and addresses, calls the C entry point and returns its status.
 * Whatever is not as the entry point wants it - a shape, a stride, a type -
 * makes it return None without a call, and loco.py's own path then raises the
 * error with its text.  No torch headers: tensors are read through their Python
 * attributes.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

#include "loco.h"

static PyObject *s_shape, *s_stride, *s_data_ptr, *s_dtype, *s_is_contiguous;
static PyObject *t_f32, *t_bf16, *t_i8, *t_u8; /* torch's dtype objects, set by init() */
static double align_work;                        /* loco.py's ALIGN_WORK and ALIGN_ROWS, set by init() */
static int64_t align_rows;

/* One argument: 1 found, 0 not as wanted (the caller gives up), never an exception left behind. */
typedef struct {
  void* p;
  int64_t rows, cols, ld;
  int dtype; /* loco_dtype, or -1 */
} Mat;

static int address(PyObject* t, void** p) {
  PyObject* v = PyObject_CallMethodNoArgs(t, s_data_ptr);
  if (v == NULL) return 0;
  *p = (void*)PyLong_AsUnsignedLongLong(v);
  Py_DECREF(v);
  return !PyErr_Occurred();
}

static int type_of(PyObject* t) {
  PyObject* d = PyObject_GetAttr(t, s_dtype);
  if (d == NULL) return -1;
  const int r = d == t_f32 ? LOCO_F32 : d == t_bf16 ? LOCO_BF16 : -1;
  Py_DECREF(d);
  return r;
}

/* The integers of a tuple of n of them. */
static int ints(PyObject* v, Py_ssize_t n, int64_t* out) {
  int ok = v != NULL && PyTuple_Check(v) && PyTuple_GET_SIZE(v) == n;
  for (Py_ssize_t i = 0; ok && i < n; ++i) {
    out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(v, i));
    ok = !(out[i] == -1 && PyErr_Occurred());
  }
  Py_XDECREF(v);
  return ok;
}

/* A matrix; rows and cols are checked where they are not negative. */
static int mat(PyObject* t, int64_t rows, int64_t cols, Mat* m) {
  int64_t v[2];
  if (t == Py_None) {
    m->p = NULL, m->ld = 0, m->dtype = -1;
    return 1;
  }
  if (!ints(PyObject_GetAttr(t, s_shape), 2, v)) return 0;
  if ((rows >= 0 && v[0] != rows) || (cols >= 0 && v[1] != cols)) return 0;
  m->rows = v[0], m->cols = v[1];
  if (!ints(PyObject_CallMethodNoArgs(t, s_stride), 2, v)) return 0;
  if (v[1] != 1 && m->cols > 1) return 0;
  m->ld = m->rows <= 1 && v[0] < m->cols ? m->cols : v[0];
  m->dtype = type_of(t);
  return m->dtype >= 0 && address(t, &m->p);
}

/* A contiguous vector of count elements; dtype: as wanted, or -1 for either (which one goes to it). */
static int vec(PyObject* t, int64_t count, int* dtype, void** p) {
  int64_t v;
  *p = NULL;
  if (t == Py_None) return 1;
  if (!ints(PyObject_GetAttr(t, s_shape), 1, &v) || v != count) return 0;
  if (count > 1 && (!ints(PyObject_CallMethodNoArgs(t, s_stride), 1, &v) || v != 1)) return 0;
  const int d = type_of(t);
  if (d < 0 || (*dtype >= 0 && d != *dtype)) return 0;
  *dtype = d;
  return address(t, p);
}

/* Codes and scales of a checkpoint of [rows, cols]: contiguous, of the sizes the library states. */
static int part(PyObject* t, PyObject* want, int64_t size, void** p) {
  *p = NULL;
  if (t == Py_None) return 1;
  PyObject* d = PyObject_GetAttr(t, s_dtype);
  Py_XDECREF(d);
  if (d != want) return 0;
  PyObject* shape = PyObject_GetAttr(t, s_shape);
  if (shape == NULL || !PyTuple_Check(shape)) {
    Py_XDECREF(shape);
    return 0;
  }
  int64_t n = 1;
  for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(shape); ++i) n *= PyLong_AsLongLong(PyTuple_GET_ITEM(shape, i));
  Py_DECREF(shape);
  if (PyErr_Occurred() || n != size) return 0;
  PyObject* c = PyObject_CallMethodNoArgs(t, s_is_contiguous);
  Py_XDECREF(c);
  return c == Py_True && address(t, p);
}
static int ckpt(PyObject* codes, PyObject* scales, int64_t rows, int64_t cols, void** c, void** s) {
  const int64_t nb = (cols + LOCO_CKPT_BLOCK - 1) / LOCO_CKPT_BLOCK;
  return part(codes, t_i8, rows * nb * LOCO_CKPT_BLOCK, c) && part(scales, t_u8, rows * nb, s);
}
/* A workspace: a contiguous vector of bytes. */
static int bytes_of(PyObject* t, void** p, int64_t* n) {
  *p = NULL, *n = 0;
  if (t == Py_None) return 1;
  int64_t stride;
  if (!ints(PyObject_GetAttr(t, s_shape), 1, n) || !ints(PyObject_CallMethodNoArgs(t, s_stride), 1, &stride)) return 0;
  PyObject* d = PyObject_GetAttr(t, s_dtype);
  Py_XDECREF(d);
  return d == t_u8 && (stride == 1 || *n <= 1) && address(t, p);
}

/* An output of a product: a matrix of elements of so many bytes, a contiguous one as one row of bytes. */
typedef struct {
  const void* p;
  int64_t ld, rows, cols;
  int elem;
} Out;
static int size_of(int dtype) { return dtype == LOCO_BF16 ? 2 : 4; }
static Out out_mat(const Mat* m) { return (Out){m->p, m->ld, m->rows, m->cols, size_of(m->dtype)}; }
static Out out_row(const void* p, int64_t bytes) { return (Out){p, bytes, 1, bytes, 1}; }

/*
 * Copies the operands of a product over t rows to aligned rows where that pays (loco.py says when; least: the
 * fewest rows), in one piece of memory of alloc(bytes), which the caller releases after its call; without
 * alloc it gives up.  Operands stay as they lie where an output overlaps one: the call then refuses them.
 * Returns 1, or 0 to give up, or -1 for a failed copy with its status in *status.
 */
static int align(Mat* x, Mat* w, int64_t t, int64_t n, int64_t k, int64_t least, const Out* outs, int n_outs,
                 PyObject* alloc, loco_stream_t st, PyObject** held, int* status) {
  Mat* m[2] = {x, w};
  int64_t at[2] = {0, 0}, bytes = 0;
  *held = NULL;
  if (t < least || (double)t * (double)n * (double)k < align_work) return 1;
  for (int i = 0; i < 2; ++i) {
    if (m[i]->p == NULL || ((uintptr_t)m[i]->p % 16 == 0 && (m[i]->rows <= 1 || m[i]->ld % 8 == 0))) continue;
    for (int o = 0; o < n_outs; ++o)
      if (loco_matrices_overlap(m[i]->p, m[i]->ld, m[i]->rows, m[i]->cols, 2, outs[o].p, outs[o].ld, outs[o].rows,
                                outs[o].cols, outs[o].elem))
        return 1;
    at[i] = bytes;
    bytes += (m[i]->rows * ((m[i]->cols + 7) / 8 * 16) + 255) / 256 * 256;
    m[i]->dtype = -3; /* to be copied */
  }
  if (bytes == 0) return 1;
  if (alloc == Py_None) return 0;
  PyObject* size = PyLong_FromLongLong(bytes);
  *held = size == NULL ? NULL : PyObject_CallOneArg(alloc, size);
  Py_XDECREF(size);
  void* base;
  if (*held == Py_None) return 1; /* no memory: the product reads them as they lie */
  if (*held == NULL || !address(*held, &base)) return 0;
  for (int i = 0; i < 2; ++i) {
    if (m[i]->dtype != -3) continue;
    const int64_t pitch = (m[i]->cols + 7) / 8 * 8;
    *status = loco_linear_align(m[i]->p, m[i]->ld, m[i]->rows, m[i]->cols, (char*)base + at[i], pitch, st);
    if (*status != LOCO_OK) return -1;
    m[i]->p = (char*)base + at[i], m[i]->ld = pitch;
  }
  return 1;
}
/* The outputs follow alloc. */
#define ALIGN(x, w, t, n, k, least, alloc, ...)                                                                     \
  const Out outs[] = {__VA_ARGS__};                                                                                 \
  PyObject* held;                                                                                                   \
  int status;                                                                                                       \
  const int ready =                                                                                                 \
      align(x, w, t, n, k, least, outs, (int)(sizeof outs / sizeof outs[0]), alloc, st, &held, &status);            \
  if (ready < 1) {                                                                                                  \
    Py_XDECREF(held);                                                                                               \
    return ready < 0 ? PyLong_FromLong(status) : give_up();                                                         \
  }
#define CALL_ALIGNED(call)                       \
  Py_BEGIN_ALLOW_THREADS status = (call);        \
  Py_END_ALLOW_THREADS Py_XDECREF(held);         \
  return PyLong_FromLong(status)

/* The one type of two tensors, where -1 is a tensor that is not there; -2, and so on from there, where they differ. */
static int one(int a, int b) { return a == -1 ? b : b == -1 || a == b ? a : -2; }
static int or_f32(int d) { return d == -1 ? LOCO_F32 : d; }

static int64_t integer(PyObject* o) { return PyLong_AsLongLong(o); }
static PyObject* give_up(void) {
  PyErr_Clear();
  Py_RETURN_NONE;
}
#define WANT(cond) \
  if (!(cond) || PyErr_Occurred()) return give_up()
#define ARGS(count)                                                        \
  if (n != (count)) {                                                      \
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");         \
    return NULL;                                                           \
  }                                                                        \
  if (t_f32 == NULL) Py_RETURN_NONE
#define STREAM(o) ((loco_stream_t)(uintptr_t)PyLong_AsUnsignedLongLong(o))
#define CALL(call)                          \
  int status;                               \
  Py_BEGIN_ALLOW_THREADS status = (call);   \
  Py_END_ALLOW_THREADS return PyLong_FromLong(status)

/* (x, codes, scales, stream) */
static PyObject* ckpt_encode(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  ARGS(4);
  Mat x;
  void *c, *s;
  WANT(a[0] != Py_None && mat(a[0], -1, -1, &x) && ckpt(a[1], a[2], x.rows, x.cols, &c, &s));
  const loco_stream_t st = STREAM(a[3]);
  WANT(1);
  CALL(loco_ckpt_encode(x.p, x.dtype, x.ld, x.rows, x.cols, c, s, st));
}

/* (codes, scales, out, act, gamma, beta, stream) */
static PyObject* ckpt_decode(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  ARGS(7);
  Mat o;
  void *c, *s, *g, *b;
  int pd = -1;
  WANT(a[2] != Py_None && mat(a[2], -1, -1, &o) && ckpt(a[0], a[1], o.rows, o.cols, &c, &s));
  WANT(vec(a[4], o.cols, &pd, &g) && vec(a[5], o.cols, &pd, &b));
  const int act = (int)integer(a[3]);
  const loco_stream_t st = STREAM(a[6]);
  WANT(1);
  CALL(loco_ckpt_decode(c, s, o.rows, o.cols, act, g, b, or_f32(pd), o.p, o.dtype, o.ld, st));
}

/* (kind, eps, x, gamma, beta, y, mean, rstd, codes, scales, stream) */
static PyObject* norm_forward(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  ARGS(11);
  Mat x, y;
  void *g, *b, *m, *r, *c, *s;
  int pd = -1, f = LOCO_F32;
  WANT(a[2] != Py_None && a[5] != Py_None && mat(a[2], -1, -1, &x) && mat(a[5], x.rows, x.cols, &y));
  WANT(vec(a[3], x.cols, &pd, &g) && vec(a[4], x.cols, &pd, &b) && vec(a[6], x.rows, &f, &m) && vec(a[7], x.rows, &f, &r));
  WANT(ckpt(a[8], a[9], x.rows, x.cols, &c, &s));
  const loco_norm_config cfg = {(int32_t)integer(a[0]), (float)PyFloat_AsDouble(a[1]), x.dtype, y.dtype, or_f32(pd),
                                LOCO_F32};
  const loco_stream_t st = STREAM(a[10]);
  WANT(1);
  CALL(loco_norm_forward(&cfg, x.p, x.ld, x.rows, x.cols, g, b, y.p, y.ld, m, r, c, s, st));
}

/* (kind, eps, dy, gamma, rstd, dx, x, mean, codes, scales, residual, dgamma, dbeta, workspace, stream) */
static PyObject* norm_backward(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  ARGS(15);
  Mat dy, dx, x, res;
  void *g, *r, *m, *c, *s, *dg, *db, *w;
  int64_t nw;
  int pd = -1, gd = -1, f = LOCO_F32;
  WANT(a[2] != Py_None && a[5] != Py_None && mat(a[2], -1, -1, &dy) && mat(a[5], dy.rows, dy.cols, &dx));
  WANT(mat(a[6], dy.rows, dy.cols, &x) && mat(a[10], dy.rows, dy.cols, &res));
  WANT(vec(a[3], dy.cols, &pd, &g) && vec(a[4], dy.rows, &f, &r) && vec(a[7], dy.rows, &f, &m));
  WANT(vec(a[11], dy.cols, &gd, &dg) && vec(a[12], dy.cols, &gd, &db) && bytes_of(a[13], &w, &nw));
  WANT(ckpt(a[8], a[9], dy.rows, dy.cols, &c, &s));
  const int xd = one(one(x.dtype, res.dtype), dx.dtype);
  WANT(xd >= 0);
  const loco_norm_config cfg = {(int32_t)integer(a[0]), (float)PyFloat_AsDouble(a[1]), xd, dy.dtype, or_f32(pd),
                                or_f32(gd)};
  const loco_stream_t st = STREAM(a[14]);
  WANT(1);
  CALL(loco_norm_backward(&cfg, dy.p, dy.ld, x.p, x.ld, c, s, m, r, dy.rows, dy.cols, g, res.p, res.ld, dx.p, dx.ld, dg,
                          db, w, nw, st));
}

/* (x, w, y, act, bias, residual, codes, scales, stream, alloc) */
static PyObject* linear_forward(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  ARGS(10);
  Mat x, w, y, res;
  void *b, *c, *s;
  int pd = -1;
  WANT(a[0] != Py_None && a[1] != Py_None && a[2] != Py_None && mat(a[0], -1, -1, &x) && mat(a[1], -1, x.cols, &w));
  WANT(x.dtype == LOCO_BF16 && w.dtype == LOCO_BF16 && mat(a[2], x.rows, w.rows, &y) && mat(a[5], x.rows, w.rows, &res));
  WANT(vec(a[4], w.rows, &pd, &b) && ckpt(a[6], a[7], x.rows, w.rows, &c, &s));
  const loco_linear_config cfg = {(int32_t)integer(a[3]), one(y.dtype, res.dtype), or_f32(pd)};
  const loco_stream_t st = STREAM(a[8]);
  WANT(cfg.out_dtype >= 0);
  ALIGN(&x, &w, x.rows, w.rows, x.cols, align_rows, a[9], out_mat(&y), out_row(c, loco_ckpt_code_bytes(x.rows, w.rows)),
        out_row(s, loco_ckpt_scale_bytes(x.rows, w.rows)));
  CALL_ALIGNED(loco_linear_forward(&cfg, x.p, x.ld, w.p, w.ld, b, res.p, res.ld, x.rows, w.rows, x.cols, y.p, y.ld, c, s,
                                   st));
}

/* (dy, w, dx, act, codes, scales, residual, stream, alloc) */
static PyObject* linear_backward_input(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  ARGS(9);
  Mat dy, w, dx, res;
  void *c, *s;
  WANT(a[0] != Py_None && a[1] != Py_None && a[2] != Py_None && mat(a[0], -1, -1, &dy) && mat(a[1], dy.cols, -1, &w));
  WANT(dy.dtype == LOCO_BF16 && w.dtype == LOCO_BF16 && mat(a[2], dy.rows, w.cols, &dx) && mat(a[6], dy.rows, w.cols, &res));
  WANT(ckpt(a[4], a[5], dy.rows, w.cols, &c, &s));
  const loco_linear_config cfg = {(int32_t)integer(a[3]), one(dx.dtype, res.dtype), LOCO_F32};
  const loco_stream_t st = STREAM(a[7]);
  WANT(cfg.out_dtype >= 0);
  ALIGN(&dy, &w, dy.rows, dy.cols, w.cols, align_rows, a[8], out_mat(&dx));
  CALL_ALIGNED(loco_linear_backward_input(&cfg, dy.p, dy.ld, w.p, w.ld, c, s, res.p, res.ld, dy.rows, dy.cols, w.cols,
                                          dx.p, dx.ld, st));
}

/* (dy, dw, x, codes, scales, gamma, beta, db, workspace, stream, alloc) */
static PyObject* linear_backward_weight(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  ARGS(11);
  Mat dy, dw, x;
  void *c, *s, *g, *b, *db, *w;
  int64_t nw;
  int pd = -1, od;
  WANT(a[0] != Py_None && a[1] != Py_None && mat(a[0], -1, -1, &dy) && mat(a[1], dy.cols, -1, &dw));
  WANT(dy.dtype == LOCO_BF16 && mat(a[2], dy.rows, dw.cols, &x) && (x.p == NULL || x.dtype == LOCO_BF16));
  od = dw.dtype;
  WANT(ckpt(a[3], a[4], dy.rows, dw.cols, &c, &s) && vec(a[5], dw.cols, &pd, &g) && vec(a[6], dw.cols, &pd, &b));
  WANT(vec(a[7], dy.cols, &od, &db) && bytes_of(a[8], &w, &nw));
  const loco_linear_config cfg = {LOCO_ACT_NONE, od, or_f32(pd)};
  const loco_stream_t st = STREAM(a[9]);
  WANT(1);
  ALIGN(&dy, &x, dy.rows, dy.cols, dw.cols, 0, a[10], out_mat(&dw), out_row(db, dy.cols * size_of(od)),
        out_row(w, x.p == NULL && b != NULL ? loco_linear_workspace_bytes(dy.cols) : 0));
  CALL_ALIGNED(loco_linear_backward_weight(&cfg, dy.p, dy.ld, x.p, x.ld, c, s, g, b, dy.rows, dy.cols, dw.cols, dw.p,
                                           dw.ld, db, w, nw, st));
}

/* init(float32, bfloat16, int8, uint8, ALIGN_WORK, ALIGN_ROWS).  Until then every function returns None. */
static PyObject* init(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  if (n != 6) {
    PyErr_SetString(PyExc_TypeError, "four dtypes and two numbers");
    return NULL;
  }
  align_work = PyFloat_AsDouble(a[4]), align_rows = integer(a[5]);
  if (PyErr_Occurred()) return NULL;
  PyObject** to[4] = {&t_f32, &t_bf16, &t_i8, &t_u8};
  for (int i = 0; i < 4; ++i) {
    Py_INCREF(a[i]);
    Py_XSETREF(*to[i], a[i]);
  }
  Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
#define METHOD(f) {#f, (PyCFunction)(void (*)(void))f, METH_FASTCALL, NULL}
    METHOD(init),          METHOD(ckpt_encode),    METHOD(ckpt_decode),           METHOD(norm_forward),
    METHOD(norm_backward), METHOD(linear_forward), METHOD(linear_backward_input), METHOD(linear_backward_weight),
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__marshal(void) {
  s_shape = PyUnicode_InternFromString("shape");
  s_stride = PyUnicode_InternFromString("stride");
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  s_dtype = PyUnicode_InternFromString("dtype");
  s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
  return PyModule_Create(&module);
}
