/* binding.c -- CPython entry to the calls whose host time matters (one small
 * kernel a call, in a loop over layers): chain_gb300._native.
 *
 * Argument marshalling only, as in the ctypes binding beside it: a tensor's
 * address, type, shape and strides are read through its Python methods, each
 * tensor is checked to lie on the current device and to be bf16 or f32 (int32
 * for index arrays), and the C ABI does every other check.  Building the same
 * descriptors through ctypes took 25 of a call's 35 to 50 us of host time. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "../../include/chain.h"

static PyObject *s_data_ptr, *s_dtype, *s_shape, *s_stride, *s_get_device, *s_is_contiguous;
static PyObject *t_bf16, *t_f32, *t_i32, *chain_error;

/* chain_gb300._native.setup(torch.bfloat16, torch.float32, torch.int32, ChainError) */
static PyObject *setup(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  if (n != 4) return PyErr_Format(PyExc_TypeError, "setup takes four arguments");
  Py_XSETREF(t_bf16, Py_NewRef(a[0]));
  Py_XSETREF(t_f32, Py_NewRef(a[1]));
  Py_XSETREF(t_i32, Py_NewRef(a[2]));
  Py_XSETREF(chain_error, Py_NewRef(a[3]));
  Py_RETURN_NONE;
}

/* Sizes out of a tuple of ints; -1 on error. */
static int read_sizes(PyObject *t, int64_t *out, int most) {
  if (!t) return -1;
  if (!PyTuple_Check(t)) {
    Py_DECREF(t);
    PyErr_SetString(PyExc_TypeError, "chain_gb300: not a tensor");
    return -1;
  }
  const Py_ssize_t n = PyTuple_GET_SIZE(t);
  for (Py_ssize_t i = 0; i < n && i < most; ++i) {
    out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(t, i));
    if (out[i] == -1 && PyErr_Occurred()) {
      Py_DECREF(t);
      return -1;
    }
  }
  Py_DECREF(t);
  return (int)n;
}

/* dev < 0: any. */
static int on_device(PyObject *t, long dev) {
  PyObject *g = PyObject_CallMethodNoArgs(t, s_get_device);
  if (!g) return -1;
  const long d = PyLong_AsLong(g);
  Py_DECREF(g);
  if (d == -1 && PyErr_Occurred()) return -1;
  if (d == dev || dev < 0) return 0;
  PyErr_Format(PyExc_ValueError, "chain_gb300: tensors must be on the current device, cuda:%ld", dev);
  return -1;
}

static int address(PyObject *t, void **out) {
  PyObject *p = PyObject_CallMethodNoArgs(t, s_data_ptr);
  if (!p) return -1;
  *out = PyLong_AsVoidPtr(p);
  Py_DECREF(p);
  return PyErr_Occurred() ? -1 : 0;
}

/* bf16 or f32 tensor; None gives a null descriptor where `optional`. */
static int tensor(PyObject *t, long dev, int optional, chain_tensor_t *d, chain_tensor_t **out) {
  *out = d;
  if (optional && t == Py_None) {
    *out = NULL;
    return 0;
  }
  PyObject *dt = PyObject_GetAttr(t, s_dtype);
  if (!dt) return -1;
  d->dtype = dt == t_bf16 ? CHAIN_BF16 : (dt == t_f32 ? CHAIN_F32 : -1);
  if (d->dtype < 0) PyErr_Format(PyExc_TypeError, "chain_gb300: bf16 or f32 tensors only, not %R", dt);
  Py_DECREF(dt);
  if (d->dtype < 0 || on_device(t, dev) || address(t, &d->ptr)) return -1;
  for (int i = 0; i < 4; ++i) d->shape[i] = d->stride[i] = 0;
  d->ndim = read_sizes(PyObject_GetAttr(t, s_shape), d->shape, 4);
  if (d->ndim < 0 || read_sizes(PyObject_CallMethodNoArgs(t, s_stride), d->stride, 4) < 0) return -1;
  if (d->ndim < 1 || d->ndim > 4) {
    PyErr_SetString(PyExc_ValueError, "chain_gb300: tensors must have 1 to 4 dimensions");
    return -1;
  }
  return 0;
}

/* int32 index array of `nd` dimensions, innermost contiguous */
static int indices(PyObject *t, long dev, const char *what, int nd, void **ptr, int64_t *shape,
                   int64_t *stride) {
  PyObject *dt = PyObject_GetAttr(t, s_dtype);
  if (!dt) return -1;
  const int ok = dt == t_i32;
  Py_DECREF(dt);
  if (on_device(t, dev) || address(t, ptr)) return -1;
  const int n = read_sizes(PyObject_GetAttr(t, s_shape), shape, nd);
  if (n < 0 || read_sizes(PyObject_CallMethodNoArgs(t, s_stride), stride, nd) < 0) return -1;
  if (!ok || n != nd) {
    PyErr_Format(PyExc_ValueError, "%s must be a CUDA int32 tensor of %d dimension%s", what, nd,
                 nd > 1 ? "s" : "");
    return -1;
  }
  if (shape[nd - 1] > 1 && stride[nd - 1] != 1) {
    PyErr_Format(PyExc_ValueError, "%s must be contiguous", what);
    return -1;
  }
  return 0;
}

/* 1 or 0; -1 on error */
static int is_dense(PyObject *t) {
  PyObject *c = PyObject_CallMethodNoArgs(t, s_is_contiguous);
  if (!c) return -1;
  const int dense = PyObject_IsTrue(c);
  Py_DECREF(c);
  return dense;
}

/* positions: one int32 for each of `tokens`, any shape, or None */
static int positions(PyObject *t, long dev, int64_t tokens, void **ptr) {
  *ptr = NULL;
  if (t == Py_None) return 0;
  PyObject *dt = PyObject_GetAttr(t, s_dtype);
  if (!dt) return -1;
  const int ok = dt == t_i32;
  Py_DECREF(dt);
  if (!ok) {
    PyErr_SetString(PyExc_ValueError, "positions must be a CUDA int32 tensor");
    return -1;
  }
  if (on_device(t, dev) || address(t, ptr)) return -1;
  const int dense = is_dense(t);
  if (dense < 0) return -1;
  int64_t shape[8];
  const int n = read_sizes(PyObject_GetAttr(t, s_shape), shape, 8);
  if (n < 0) return -1;
  int64_t count = 1;
  for (int i = 0; i < n && i < 8; ++i) count *= shape[i];
  if (dense != 1 || n > 8) {
    PyErr_SetString(PyExc_ValueError, "positions must be contiguous");
    return -1;
  }
  if (count != tokens) {
    PyErr_SetString(PyExc_ValueError, "positions must hold one position for each token");
    return -1;
  }
  return 0;
}

typedef struct {
  void *cu, *lens, *table;
  int64_t stride;
  int batch, max_pages;
} paged_t;

static int paged(PyObject *cu, PyObject *lens, PyObject *table, long dev, paged_t *p) {
  int64_t sc[2], sl[2], st[2], tc[2], tl[2], tt[2];
  if (indices(cu, dev, "cu_seqlens", 1, &p->cu, sc, tc) || indices(lens, dev, "kv_lens", 1, &p->lens, sl, tl) ||
      indices(table, dev, "page_table", 2, &p->table, st, tt))
    return -1;
  if (sc[0] != sl[0] + 1 || st[0] != sl[0] || sl[0] > 0x7fffffff || st[1] > 0x7fffffff) {
    PyErr_SetString(PyExc_ValueError, "cu_seqlens [batch + 1], kv_lens [batch] and page_table [batch][max_pages] "
                                      "must agree on the batch");
    return -1;
  }
  p->batch = (int)sl[0];
  p->max_pages = (int)st[1];
  p->stride = p->batch > 1 ? tt[0] : st[1];
  return 0;
}

/* A workspace: any contiguous tensor; its bytes are given beside it. */
static int workspace(PyObject *t, long dev, void **ptr) {
  if (on_device(t, dev) || address(t, ptr)) return -1;
  const int dense = is_dense(t);
  if (dense == 0) PyErr_SetString(PyExc_ValueError, "the workspace must be contiguous");
  return dense == 1 ? 0 : -1;
}

/* Each call below is made without the interpreter's lock: a launch waits while the queue of the
 * stream is full, and the program's other threads go on meanwhile. */
static PyObject *done(int rc, const char *what) {
  if (rc == CHAIN_OK) Py_RETURN_NONE;
  PyObject *e = PyObject_CallFunction(chain_error, "is", rc, what);
  if (e) {
    PyErr_SetObject(chain_error, e);
    Py_DECREF(e);
  }
  return NULL;
}

static int count(Py_ssize_t n, Py_ssize_t want, const char *what) {
  if (n == want) return 0;
  PyErr_Format(PyExc_TypeError, "%s: %zd arguments, %zd wanted", what, n, want);
  return -1;
}

/* Every call's last two arguments: the current device and its stream's handle. */
#define DEV_STREAM(at)                        \
  const long dev = PyLong_AsLong(a[at]);      \
  void *stream = PyLong_AsVoidPtr(a[(at) + 1]); \
  if (PyErr_Occurred()) return NULL
#define TENSOR(i, name)          \
  chain_tensor_t name##_, *name; \
  if (tensor(a[i], dev, 0, &name##_, &name)) return NULL
#define OPTIONAL(i, name)        \
  chain_tensor_t name##_, *name; \
  if (tensor(a[i], dev, 1, &name##_, &name)) return NULL

static int64_t tokens_of(const chain_tensor_t *q) {
  int64_t t = 1;
  for (int i = 0; i + 2 < q->ndim; ++i) t *= q->shape[i];
  return t;
}

static PyObject *qk_norm_rope(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  if (count(n, 12, "chain_qk_norm_rope")) return NULL;
  DEV_STREAM(10);
  TENSOR(0, Q);
  TENSOR(1, K);
  TENSOR(2, gq);
  TENSOR(3, gk);
  OPTIONAL(4, w);
  TENSOR(8, Qo);
  TENSOR(9, Ko);
  void *pos;
  if (positions(a[5], dev, tokens_of(Q), &pos)) return NULL;
  const double eps = PyFloat_AsDouble(a[6]);
  const long pairs = PyLong_AsLong(a[7]);
  if (PyErr_Occurred()) return NULL;
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = chain_qk_norm_rope(Q, K, gq, gk, w, (const int32_t *)pos, (float)eps, (int)pairs, Qo, Ko, stream);
  Py_END_ALLOW_THREADS
  return done(rc, "chain_qk_norm_rope");
}

static PyObject *qk_norm_rope_bwd(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  if (count(n, 18, "chain_qk_norm_rope_bwd")) return NULL;
  DEV_STREAM(16);
  TENSOR(0, dQo);
  TENSOR(1, dKo);
  TENSOR(2, Q);
  TENSOR(3, K);
  TENSOR(4, gq);
  TENSOR(5, gk);
  OPTIONAL(6, w);
  TENSOR(10, dQ);
  TENSOR(11, dK);
  TENSOR(12, dgq);
  TENSOR(13, dgk);
  void *pos, *ws;
  if (positions(a[7], dev, tokens_of(Q), &pos) || workspace(a[14], dev, &ws)) return NULL;
  const double eps = PyFloat_AsDouble(a[8]);
  const long pairs = PyLong_AsLong(a[9]);
  const size_t bytes = PyLong_AsSize_t(a[15]);
  if (PyErr_Occurred()) return NULL;
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = chain_qk_norm_rope_bwd(dQo, dKo, Q, K, gq, gk, w, (const int32_t *)pos, (float)eps, (int)pairs, dQ, dK, dgq,
                              dgk, ws, bytes, stream);
  Py_END_ALLOW_THREADS
  return done(rc, "chain_qk_norm_rope_bwd");
}

/* Sizes only: Q may lie on any device. */
static PyObject *qk_norm_rope_bwd_workspace_size(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  if (count(n, 1, "chain_qk_norm_rope_bwd_workspace_size")) return NULL;
  chain_tensor_t q, *Q;
  if (tensor(a[0], -1, 0, &q, &Q)) return NULL;
  return PyLong_FromSize_t(chain_qk_norm_rope_bwd_workspace_size(Q));
}

static PyObject *paged_append(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  if (count(n, 9, "chain_paged_append")) return NULL;
  DEV_STREAM(7);
  TENSOR(0, K);
  TENSOR(1, V);
  TENSOR(5, Kc);
  TENSOR(6, Vc);
  paged_t p;
  if (paged(a[2], a[3], a[4], dev, &p)) return NULL;
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = chain_paged_append(K, V, (const int32_t *)p.cu, (const int32_t *)p.lens, (const int32_t *)p.table, p.stride,
                          p.batch, p.max_pages, Kc, Vc, stream);
  Py_END_ALLOW_THREADS
  return done(rc, "chain_paged_append");
}

static PyObject *qk_norm_rope_append(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  if (count(n, 16, "chain_qk_norm_rope_append")) return NULL;
  DEV_STREAM(14);
  TENSOR(0, Q);
  TENSOR(1, K);
  TENSOR(2, V);
  TENSOR(3, gq);
  TENSOR(4, gk);
  OPTIONAL(5, w);
  TENSOR(11, Kc);
  TENSOR(12, Vc);
  TENSOR(13, Qo);
  paged_t p;
  if (paged(a[8], a[9], a[10], dev, &p)) return NULL;
  const double eps = PyFloat_AsDouble(a[6]);
  const long pairs = PyLong_AsLong(a[7]);
  if (PyErr_Occurred()) return NULL;
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = chain_qk_norm_rope_append(Q, K, V, gq, gk, w, (float)eps, (int)pairs, (const int32_t *)p.cu,
                                 (const int32_t *)p.lens, (const int32_t *)p.table, p.stride, p.batch, p.max_pages,
                                 Kc, Vc, Qo, stream);
  Py_END_ALLOW_THREADS
  return done(rc, "chain_qk_norm_rope_append");
}

static PyObject *fwd_paged(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  if (count(n, 14, "chain_fwd_paged")) return NULL;
  DEV_STREAM(12);
  TENSOR(0, Q);
  TENSOR(1, Kc);
  TENSOR(2, Vc);
  TENSOR(8, O);
  TENSOR(9, LSE);
  paged_t p;
  void *ws;
  if (paged(a[3], a[4], a[5], dev, &p) || workspace(a[10], dev, &ws)) return NULL;
  const long mask = PyLong_AsLong(a[6]);
  const double scale = PyFloat_AsDouble(a[7]);
  const size_t bytes = PyLong_AsSize_t(a[11]);
  if (PyErr_Occurred()) return NULL;
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = chain_fwd_paged(Q, Kc, Vc, (const int32_t *)p.cu, (const int32_t *)p.lens, (const int32_t *)p.table,
                       p.stride, p.batch, p.max_pages, (int)mask, (float)scale, O, LSE, ws, bytes, stream);
  Py_END_ALLOW_THREADS
  return done(rc, "chain_fwd_paged");
}

#define METHOD(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {METHOD(setup),        METHOD(qk_norm_rope),        METHOD(qk_norm_rope_bwd),
                                METHOD(paged_append), METHOD(qk_norm_rope_append), METHOD(fwd_paged),
                                METHOD(qk_norm_rope_bwd_workspace_size),
                                {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__native(void) {
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  s_dtype = PyUnicode_InternFromString("dtype");
  s_shape = PyUnicode_InternFromString("shape");
  s_stride = PyUnicode_InternFromString("stride");
  s_get_device = PyUnicode_InternFromString("get_device");
  s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
  return PyModule_Create(&module);
}
