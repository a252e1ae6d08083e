/*
 * The binding's calls that a decode step makes, as a CPython extension: the same checks and
 * arguments as the Python functions of the same names in _lib.py, which stay the reference and are
 * used where this extension has not been built. Marshalling a call in Python takes 3 to 8 us, more
 * than most of these calls' kernels run for few tokens; here it takes about 1 us.
 *
 * bind() receives the addresses of the C entry points of the loaded library, so that the release and
 * the debug build both work.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <limits.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/moe_gg.h"

#define DTYPE_F32 MOE_DTYPE_F32
#define DTYPE_BF16 MOE_DTYPE_BF16

#define FUNCTIONS(X)                                                                                         \
  X(moe_layer_norm_fwd) X(moe_layer_norm_bwd) X(moe_gate_fwd) X(moe_gate_bwd) X(moe_mx4_quantize_rows)        \
  X(moe_mx4_dequantize_rows) X(moe_permute_mxfp4) X(moe_grouped_swiglu_fwd_mxfp4) X(moe_unpermute_combine)    \
  X(moe_route_offsets)
#define DECLARE(f) static __typeof__(&f) p_##f;
FUNCTIONS(DECLARE)

static PyObject *g_bf16, *g_f32, *g_i32, *g_u8, *g_bool; /* torch dtypes */
static PyObject *g_raise, *g_raw_stream, *g_get_device;
static PyObject *s_is_cuda, *s_is_contiguous, *s_data_ptr, *s_dtype, *s_numel, *s_element_size, *s_shape, *s_stride,
    *s_cuda_stream;

/* ------------------------------------------------------------------ arguments */
/* Positional and keyword arguments in the order of `names`; NULL entries of optional ones become None. */
static int collect(const char* fn, const char* const* names, int n, int required, PyObject* const* args,
                   Py_ssize_t nargs, PyObject* kwnames, PyObject** out) {
  if (nargs > n) {
    PyErr_Format(PyExc_TypeError, "%s() takes at most %d arguments (%zd given)", fn, n, nargs);
    return -1;
  }
  for (int i = 0; i < n; ++i) out[i] = i < nargs ? args[i] : NULL;
  const Py_ssize_t nk = kwnames ? PyTuple_GET_SIZE(kwnames) : 0;
  for (Py_ssize_t k = 0; k < nk; ++k) {
    PyObject* key = PyTuple_GET_ITEM(kwnames, k);
    int i = 0;
    while (i < n && PyUnicode_CompareWithASCIIString(key, names[i]) != 0) ++i;
    if (i == n || out[i] != NULL) {
      PyErr_Format(PyExc_TypeError, "%s() got an unexpected or repeated argument '%U'", fn, key);
      return -1;
    }
    out[i] = args[nargs + k];
  }
  for (int i = 0; i < n; ++i) {
    if (out[i] != NULL) continue;
    if (i < required) {
      PyErr_Format(PyExc_TypeError, "%s() missing argument '%s'", fn, names[i]);
      return -1;
    }
    out[i] = Py_None;
  }
  return 0;
}

static int as_int(PyObject* o, int* v) {
  const long x = PyLong_AsLong(o);
  if (x == -1 && PyErr_Occurred()) return -1;
  if (x < INT_MIN || x > INT_MAX) {
    PyErr_SetString(PyExc_OverflowError, "an argument does not fit a C int");
    return -1;
  }
  *v = (int)x;
  return 0;
}

static int flag(PyObject* o) { /* a bool result: 1, 0, -1 on error; takes the reference */
  if (o == NULL) return -1;
  const int r = o == Py_True ? 1 : o == Py_False ? 0 : PyObject_IsTrue(o);
  Py_DECREF(o);
  return r;
}

static int is_plain(PyObject* t) { /* on the GPU and contiguous */
  const int c = flag(PyObject_GetAttr(t, s_is_cuda));
  return c <= 0 ? c : flag(PyObject_CallMethodNoArgs(t, s_is_contiguous));
}

static int number(PyObject* t, PyObject* method, long long* v) {
  PyObject* o = PyObject_CallMethodNoArgs(t, method);
  if (o == NULL) return -1;
  *v = PyLong_AsLongLong(o);
  Py_DECREF(o);
  return *v == -1 && PyErr_Occurred() ? -1 : 0;
}

static int address(PyObject* t, void** p) {
  PyObject* o = PyObject_CallMethodNoArgs(t, s_data_ptr);
  if (o == NULL) return -1;
  *p = PyLong_AsVoidPtr(o);
  Py_DECREF(o);
  return *p == NULL && PyErr_Occurred() ? -1 : 0;
}

/* None, or a contiguous CUDA tensor */
static int plain(PyObject* t, void** p) {
  *p = NULL;
  if (t == Py_None) return 0;
  const int ok = is_plain(t);
  if (ok < 0) return -1;
  if (!ok) {
    PyErr_SetString(PyExc_ValueError, "tensors passed to the library must be contiguous CUDA tensors");
    return -1;
  }
  return address(t, p);
}

static PyObject* dtype_of(PyObject* t) { /* borrowed: torch keeps its dtypes */
  PyObject* d = PyObject_GetAttr(t, s_dtype);
  Py_XDECREF(d);
  return d;
}

/* None, or a contiguous CUDA tensor of a type with at least `numel` elements */
static int typed(PyObject* t, PyObject* dtype, long long numel, const char* name, void** p) {
  *p = NULL;
  if (t == Py_None) return 0;
  PyObject* d = dtype_of(t);
  long long n = 0;
  if (d == NULL || number(t, s_numel, &n) < 0) return -1;
  int ok = d == dtype && n >= numel;
  if (ok) ok = is_plain(t);
  if (ok < 0) return -1;
  if (!ok) {
    PyErr_Format(PyExc_ValueError, "%s: expected a contiguous CUDA tensor of at least %lld elements of %S", name, numel, dtype);
    return -1;
  }
  return address(t, p);
}

static int bytes_of(PyObject* t, size_t* b) {
  long long n = 0, e = 0;
  *b = 0;
  if (t == Py_None) return 0;
  if (number(t, s_numel, &n) < 0 || number(t, s_element_size, &e) < 0) return -1;
  *b = (size_t)(n * e);
  return 0;
}

/* pointer and row pitch of a [>= T, width] tensor whose rows are contiguous */
static int rows(PyObject* t, int T, int width, void** p, long long* ld) {
  PyObject* shape = PyObject_GetAttr(t, s_shape);
  if (shape == NULL) return -1;
  long long s0 = -1, s1 = -1;
  if (PyTuple_Check(shape) && PyTuple_GET_SIZE(shape) == 2) {
    s0 = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, 0));
    s1 = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, 1));
  }
  Py_DECREF(shape);
  if (PyErr_Occurred()) return -1;
  int ok = flag(PyObject_GetAttr(t, s_is_cuda));
  if (ok < 0) return -1;
  ok = ok && s0 >= T && s1 == width;
  *ld = width;
  if (ok) {
    const int c = flag(PyObject_CallMethodNoArgs(t, s_is_contiguous));
    if (c < 0) return -1;
    if (!c) {
      PyObject* st = PyObject_CallMethodNoArgs(t, s_stride);
      if (st == NULL) return -1;
      const long long t0 = PyLong_AsLongLong(PyTuple_GET_ITEM(st, 0)), t1 = PyLong_AsLongLong(PyTuple_GET_ITEM(st, 1));
      Py_DECREF(st);
      if (PyErr_Occurred()) return -1;
      ok = t1 == 1 || width <= 1;
      if (T > 1) *ld = t0;
    }
  }
  if (!ok) {
    PyErr_Format(PyExc_ValueError, "expected a CUDA tensor of at least %d rows of %d contiguous elements", T, width);
    return -1;
  }
  return address(t, p);
}

static int element_type(PyObject* t, int* v) {
  PyObject* d = dtype_of(t);
  if (d == NULL) return -1;
  if (d == g_bf16) *v = DTYPE_BF16;
  else if (d == g_f32) *v = DTYPE_F32;
  else {
    PyErr_Format(PyExc_ValueError, "expected a bfloat16 or float32 tensor, not %S", d);
    return -1;
  }
  return 0;
}

static int same_type(PyObject* a, PyObject* b, const char* what) {
  PyObject *x = dtype_of(a), *y = dtype_of(b);
  if (x == NULL || y == NULL) return -1;
  if (x == y) return 0;
  PyErr_SetString(PyExc_ValueError, what);
  return -1;
}

static int as_stream(PyObject* o, moe_stream_t* s) {
  PyObject* v;
  if (o == Py_None) {
    PyObject* dev = PyObject_CallNoArgs(g_get_device);
    if (dev == NULL) return -1;
    v = PyObject_CallOneArg(g_raw_stream, dev);
    Py_DECREF(dev);
  } else {
    v = PyObject_GetAttr(o, s_cuda_stream);
  }
  if (v == NULL) return -1;
  *s = (moe_stream_t)PyLong_AsVoidPtr(v);
  Py_DECREF(v);
  return *s == NULL && PyErr_Occurred() ? -1 : 0;
}

static PyObject* finish(const char* fn, moe_status_t st) {
  if (st == MOE_OK) Py_RETURN_NONE;
  PyObject* r = PyObject_CallFunction(g_raise, "si", fn, (int)st);
  Py_XDECREF(r);
  if (!PyErr_Occurred()) PyErr_Format(PyExc_RuntimeError, "%s returned %d", fn, (int)st);
  return NULL;
}

/* the weights' type: all bf16 or all fp32, [d] each; fp32 when there are none */
static int weight_type(PyObject* const* w, int n, int d, int* v) {
  PyObject *one = NULL, *first = NULL;
  *v = DTYPE_F32;
  for (int i = 0; i < n; ++i) {
    if (w[i] == Py_None) continue;
    long long numel = 0;
    PyObject* t = dtype_of(w[i]);
    if (t == NULL || number(w[i], s_numel, &numel) < 0) return -1;
    if (numel != d || (one != NULL && t != one)) {
      PyErr_Format(PyExc_ValueError, "the weights have to be [%d] and of one type", d);
      return -1;
    }
    one = t;
    first = w[i];
  }
  return first == NULL ? 0 : element_type(first, v);
}

#define ARGS PyObject *self, PyObject *const *args, Py_ssize_t nargs, PyObject *kwnames
#define COLLECT(fn, required, ...)                                                        \
  static const char* const names[] = {__VA_ARGS__};                                       \
  enum { N = sizeof(names) / sizeof(names[0]) };                                          \
  PyObject* a[N];                                                                         \
  (void)self;                                                                             \
  if (collect(fn, names, N, required, args, nargs, kwnames, a) < 0) return NULL

/* ------------------------------------------------------------------ the calls */
static PyObject* layer_norm_fwd(ARGS) {
  COLLECT("moe_layer_norm_fwd", 7, "x", "gamma", "beta", "T", "d", "eps", "y", "mean", "rstd", "stream");
  int T, d, dt, wt;
  void *x, *y, *gamma, *beta, *mean, *rstd;
  long long ldx, ldy;
  moe_stream_t s;
  if (as_int(a[3], &T) < 0 || as_int(a[4], &d) < 0) return NULL;
  const double eps = PyFloat_AsDouble(a[5]);
  if (eps == -1.0 && PyErr_Occurred()) return NULL;
  if (rows(a[0], T, d, &x, &ldx) < 0 || rows(a[6], T, d, &y, &ldy) < 0 ||
      same_type(a[0], a[6], "y has to have x's type") < 0 || element_type(a[0], &dt) < 0 || plain(a[1], &gamma) < 0 ||
      plain(a[2], &beta) < 0 || weight_type(a + 1, 2, d, &wt) < 0 || typed(a[7], g_f32, T, "mean", &mean) < 0 ||
      typed(a[8], g_f32, T, "rstd", &rstd) < 0 || as_stream(a[9], &s) < 0)
    return NULL;
  return finish("moe_layer_norm_fwd", p_moe_layer_norm_fwd(x, dt, ldx, gamma, beta, wt, T, d, (float)eps, y, ldy, mean, rstd, s));
}

static PyObject* layer_norm_bwd(ARGS) {
  COLLECT("moe_layer_norm_bwd", 8, "dy", "x", "gamma", "mean", "rstd", "T", "d", "dx", "dgamma", "dbeta", "ws", "stream");
  int T, d, dt, wt;
  void *dy, *x, *dx, *gamma, *mean, *rstd, *dgamma, *dbeta, *ws;
  long long lddy, ldx, lddx;
  size_t n;
  moe_stream_t s;
  static const char* const types = "x, dy and dx have to have one type";
  if (as_int(a[5], &T) < 0 || as_int(a[6], &d) < 0 || rows(a[0], T, d, &dy, &lddy) < 0 || rows(a[1], T, d, &x, &ldx) < 0 ||
      rows(a[7], T, d, &dx, &lddx) < 0 || same_type(a[0], a[1], types) < 0 || same_type(a[1], a[7], types) < 0 ||
      element_type(a[1], &dt) < 0 || plain(a[2], &gamma) < 0 || weight_type(a + 2, 1, d, &wt) < 0 ||
      typed(a[3], g_f32, T, "mean", &mean) < 0 || typed(a[4], g_f32, T, "rstd", &rstd) < 0 ||
      typed(a[8], g_f32, d, "dgamma", &dgamma) < 0 || typed(a[9], g_f32, d, "dbeta", &dbeta) < 0 ||
      plain(a[10], &ws) < 0 || bytes_of(a[10], &n) < 0 || as_stream(a[11], &s) < 0)
    return NULL;
  return finish("moe_layer_norm_bwd", p_moe_layer_norm_bwd(dy, lddy, x, ldx, dt, gamma, wt, mean, rstd, T, d, dx, lddx, dgamma,
                                                           dbeta, ws, n, s));
}

static PyObject* gate_fwd(ARGS) {
  COLLECT("moe_gate_fwd", 8, "logits", "token_mask", "T", "top_k", "E", "flags", "ids", "weights", "lse", "counts", "n_valid",
          "prob_sum", "loss", "ws", "stream");
  int T, k, E, flags, dt;
  void *x, *mask, *ids, *w, *lse, *counts, *nv, *ps, *loss, *ws;
  long long ld;
  size_t n;
  moe_stream_t s;
  if (as_int(a[2], &T) < 0 || as_int(a[3], &k) < 0 || as_int(a[4], &E) < 0 || as_int(a[5], &flags) < 0 ||
      rows(a[0], T, E, &x, &ld) < 0 || element_type(a[0], &dt) < 0)
    return NULL;
  PyObject* mt = g_u8;
  if (a[1] != Py_None) {
    PyObject* d = dtype_of(a[1]);
    if (d == NULL) return NULL;
    if (d == g_bool) mt = g_bool; /* the same bytes */
  }
  const long long n_slots = (long long)T * k;
  if (typed(a[1], mt, T, "token_mask", &mask) < 0 || typed(a[6], g_i32, n_slots, "ids", &ids) < 0 ||
      typed(a[7], g_f32, n_slots, "weights", &w) < 0 || typed(a[8], g_f32, T, "lse", &lse) < 0 ||
      typed(a[9], g_i32, E, "counts", &counts) < 0 || typed(a[10], g_i32, 1, "n_valid", &nv) < 0 ||
      typed(a[11], g_f32, E, "prob_sum", &ps) < 0 || typed(a[12], g_f32, 2, "loss", &loss) < 0 || plain(a[13], &ws) < 0 ||
      bytes_of(a[13], &n) < 0 || as_stream(a[14], &s) < 0)
    return NULL;
  return finish("moe_gate_fwd", p_moe_gate_fwd(x, dt, ld, mask, T, k, E, flags, ids, w, lse, counts, nv, ps, loss, ws, n, s));
}

static PyObject* gate_bwd(ARGS) {
  COLLECT("moe_gate_bwd", 13, "logits", "lse", "ids", "weights", "counts", "n_valid", "d_weights", "d_loss", "T", "top_k", "E",
          "flags", "dlogits", "stream");
  int T, k, E, flags, dt;
  void *x, *o, *lse, *ids, *w, *counts, *nv, *dw, *dl;
  long long ld, ldd;
  moe_stream_t s;
  if (as_int(a[8], &T) < 0 || as_int(a[9], &k) < 0 || as_int(a[10], &E) < 0 || as_int(a[11], &flags) < 0) return NULL;
  const long long n_slots = (long long)T * k;
  if (rows(a[0], T, E, &x, &ld) < 0 || rows(a[12], T, E, &o, &ldd) < 0 ||
      same_type(a[0], a[12], "dlogits has to have the logits' type") < 0 || element_type(a[0], &dt) < 0 ||
      typed(a[1], g_f32, T, "lse", &lse) < 0 || typed(a[2], g_i32, n_slots, "ids", &ids) < 0 ||
      typed(a[3], g_f32, n_slots, "weights", &w) < 0 || typed(a[4], g_i32, E, "counts", &counts) < 0 ||
      typed(a[5], g_i32, 1, "n_valid", &nv) < 0 || typed(a[6], g_f32, n_slots, "d_weights", &dw) < 0 ||
      typed(a[7], g_f32, 2, "d_loss", &dl) < 0 || as_stream(a[13], &s) < 0)
    return NULL;
  return finish("moe_gate_bwd", p_moe_gate_bwd(x, dt, ld, lse, ids, w, counts, nv, dw, dl, T, k, E, flags, o, ldd, s));
}

static PyObject* mx4_quantize_rows(ARGS) {
  COLLECT("moe_mx4_quantize_rows", 7, "x", "offsets", "E", "cap", "K", "q", "sf", "dev_status", "stream");
  int E, cap, K;
  void *x, *off, *q, *sf, *st;
  moe_stream_t s;
  if (plain(a[0], &x) < 0 || plain(a[1], &off) < 0 || as_int(a[2], &E) < 0 || as_int(a[3], &cap) < 0 || as_int(a[4], &K) < 0 ||
      plain(a[5], &q) < 0 || plain(a[6], &sf) < 0 || plain(a[7], &st) < 0 || as_stream(a[8], &s) < 0)
    return NULL;
  return finish("moe_mx4_quantize_rows", p_moe_mx4_quantize_rows(x, off, E, cap, K, q, sf, st, s));
}

static PyObject* mx4_dequantize_rows(ARGS) {
  COLLECT("moe_mx4_dequantize_rows", 7, "q", "sf", "offsets", "E", "cap", "K", "x", "dev_status", "stream");
  int E, cap, K;
  void *x, *off, *q, *sf, *st;
  moe_stream_t s;
  if (plain(a[0], &q) < 0 || plain(a[1], &sf) < 0 || plain(a[2], &off) < 0 || as_int(a[3], &E) < 0 || as_int(a[4], &cap) < 0 ||
      as_int(a[5], &K) < 0 || plain(a[6], &x) < 0 || plain(a[7], &st) < 0 || as_stream(a[8], &s) < 0)
    return NULL;
  return finish("moe_mx4_dequantize_rows", p_moe_mx4_dequantize_rows(q, sf, off, E, cap, K, x, st, s));
}

static PyObject* permute_mxfp4(ARGS) {
  COLLECT("moe_permute_mxfp4", 9, "x", "inv_map", "offsets", "T", "top_k", "E", "d", "q", "sf", "dev_status", "stream");
  int T, k, E, d;
  void *x, *inv, *off, *q, *sf, *st;
  moe_stream_t s;
  if (plain(a[0], &x) < 0 || plain(a[1], &inv) < 0 || plain(a[2], &off) < 0 || as_int(a[3], &T) < 0 || as_int(a[4], &k) < 0 ||
      as_int(a[5], &E) < 0 || as_int(a[6], &d) < 0 || plain(a[7], &q) < 0 || plain(a[8], &sf) < 0 || plain(a[9], &st) < 0 ||
      as_stream(a[10], &s) < 0)
    return NULL;
  return finish("moe_permute_mxfp4", p_moe_permute_mxfp4(x, inv, off, T, k, E, d, q, sf, st, s));
}

static PyObject* grouped_swiglu_fwd_mxfp4(ARGS) {
  COLLECT("moe_grouped_swiglu_fwd_mxfp4", 10, "xq", "xsf", "offsets", "E", "cap", "d", "h", "mxw", "y", "ws", "dev_status",
          "stream");
  int E, cap, d, h;
  void *xq, *xsf, *off, *mxw, *y, *ws, *st;
  size_t n;
  moe_stream_t s;
  if (plain(a[0], &xq) < 0 || plain(a[1], &xsf) < 0 || plain(a[2], &off) < 0 || as_int(a[3], &E) < 0 || as_int(a[4], &cap) < 0 ||
      as_int(a[5], &d) < 0 || as_int(a[6], &h) < 0 || plain(a[7], &mxw) < 0 || plain(a[8], &y) < 0 || plain(a[9], &ws) < 0 ||
      bytes_of(a[9], &n) < 0 || plain(a[10], &st) < 0 || as_stream(a[11], &s) < 0)
    return NULL;
  return finish("moe_grouped_swiglu_fwd_mxfp4",
                p_moe_grouped_swiglu_fwd_mxfp4(xq, xsf, off, E, cap, d, h, mxw, y, ws, n, st, s));
}

static PyObject* unpermute_combine(ARGS) {
  COLLECT("moe_unpermute_combine", 7, "y", "inv_map", "weights", "T", "top_k", "d", "out", "stream");
  int T, k, d;
  void *y, *inv, *w, *out;
  moe_stream_t s;
  if (plain(a[0], &y) < 0 || plain(a[1], &inv) < 0 || plain(a[2], &w) < 0 || as_int(a[3], &T) < 0 || as_int(a[4], &k) < 0 ||
      as_int(a[5], &d) < 0 || plain(a[6], &out) < 0 || as_stream(a[7], &s) < 0)
    return NULL;
  return finish("moe_unpermute_combine", p_moe_unpermute_combine(y, inv, w, T, k, d, out, s));
}

static PyObject* route_offsets(ARGS) {
  COLLECT("moe_route_offsets", 9, "ids", "T", "top_k", "E", "counts", "offsets", "sorted_src", "inv_map", "ws", "stream");
  int T, k, E;
  void *ids, *counts, *off, *src, *inv, *ws;
  size_t n;
  moe_stream_t s;
  if (plain(a[0], &ids) < 0 || as_int(a[1], &T) < 0 || as_int(a[2], &k) < 0 || as_int(a[3], &E) < 0 || plain(a[4], &counts) < 0 ||
      plain(a[5], &off) < 0 || plain(a[6], &src) < 0 || plain(a[7], &inv) < 0 || plain(a[8], &ws) < 0 ||
      bytes_of(a[8], &n) < 0 || as_stream(a[9], &s) < 0)
    return NULL;
  return finish("moe_route_offsets", p_moe_route_offsets(ids, T, k, E, counts, off, src, inv, ws, n, s));
}

/* ------------------------------------------------------------------ module */
/* bind(addresses: dict, torch dtypes (bf16, f32, i32, u8, bool), raise_, raw_stream, get_device) */
static PyObject* bind(PyObject* self, PyObject* args) {
  (void)self;
  PyObject *table, *bf16, *f32, *i32, *u8, *b, *raise, *raw, *dev;
  if (!PyArg_ParseTuple(args, "O!OOOOOOOO", &PyDict_Type, &table, &bf16, &f32, &i32, &u8, &b, &raise, &raw, &dev)) return NULL;
#define ADDRESS(f)                                                        \
  {                                                                       \
    PyObject* o = PyDict_GetItemString(table, #f);                        \
    void* p = o ? PyLong_AsVoidPtr(o) : NULL;                             \
    if (p == NULL) {                                                      \
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_KeyError, #f);         \
      return NULL;                                                        \
    }                                                                     \
    p_##f = (__typeof__(p_##f))p;                                         \
  }
  FUNCTIONS(ADDRESS)
#define KEEP(slot, v) \
  Py_INCREF(v);       \
  Py_XSETREF(slot, v)
  KEEP(g_bf16, bf16);
  KEEP(g_f32, f32);
  KEEP(g_i32, i32);
  KEEP(g_u8, u8);
  KEEP(g_bool, b);
  KEEP(g_raise, raise);
  KEEP(g_raw_stream, raw);
  KEEP(g_get_device, dev);
  Py_RETURN_NONE;
}

#define CALL(f) {"moe_" #f, (PyCFunction)(void (*)(void))f, METH_FASTCALL | METH_KEYWORDS, NULL}
static PyMethodDef methods[] = {{"bind", bind, METH_VARARGS, NULL},
                                CALL(layer_norm_fwd),
                                CALL(layer_norm_bwd),
                                CALL(gate_fwd),
                                CALL(gate_bwd),
                                CALL(mx4_quantize_rows),
                                CALL(mx4_dequantize_rows),
                                CALL(permute_mxfp4),
                                CALL(grouped_swiglu_fwd_mxfp4),
                                CALL(unpermute_combine),
                                CALL(route_offsets),
                                {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__binding(void) {
  s_is_cuda = PyUnicode_InternFromString("is_cuda");
  s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  s_dtype = PyUnicode_InternFromString("dtype");
  s_numel = PyUnicode_InternFromString("numel");
  s_element_size = PyUnicode_InternFromString("element_size");
  s_shape = PyUnicode_InternFromString("shape");
  s_stride = PyUnicode_InternFromString("stride");
  s_cuda_stream = PyUnicode_InternFromString("cuda_stream");
  return PyModule_Create(&module);
}
