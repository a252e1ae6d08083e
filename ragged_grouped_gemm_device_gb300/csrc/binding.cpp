// The binding's calls that a decode step makes, as a CPython extension: the same checks and
// arguments as the Python functions of the same names in _lib.py, which stay the reference and are
// used where this extension has not been built. Marshalling a call in Python takes 3 to 8 us, more
// than most of these calls' kernels run for few tokens. Here it takes 0.2 to 0.3 us, a tenth of a
// launch: tensors are read through torch's C++ interface (by their Python attributes 0.8 to 1.7).
//
// bind() receives the addresses of the C entry points of the loaded library, so that the release and
// the debug build both work.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <exception>

#include "../../include/moe_gg.h"

#define FUNCTIONS(X)                                                                                         \
  X(moe_layer_norm_fwd) X(moe_layer_norm_bwd) X(moe_gate_fwd) X(moe_gate_bwd) X(moe_mx4_quantize_rows)        \
  X(moe_mx4_dequantize_rows) X(moe_permute_mxfp4) X(moe_grouped_swiglu_fwd_mxfp4) X(moe_unpermute_combine)    \
  X(moe_route_offsets) X(moe_workspace_bytes)
#define DECLARE(f) static __typeof__(&f) p_##f;
FUNCTIONS(DECLARE)

PyObject* g_raise;

namespace {

// an address for any of the entry points' pointer types
struct Any {
  void* p = nullptr;
  template <typename T>
  operator T*() const { return static_cast<T*>(p); }
};

// ------------------------------------------------------------------ arguments
// Positional and keyword arguments in the order of `names`; nullptr entries of optional ones become None.
int collect(const char* fn, const char* const* names, int n, int required, PyObject* const* args,
                   Py_ssize_t nargs, PyObject* kwnames, PyObject** out) {
  if (nargs > n) {
    PyErr_Format(PyExc_TypeError, "%s() takes at most %d arguments (%zd given)", fn, n, nargs);
    return -1;
  }
  for (int i = 0; i < n; ++i) out[i] = i < nargs ? args[i] : nullptr;
  const Py_ssize_t nk = kwnames ? PyTuple_GET_SIZE(kwnames) : 0;
  for (Py_ssize_t k = 0; k < nk; ++k) {
    PyObject* key = PyTuple_GET_ITEM(kwnames, k);
    int i = 0;
    while (i < n && PyUnicode_CompareWithASCIIString(key, names[i]) != 0) ++i;
    if (i == n || out[i] != nullptr) {
      PyErr_Format(PyExc_TypeError, "%s() got an unexpected or repeated argument '%U'", fn, key);
      return -1;
    }
    out[i] = args[nargs + k];
  }
  for (int i = 0; i < n; ++i) {
    if (out[i] != nullptr) continue;
    if (i < required) {
      PyErr_Format(PyExc_TypeError, "%s() missing argument '%s'", fn, names[i]);
      return -1;
    }
    out[i] = Py_None;
  }
  return 0;
}

int as_int(PyObject* o, int* v) {
  const long x = PyLong_AsLong(o);
  if (x == -1 && PyErr_Occurred()) return -1;
  if (x < INT_MIN || x > INT_MAX) {
    PyErr_SetString(PyExc_OverflowError, "an argument does not fit a C int");
    return -1;
  }
  *v = (int)x;
  return 0;
}

const at::Tensor* tensor(PyObject* o) {
  if (THPVariable_Check(o)) return &THPVariable_Unpack(o);
  PyErr_Format(PyExc_TypeError, "expected a tensor, not %s", Py_TYPE(o)->tp_name);
  return nullptr;
}

// None, or a contiguous CUDA tensor
int plain(PyObject* o, Any* p) {
  p->p = nullptr;
  if (o == Py_None) return 0;
  const at::Tensor* t = tensor(o);
  if (t == nullptr) return -1;
  if (!t->is_cuda() || !t->is_contiguous()) {
    PyErr_SetString(PyExc_ValueError, "tensors passed to the library must be contiguous CUDA tensors");
    return -1;
  }
  p->p = t->mutable_data_ptr();
  return 0;
}

// None, or a contiguous CUDA tensor of a type with at least `numel` elements
int typed(PyObject* o, at::ScalarType type, long long numel, const char* name, Any* p) {
  p->p = nullptr;
  if (o == Py_None) return 0;
  const at::Tensor* t = tensor(o);
  if (t == nullptr) return -1;
  if (t->scalar_type() != type || t->numel() < numel || !t->is_cuda() || !t->is_contiguous()) {
    PyErr_Format(PyExc_ValueError, "%s: expected a contiguous CUDA tensor of at least %lld elements of %s", name, numel,
                 c10::toString(type));
    return -1;
  }
  p->p = t->mutable_data_ptr();
  return 0;
}

// None, or a contiguous CUDA tensor of any type with at least `nbytes` bytes: codes, scales, prepared weights
int raw(PyObject* o, long long nbytes, const char* name, Any* p) {
  p->p = nullptr;
  if (o == Py_None) return 0;
  const at::Tensor* t = tensor(o);
  if (t == nullptr) return -1;
  if (static_cast<long long>(t->numel()) * static_cast<long long>(t->element_size()) < nbytes || !t->is_cuda() ||
      !t->is_contiguous()) {
    PyErr_Format(PyExc_ValueError, "%s: expected a contiguous CUDA tensor of at least %lld bytes", name, nbytes);
    return -1;
  }
  p->p = t->mutable_data_ptr();
  return 0;
}

// None, or a device status word
int status(PyObject* o, Any* p) { return typed(o, at::kInt, 1, "dev_status", p); }

// bytes of the scale atoms of `rows` rows of K elements (0 without rows and for sizes that the library refuses)
long long scale_bytes(long long rows, int E, int K) {
  if (rows <= 0 || rows > INT_MAX) return 0;
  return static_cast<long long>(p_moe_workspace_bytes(MOE_OP_MX4_ROW_SCALES, static_cast<int>(rows), 1, E, K, 32, 0));
}

int bytes_of(PyObject* o, size_t* b) {
  *b = 0;
  if (o == Py_None) return 0;
  const at::Tensor* t = tensor(o);
  if (t == nullptr) return -1;
  *b = static_cast<size_t>(t->numel()) * t->element_size();
  return 0;
}

// pointer and row pitch of a [>= T, width] tensor whose rows are contiguous
int rows(PyObject* o, int T, int width, Any* p, long long* ld) {
  const at::Tensor* t = tensor(o);
  if (t == nullptr) return -1;
  if (t->dim() != 2 || !t->is_cuda() || t->size(0) < T || t->size(1) != width || (width > 1 && t->stride(1) != 1)) {
    PyErr_Format(PyExc_ValueError, "expected a CUDA tensor of at least %d rows of %d contiguous elements", T, width);
    return -1;
  }
  *ld = T > 1 && !t->is_contiguous() ? t->stride(0) : width;
  p->p = t->mutable_data_ptr();
  return 0;
}

int element_type(PyObject* o, int* v) {
  const at::Tensor* t = tensor(o);
  if (t == nullptr) return -1;
  if (t->scalar_type() == at::kBFloat16) *v = MOE_DTYPE_BF16;
  else if (t->scalar_type() == at::kFloat) *v = MOE_DTYPE_F32;
  else {
    PyErr_Format(PyExc_ValueError, "expected a bfloat16 or float32 tensor, not %s", c10::toString(t->scalar_type()));
    return -1;
  }
  return 0;
}

int same_type(PyObject* a, PyObject* b, const char* what) {
  const at::Tensor *x = tensor(a), *y = x ? tensor(b) : nullptr;
  if (y == nullptr) return -1;
  if (x->scalar_type() == y->scalar_type()) return 0;
  PyErr_SetString(PyExc_ValueError, what);
  return -1;
}

int as_stream(PyObject* o, moe_stream_t* s) {
  if (o == Py_None) {
    *s = reinterpret_cast<moe_stream_t>(c10::cuda::getCurrentCUDAStream().stream());
    return 0;
  }
  PyObject* v = PyObject_GetAttrString(o, "cuda_stream");
  if (v == nullptr) return -1;
  *s = reinterpret_cast<moe_stream_t>(PyLong_AsVoidPtr(v));
  Py_DECREF(v);
  return *s == nullptr && PyErr_Occurred() ? -1 : 0;
}

// The interpreter lock given up for a scope, which an exception may leave too
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};

// Calls the library without the interpreter lock, like ctypes: a launch waits while the stream's queue is full
// (and in the debug build for the stream), and other threads have to run meanwhile.
template <typename Call>
PyObject* finish(const char* fn, Call call) {
  const moe_status_t st = [&] {
    Unlocked unlocked;
    return call();
  }();
  if (st == MOE_OK) Py_RETURN_NONE;
  PyObject* r = PyObject_CallFunction(g_raise, "si", fn, (int)st);
  Py_XDECREF(r);
  if (!PyErr_Occurred()) PyErr_Format(PyExc_RuntimeError, "%s returned %d", fn, (int)st);
  return nullptr;
}

// the weights' type: all bf16 or all fp32, [d] each; fp32 when there are none
int weight_type(PyObject* const* w, int n, int d, int* v) {
  PyObject* first = nullptr;
  *v = MOE_DTYPE_F32;
  for (int i = 0; i < n; ++i) {
    if (w[i] == Py_None) continue;
    const at::Tensor* t = tensor(w[i]);
    if (t == nullptr) return -1;
    if (t->numel() != d || (first != nullptr && t->scalar_type() != THPVariable_Unpack(first).scalar_type())) {
      PyErr_Format(PyExc_ValueError, "the weights have to be [%d] and of one type", d);
      return -1;
    }
    first = w[i];
  }
  return first == nullptr ? 0 : element_type(first, v);
}

#define ARGS PyObject *self, PyObject *const *args, Py_ssize_t nargs, PyObject *kwnames
#define COLLECT(fn, required, ...)                                                        \
  static const char* const names[] = {__VA_ARGS__};                                       \
  enum { N = sizeof(names) / sizeof(names[0]) };                                          \
  PyObject* a[N];                                                                         \
  (void)self;                                                                             \
  if (collect(fn, names, N, required, args, nargs, kwnames, a) < 0) return nullptr

// ------------------------------------------------------------------ the calls
PyObject* layer_norm_fwd(ARGS) {
  COLLECT("moe_layer_norm_fwd", 7, "x", "gamma", "beta", "T", "d", "eps", "y", "mean", "rstd", "stream");
  int T, d, dt, wt;
  Any x, y, gamma, beta, mean, rstd;
  long long ldx, ldy;
  moe_stream_t s;
  if (as_int(a[3], &T) < 0 || as_int(a[4], &d) < 0) return nullptr;
  const double eps = PyFloat_AsDouble(a[5]);
  if (eps == -1.0 && PyErr_Occurred()) return nullptr;
  if (rows(a[0], T, d, &x, &ldx) < 0 || rows(a[6], T, d, &y, &ldy) < 0 ||
      same_type(a[0], a[6], "y has to have x's type") < 0 || element_type(a[0], &dt) < 0 || plain(a[1], &gamma) < 0 ||
      plain(a[2], &beta) < 0 || weight_type(a + 1, 2, d, &wt) < 0 || typed(a[7], at::kFloat, T, "mean", &mean) < 0 ||
      typed(a[8], at::kFloat, T, "rstd", &rstd) < 0 || as_stream(a[9], &s) < 0)
    return nullptr;
  return finish("moe_layer_norm_fwd", [&] {
    return p_moe_layer_norm_fwd(x, dt, ldx, gamma, beta, wt, T, d, (float)eps, y, ldy, mean, rstd, s);
  });
}

PyObject* layer_norm_bwd(ARGS) {
  COLLECT("moe_layer_norm_bwd", 8, "dy", "x", "gamma", "mean", "rstd", "T", "d", "dx", "dgamma", "dbeta", "ws", "stream");
  int T, d, dt, wt;
  Any dy, x, dx, gamma, mean, rstd, dgamma, dbeta, ws;
  long long lddy, ldx, lddx;
  size_t n;
  moe_stream_t s;
  static const char* const types = "x, dy and dx have to have one type";
  if (as_int(a[5], &T) < 0 || as_int(a[6], &d) < 0 || rows(a[0], T, d, &dy, &lddy) < 0 || rows(a[1], T, d, &x, &ldx) < 0 ||
      rows(a[7], T, d, &dx, &lddx) < 0 || same_type(a[0], a[1], types) < 0 || same_type(a[1], a[7], types) < 0 ||
      element_type(a[1], &dt) < 0 || plain(a[2], &gamma) < 0 || weight_type(a + 2, 1, d, &wt) < 0 ||
      typed(a[3], at::kFloat, T, "mean", &mean) < 0 || typed(a[4], at::kFloat, T, "rstd", &rstd) < 0 ||
      typed(a[8], at::kFloat, d, "dgamma", &dgamma) < 0 || typed(a[9], at::kFloat, d, "dbeta", &dbeta) < 0 ||
      plain(a[10], &ws) < 0 || bytes_of(a[10], &n) < 0 || as_stream(a[11], &s) < 0)
    return nullptr;
  return finish("moe_layer_norm_bwd", [&] {
    return p_moe_layer_norm_bwd(dy, lddy, x, ldx, dt, gamma, wt, mean, rstd, T, d, dx, lddx, dgamma, dbeta, ws, n, s);
  });
}

PyObject* gate_fwd(ARGS) {
  COLLECT("moe_gate_fwd", 8, "logits", "token_mask", "T", "top_k", "E", "flags", "ids", "weights", "lse", "counts", "n_valid",
          "prob_sum", "loss", "ws", "stream");
  int T, k, E, flags, dt;
  Any x, mask, ids, w, lse, counts, nv, ps, loss, ws;
  long long ld;
  size_t n;
  moe_stream_t s;
  if (as_int(a[2], &T) < 0 || as_int(a[3], &k) < 0 || as_int(a[4], &E) < 0 || as_int(a[5], &flags) < 0 ||
      rows(a[0], T, E, &x, &ld) < 0 || element_type(a[0], &dt) < 0)
    return nullptr;
  // the same bytes
  const at::ScalarType mt = THPVariable_Check(a[1]) && THPVariable_Unpack(a[1]).scalar_type() == at::kBool ? at::kBool : at::kByte;
  const long long n_slots = (long long)T * k;
  if (typed(a[1], mt, T, "token_mask", &mask) < 0 || typed(a[6], at::kInt, n_slots, "ids", &ids) < 0 ||
      typed(a[7], at::kFloat, n_slots, "weights", &w) < 0 || typed(a[8], at::kFloat, T, "lse", &lse) < 0 ||
      typed(a[9], at::kInt, E, "counts", &counts) < 0 || typed(a[10], at::kInt, 1, "n_valid", &nv) < 0 ||
      typed(a[11], at::kFloat, E, "prob_sum", &ps) < 0 || typed(a[12], at::kFloat, 2, "loss", &loss) < 0 || plain(a[13], &ws) < 0 ||
      bytes_of(a[13], &n) < 0 || as_stream(a[14], &s) < 0)
    return nullptr;
  return finish("moe_gate_fwd", [&] {
    return p_moe_gate_fwd(x, dt, ld, mask, T, k, E, flags, ids, w, lse, counts, nv, ps, loss, ws, n, s);
  });
}

PyObject* gate_bwd(ARGS) {
  COLLECT("moe_gate_bwd", 13, "logits", "lse", "ids", "weights", "counts", "n_valid", "d_weights", "d_loss", "T", "top_k", "E",
          "flags", "dlogits", "stream");
  int T, k, E, flags, dt;
  Any x, o, lse, ids, w, counts, nv, dw, dl;
  long long ld, ldd;
  moe_stream_t s;
  if (as_int(a[8], &T) < 0 || as_int(a[9], &k) < 0 || as_int(a[10], &E) < 0 || as_int(a[11], &flags) < 0) return nullptr;
  const long long n_slots = (long long)T * k;
  if (rows(a[0], T, E, &x, &ld) < 0 || rows(a[12], T, E, &o, &ldd) < 0 ||
      same_type(a[0], a[12], "dlogits has to have the logits' type") < 0 || element_type(a[0], &dt) < 0 ||
      typed(a[1], at::kFloat, T, "lse", &lse) < 0 || typed(a[2], at::kInt, n_slots, "ids", &ids) < 0 ||
      typed(a[3], at::kFloat, n_slots, "weights", &w) < 0 || typed(a[4], at::kInt, E, "counts", &counts) < 0 ||
      typed(a[5], at::kInt, 1, "n_valid", &nv) < 0 || typed(a[6], at::kFloat, n_slots, "d_weights", &dw) < 0 ||
      typed(a[7], at::kFloat, 2, "d_loss", &dl) < 0 || as_stream(a[13], &s) < 0)
    return nullptr;
  return finish("moe_gate_bwd", [&] {
    return p_moe_gate_bwd(x, dt, ld, lse, ids, w, counts, nv, dw, dl, T, k, E, flags, o, ldd, s);
  });
}

PyObject* mx4_quantize_rows(ARGS) {
  COLLECT("moe_mx4_quantize_rows", 7, "x", "offsets", "E", "cap", "K", "q", "sf", "dev_status", "stream");
  int E, cap, K;
  Any x, off, q, sf, st;
  moe_stream_t s;
  if (as_int(a[2], &E) < 0 || as_int(a[3], &cap) < 0 || as_int(a[4], &K) < 0) return nullptr;
  const long long n = (long long)cap * K;
  if (typed(a[0], at::kBFloat16, n, "x", &x) < 0 || typed(a[1], at::kInt, E, "offsets", &off) < 0 ||
      raw(a[5], n / 2, "q", &q) < 0 || raw(a[6], scale_bytes(cap, E, K), "sf", &sf) < 0 || status(a[7], &st) < 0 ||
      as_stream(a[8], &s) < 0)
    return nullptr;
  return finish("moe_mx4_quantize_rows", [&] {
    return p_moe_mx4_quantize_rows(x, off, E, cap, K, q, sf, st, s);
  });
}

PyObject* mx4_dequantize_rows(ARGS) {
  COLLECT("moe_mx4_dequantize_rows", 7, "q", "sf", "offsets", "E", "cap", "K", "x", "dev_status", "stream");
  int E, cap, K;
  Any x, off, q, sf, st;
  moe_stream_t s;
  if (as_int(a[3], &E) < 0 || as_int(a[4], &cap) < 0 || as_int(a[5], &K) < 0) return nullptr;
  const long long n = (long long)cap * K;
  if (raw(a[0], n / 2, "q", &q) < 0 || raw(a[1], scale_bytes(cap, E, K), "sf", &sf) < 0 ||
      typed(a[2], at::kInt, E, "offsets", &off) < 0 || typed(a[6], at::kBFloat16, n, "x", &x) < 0 || status(a[7], &st) < 0 ||
      as_stream(a[8], &s) < 0)
    return nullptr;
  return finish("moe_mx4_dequantize_rows", [&] {
    return p_moe_mx4_dequantize_rows(q, sf, off, E, cap, K, x, st, s);
  });
}

PyObject* permute_mxfp4(ARGS) {
  COLLECT("moe_permute_mxfp4", 9, "x", "inv_map", "offsets", "T", "top_k", "E", "d", "q", "sf", "dev_status", "stream");
  int T, k, E, d;
  Any x, inv, off, q, sf, st;
  moe_stream_t s;
  if (as_int(a[3], &T) < 0 || as_int(a[4], &k) < 0 || as_int(a[5], &E) < 0 || as_int(a[6], &d) < 0) return nullptr;
  const long long n = (long long)T * k;
  const long long code_bytes = n > 0 && n <= INT_MAX ? n * d / 2 : 0;  // of other counts the library says what is wrong
  if (typed(a[0], at::kBFloat16, (long long)T * d, "x", &x) < 0 || typed(a[1], at::kInt, n, "inv_map", &inv) < 0 ||
      typed(a[2], at::kInt, E, "offsets", &off) < 0 || raw(a[7], code_bytes, "q", &q) < 0 ||
      raw(a[8], scale_bytes(n, E, d), "sf", &sf) < 0 || status(a[9], &st) < 0 || as_stream(a[10], &s) < 0)
    return nullptr;
  return finish("moe_permute_mxfp4", [&] {
    return p_moe_permute_mxfp4(x, inv, off, T, k, E, d, q, sf, st, s);
  });
}

PyObject* grouped_swiglu_fwd_mxfp4(ARGS) {
  COLLECT("moe_grouped_swiglu_fwd_mxfp4", 10, "xq", "xsf", "offsets", "E", "cap", "d", "h", "mxw", "y", "ws", "dev_status",
          "stream");
  int E, cap, d, h;
  Any xq, xsf, off, mxw, y, ws, st;
  size_t n;
  moe_stream_t s;
  if (as_int(a[3], &E) < 0 || as_int(a[4], &cap) < 0 || as_int(a[5], &d) < 0 || as_int(a[6], &h) < 0) return nullptr;
  const long long items = (long long)cap * d;
  if (raw(a[0], items / 2, "xq", &xq) < 0 || raw(a[1], scale_bytes(cap, E, d), "xsf", &xsf) < 0 ||
      typed(a[2], at::kInt, E, "offsets", &off) < 0 ||
      raw(a[7], static_cast<long long>(p_moe_workspace_bytes(MOE_OP_MX4_WEIGHTS, 0, 1, E, d, h, 0)), "mxw", &mxw) < 0 ||
      typed(a[8], at::kBFloat16, items, "y", &y) < 0 || plain(a[9], &ws) < 0 || bytes_of(a[9], &n) < 0 ||
      status(a[10], &st) < 0 || as_stream(a[11], &s) < 0)
    return nullptr;
  return finish("moe_grouped_swiglu_fwd_mxfp4", [&] {
    return p_moe_grouped_swiglu_fwd_mxfp4(xq, xsf, off, E, cap, d, h, mxw, y, ws, n, st, s);
  });
}

PyObject* unpermute_combine(ARGS) {
  COLLECT("moe_unpermute_combine", 7, "y", "inv_map", "weights", "T", "top_k", "d", "out", "stream");
  int T, k, d;
  Any y, inv, w, out;
  moe_stream_t s;
  if (plain(a[0], &y) < 0 || plain(a[1], &inv) < 0 || plain(a[2], &w) < 0 || as_int(a[3], &T) < 0 || as_int(a[4], &k) < 0 ||
      as_int(a[5], &d) < 0 || plain(a[6], &out) < 0 || as_stream(a[7], &s) < 0)
    return nullptr;
  return finish("moe_unpermute_combine", [&] {
    return p_moe_unpermute_combine(y, inv, w, T, k, d, out, s);
  });
}

PyObject* route_offsets(ARGS) {
  COLLECT("moe_route_offsets", 9, "ids", "T", "top_k", "E", "counts", "offsets", "sorted_src", "inv_map", "ws", "stream");
  int T, k, E;
  Any ids, counts, off, src, inv, ws;
  size_t n;
  moe_stream_t s;
  if (plain(a[0], &ids) < 0 || as_int(a[1], &T) < 0 || as_int(a[2], &k) < 0 || as_int(a[3], &E) < 0 || plain(a[4], &counts) < 0 ||
      plain(a[5], &off) < 0 || plain(a[6], &src) < 0 || plain(a[7], &inv) < 0 || plain(a[8], &ws) < 0 ||
      bytes_of(a[8], &n) < 0 || as_stream(a[9], &s) < 0)
    return nullptr;
  return finish("moe_route_offsets", [&] {
    return p_moe_route_offsets(ids, T, k, E, counts, off, src, inv, ws, n, s);
  });
}

// ------------------------------------------------------------------ module
// bind(addresses: dict, raise_)
PyObject* bind(PyObject* self, PyObject* args) {
  (void)self;
  PyObject *table, *raise;
  if (!PyArg_ParseTuple(args, "O!O", &PyDict_Type, &table, &raise)) return nullptr;
#define ADDRESS(f)                                                        \
  {                                                                       \
    PyObject* o = PyDict_GetItemString(table, #f);                        \
    void* p = o ? PyLong_AsVoidPtr(o) : nullptr;                             \
    if (p == nullptr) {                                                      \
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_KeyError, #f);         \
      return nullptr;                                                        \
    }                                                                     \
    p_##f = (__typeof__(p_##f))p;                                         \
  }
  FUNCTIONS(ADDRESS)
  Py_INCREF(raise);
  Py_XSETREF(g_raise, raise);
  Py_RETURN_NONE;
}

// no C++ exception leaves a call
template <PyObject* (*F)(ARGS)>
PyObject* guarded(ARGS) {
  try {
    return F(self, args, nargs, kwnames);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

#define CALL(f) {"moe_" #f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<f>)), METH_FASTCALL | METH_KEYWORDS, nullptr}
PyMethodDef methods[] = {{"bind", bind, METH_VARARGS, nullptr},
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
                                {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module); }
