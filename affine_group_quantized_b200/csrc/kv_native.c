/*
 * kv_native.c -- the kv_* calls of the Python binding, as a CPython module.
 *
 * A decode step makes several of these calls, of a few microseconds of GPU work
 * each: looking at some eight tensors per call (size, contiguity, type, device,
 * address) and converting seventeen arguments took the interpreter and ctypes
 * longer than the kernels.  Each function here takes what its Python wrapper was
 * given, checks it, and calls the C entry point of include/qmv.h; it returns that
 * call's status, or raises ValueError for an argument that it refuses itself.
 * Arguments are tensors, plain integer addresses or None.  Other Python threads run
 * during the call, as with ctypes: a launch waits where its stream's queue is full.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "qmv.h"

static PyObject *s_nbytes, *s_is_contiguous, *s_dtype, *s_get_device, *s_data_ptr, *s_dim,
    *s_shape, *s_stride, *s_cuda_stream;

/* torch's current-device and current-stream functions, handed over by setup() */
static PyObject *f_current_device, *f_current_stream;

/* What an argument holds, and the torch types that do (tuples, by setup()). */
enum { ANY, BF16, INT, FLOAT, KINDS };
static PyObject *types_of[KINDS];
static const char *const holds[KINDS] = {"", "bf16 values", "4-byte integers", "4-byte floats"};

static int as_ll(PyObject *o, long long *out) { /* steals o */
  if (!o) return -1;
  *out = PyLong_AsLongLong(o);
  Py_DECREF(o);
  return *out == -1 && PyErr_Occurred() ? -1 : 0;
}
static int call_ll(PyObject *t, PyObject *method, long long *out) {
  return as_ll(PyObject_CallMethodNoArgs(t, method), out);
}

/* A tensor lies on the cache's device, which is the current one, or beside a cache
 * of plain addresses (device -1) on the current one, where the launch goes. */
static int on_device(PyObject *t, const char *name, long long device) {
  long long d;
  if (call_ll(t, s_get_device, &d)) return -1;
  if (d < 0) {
    PyErr_Format(PyExc_ValueError, "%s: not on a CUDA device", name);
    return -1;
  }
  if (device < 0 && as_ll(PyObject_CallNoArgs(f_current_device), &device)) return -1;
  if (d != device) {
    PyErr_Format(PyExc_ValueError, "%s: on device %lld, the call's device is %lld", name, d, device);
    return -1;
  }
  return 0;
}

static int of_type(PyObject *t, const char *name, int kind) {
  Py_ssize_t i, n;
  PyObject *types = types_of[kind], *o;
  if (!types) return 0;
  if (!(o = PyObject_GetAttr(t, s_dtype))) return -1;
  Py_DECREF(o); /* (torch keeps its types) */
  n = PyTuple_GET_SIZE(types);
  for (i = 0; i < n; ++i)
    if (PyTuple_GET_ITEM(types, i) == o) return 0;
  PyErr_Format(PyExc_ValueError, "%s: must hold %s", name, holds[kind]);
  return -1;
}

static int plain(PyObject *t, void **out, int *done) {
  *done = 1;
  if (t == Py_None) {
    *out = NULL;
    return 0;
  }
  if (PyLong_Check(t)) {
    *out = PyLong_AsVoidPtr(t);
    return PyErr_Occurred() ? -1 : 0;
  }
  *done = 0;
  return 0;
}

static int address(PyObject *t, void **out) {
  PyObject *o = PyObject_CallMethodNoArgs(t, s_data_ptr);
  if (!o) return -1;
  *out = PyLong_AsVoidPtr(o);
  Py_DECREF(o);
  return PyErr_Occurred() ? -1 : 0;
}

/* An argument of at least `need` bytes, contiguous, of the kind's types, on the
 * cache's device. */
static int arg(PyObject *t, const char *name, long long need, int kind, long long device, void **out) {
  int done, yes;
  long long n;
  PyObject *o;
  if (plain(t, out, &done) || done) return PyErr_Occurred() ? -1 : 0;
  if (as_ll(PyObject_GetAttr(t, s_nbytes), &n)) return -1;
  if (n < need) {
    PyErr_Format(PyExc_ValueError, "%s: %lld bytes, the call needs %lld", name, n, need);
    return -1;
  }
  if (!(o = PyObject_CallMethodNoArgs(t, s_is_contiguous))) return -1;
  yes = o == Py_True;
  Py_DECREF(o);
  if (!yes) {
    PyErr_Format(PyExc_ValueError, "%s: must be contiguous", name);
    return -1;
  }
  if (of_type(t, name, kind) || on_device(t, name, device)) return -1;
  return address(t, out);
}

/* Three integers of a tuple-like attribute or call result (stolen). */
static int three(PyObject *o, long long v[3]) {
  int i;
  if (!o) return -1;
  if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 3) {
    Py_DECREF(o);
    PyErr_SetString(PyExc_ValueError, "three dimensions are wanted");
    return -1;
  }
  for (i = 0; i < 3; ++i) {
    v[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(o, i));
    if (v[i] == -1 && PyErr_Occurred()) {
      Py_DECREF(o);
      return -1;
    }
  }
  Py_DECREF(o);
  return 0;
}

/* Address and stride (elements) between the rows of a bf16 [rows, heads, dim]
 * argument whose heads lie behind one another: a tensor's own stride, or the one
 * given (heads * dim when none is). */
static int arg_rows(PyObject *t, const char *name, PyObject *given, long long rows, long long heads,
                    long long dim, long long device, void **out, long long *stride) {
  const long long packed = heads * dim;
  long long n, shape[3], st[3];
  int done;
  *stride = packed;
  if (given != Py_None) {
    *stride = PyLong_AsLongLong(given);
    if (*stride == -1 && PyErr_Occurred()) return -1;
  }
  if (plain(t, out, &done) || done) return PyErr_Occurred() ? -1 : 0;
  if (given == Py_None) {
    if (call_ll(t, s_dim, &n)) return -1;
    if (n == 3) {
      if (three(PyObject_GetAttr(t, s_shape), shape)) return -1;
      if (shape[0] == rows && shape[1] == heads && shape[2] == dim) {
        if (of_type(t, name, BF16) || three(PyObject_CallMethodNoArgs(t, s_stride), st)) return -1;
        if ((dim > 1 && st[2] != 1) || (heads > 1 && st[1] != dim)) {
          PyErr_Format(PyExc_ValueError, "%s: a row's heads must be contiguous", name);
          return -1;
        }
        if (rows > 1) *stride = st[0];
        if (on_device(t, name, device)) return -1;
        return address(t, out);
      }
    }
  }
  if (rows <= 0) return arg(t, name, 0, BF16, device, out);
  if (__builtin_mul_overflow(rows - 1, *stride, &n) || __builtin_add_overflow(n, packed, &n) ||
      __builtin_mul_overflow(n, 2, &n)) {
    PyErr_Format(PyExc_ValueError, "%s: %lld rows %lld elements apart pass 64 bits", name, rows, *stride);
    return -1;
  }
  return arg(t, name, n, BF16, device, out);
}

/* What every call begins with: the cache's struct, device and shape. */
typedef struct {
  const qmv_kv_cache *cache;
  long long device; /* -1: plain addresses */
} Cache;

static int cache_of(PyObject *address_, PyObject *device, Cache *c) {
  long long here;
  c->cache = PyLong_AsVoidPtr(address_);
  if (!c->cache) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "no cache");
    return -1;
  }
  c->device = -1;
  if (device == Py_None) return 0;
  c->device = PyLong_AsLongLong(device);
  if (c->device == -1 && PyErr_Occurred()) return -1;
  /* a launch goes to the current device */
  if (as_ll(PyObject_CallNoArgs(f_current_device), &here)) return -1;
  if (here != c->device) {
    PyErr_Format(PyExc_ValueError, "the cache is on device %lld, the current device is %lld", c->device,
                 here);
    return -1;
  }
  return 0;
}

static int stream_of(PyObject *s, const Cache *c, void **out) {
  PyObject *o = NULL;
  int rc = 0;
  if (s == Py_None) { /* the current one, of the cache's or else the current device */
    PyObject *d = c->device < 0 ? PyObject_CallNoArgs(f_current_device) : PyLong_FromLongLong(c->device);
    if (!d) return -1;
    o = PyObject_CallOneArg(f_current_stream, d);
    Py_DECREF(d);
  } else if (PyLong_Check(s)) {
    o = Py_NewRef(s);
  } else {
    o = PyObject_GetAttr(s, s_cuda_stream);
  }
  if (!o) return -1;
  *out = PyLong_AsVoidPtr(o);
  if (PyErr_Occurred()) rc = -1;
  Py_DECREF(o);
  return rc;
}

static int as_int(PyObject *o, const char *name, int *out) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) return -1;
  *out = (int)v;
  if (*out != v) {
    PyErr_Format(PyExc_ValueError, "%s: %lld is too large", name, v);
    return -1;
  }
  return 0;
}

static int count_is(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return 0;
  PyErr_Format(PyExc_TypeError, "%zd arguments, %zd are wanted", n, want);
  return -1;
}

/* append(cache, device, k, v, block_table, lens, token_starts, batch,
 *        num_tokens, table_width, seen, positions, weights, state_width,
 *        k_stride, v_stride, d_status, stream) */
static PyObject *append(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  Cache c;
  int batch, tokens, width, state, rc;
  void *k, *v, *table, *lens, *starts, *seen, *positions, *weights, *status, *stream;
  long long ks, vs, H, D, slots;
  (void)self;
  if (count_is(n, 18) || cache_of(a[0], a[1], &c) || as_int(a[7], "batch", &batch) ||
      as_int(a[8], "num_tokens", &tokens) || as_int(a[9], "table_width", &width) ||
      as_int(a[13], "state_width", &state))
    return NULL;
  H = c.cache->num_kv_heads;
  D = c.cache->head_dim;
  slots = 4LL * batch * H * state;
  if (arg_rows(a[2], "k", a[14], tokens, H, D, c.device, &k, &ks) ||
      arg_rows(a[3], "v", a[15], tokens, H, D, c.device, &v, &vs) ||
      arg(a[4], "block_table", 4LL * batch * width, INT, c.device, &table) ||
      arg(a[5], "lens", 4LL * batch, INT, c.device, &lens) ||
      arg(a[6], "token_starts", 4LL * batch + 4, INT, c.device, &starts) ||
      arg(a[10], "seen", 4LL * batch, INT, c.device, &seen) ||
      arg(a[11], "positions", slots, INT, c.device, &positions) ||
      arg(a[12], "weights", slots, FLOAT, c.device, &weights) ||
      arg(a[16], "d_status", 4, INT, c.device, &status) || stream_of(a[17], &c, &stream))
    return NULL;
  Py_BEGIN_ALLOW_THREADS
  rc = kv_append(c.cache, k, v, ks, vs, table, lens, starts, batch, tokens, width, seen, positions,
                 weights, state, status, stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(rc);
}

/* read(cache, device, k, v, block_table, lens, token_starts, batch, num_tokens,
 *      table_width, k_stride, v_stride, d_status, stream) */
static PyObject *read_(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  Cache c;
  int batch, tokens, width, rc;
  void *k, *v, *table, *lens, *starts, *status, *stream;
  long long ks, vs, H, D;
  (void)self;
  if (count_is(n, 14) || cache_of(a[0], a[1], &c) || as_int(a[7], "batch", &batch) ||
      as_int(a[8], "num_tokens", &tokens) || as_int(a[9], "table_width", &width))
    return NULL;
  H = c.cache->num_kv_heads;
  D = c.cache->head_dim;
  if (arg_rows(a[2], "k", a[10], tokens, H, D, c.device, &k, &ks) ||
      arg_rows(a[3], "v", a[11], tokens, H, D, c.device, &v, &vs) ||
      arg(a[4], "block_table", 4LL * batch * width, INT, c.device, &table) ||
      arg(a[5], "lens", 4LL * batch, INT, c.device, &lens) ||
      arg(a[6], "token_starts", 4LL * batch + 4, INT, c.device, &starts) ||
      arg(a[12], "d_status", 4, INT, c.device, &status) || stream_of(a[13], &c, &stream))
    return NULL;
  Py_BEGIN_ALLOW_THREADS
  rc = kv_read(c.cache, k, v, ks, vs, table, lens, starts, batch, tokens, width, status, stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(rc);
}

/* attention(cache, device, q, block_table, lens, out, batch, num_q_heads,
 *           table_width, scale, workspace, weights, state_width, q_stride,
 *           d_status, stream) */
static PyObject *attention(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  Cache c;
  int batch, heads, width, state, rc;
  void *q, *table, *lens, *out, *workspace, *weights, *status, *stream;
  long long qs, H, D, bytes;
  double scale;
  (void)self;
  if (count_is(n, 16) || cache_of(a[0], a[1], &c) || as_int(a[6], "batch", &batch) ||
      as_int(a[7], "num_q_heads", &heads) || as_int(a[8], "table_width", &width) ||
      as_int(a[12], "state_width", &state))
    return NULL;
  scale = PyFloat_AsDouble(a[9]);
  if (scale == -1.0 && PyErr_Occurred()) return NULL;
  if (a[10] == Py_None || PyLong_Check(a[10])) {
    PyErr_SetString(PyExc_ValueError, "workspace: must be a tensor");
    return NULL;
  }
  H = c.cache->num_kv_heads;
  D = c.cache->head_dim;
  if (arg_rows(a[2], "q", a[13], batch, heads, D, c.device, &q, &qs) ||
      arg(a[3], "block_table", 4LL * batch * width, INT, c.device, &table) ||
      arg(a[4], "lens", 4LL * batch, INT, c.device, &lens) ||
      arg(a[5], "out", 2LL * batch * heads * D, BF16, c.device, &out) ||
      arg(a[11], "weights", 4LL * batch * H * state, FLOAT, c.device, &weights) ||
      arg(a[14], "d_status", 4, INT, c.device, &status) ||
      arg(a[10], "workspace", 0, ANY, c.device, &workspace) ||
      as_ll(PyObject_GetAttr(a[10], s_nbytes), &bytes) || stream_of(a[15], &c, &stream))
    return NULL;
  Py_BEGIN_ALLOW_THREADS
  rc = kv_attention(c.cache, q, qs, table, lens, out, batch, heads, width, (float)scale, weights, state,
                    workspace, (size_t)bytes, status, stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(rc);
}

/* evict(cache, device, block_table, lens, seen, weights, positions, new_lens,
 *       new_weights, new_positions, batch, table_width, state_width, budget,
 *       recent, sinks, d_status, stream) */
static PyObject *evict(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  Cache c;
  int batch, width, state, budget, recent, sinks, rc;
  void *table, *lens, *seen, *weights, *positions, *new_lens, *new_weights, *new_positions, *status,
      *stream;
  long long slots;
  (void)self;
  if (count_is(n, 18) || cache_of(a[0], a[1], &c) || as_int(a[10], "batch", &batch) ||
      as_int(a[11], "table_width", &width) || as_int(a[12], "state_width", &state) ||
      as_int(a[13], "budget", &budget) || as_int(a[14], "recent", &recent) ||
      as_int(a[15], "sinks", &sinks))
    return NULL;
  slots = 4LL * batch * c.cache->num_kv_heads * state;
  if (arg(a[2], "block_table", 4LL * batch * width, INT, c.device, &table) ||
      arg(a[3], "lens", 4LL * batch, INT, c.device, &lens) ||
      arg(a[4], "seen", 4LL * batch, INT, c.device, &seen) ||
      arg(a[5], "weights", slots, FLOAT, c.device, &weights) ||
      arg(a[6], "positions", slots, INT, c.device, &positions) ||
      arg(a[7], "new_lens", 4LL * batch, INT, c.device, &new_lens) ||
      arg(a[8], "new_weights", slots, FLOAT, c.device, &new_weights) ||
      arg(a[9], "new_positions", slots, INT, c.device, &new_positions) ||
      arg(a[16], "d_status", 4, INT, c.device, &status) || stream_of(a[17], &c, &stream))
    return NULL;
  Py_BEGIN_ALLOW_THREADS
  rc = kv_evict(c.cache, table, lens, seen, weights, positions, new_lens, new_weights, new_positions,
                batch, width, state, budget, recent, sinks, status, stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(rc);
}

/* last_error(): the message of the last non-OK status on this thread, from the
 * library that this module calls */
static PyObject *last_error(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  (void)a;
  if (count_is(n, 0)) return NULL;
  return PyUnicode_FromString(qmv_kv_last_error());
}

/* setup(current_device, current_stream, bf16 types, int types, float types) */
static PyObject *setup(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  int k;
  (void)self;
  if (count_is(n, 5)) return NULL;
  for (k = BF16; k < KINDS; ++k)
    if (!PyTuple_Check(a[1 + k])) {
      PyErr_SetString(PyExc_TypeError, "tuples of types are wanted");
      return NULL;
    }
  Py_XSETREF(f_current_device, Py_NewRef(a[0]));
  Py_XSETREF(f_current_stream, Py_NewRef(a[1]));
  for (k = BF16; k < KINDS; ++k) Py_XSETREF(types_of[k], Py_NewRef(a[1 + k]));
  Py_RETURN_NONE;
}

#define FAST(name, f) {name, (PyCFunction)(void (*)(void))f, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {FAST("append", append), FAST("read", read_),
                                FAST("attention", attention), FAST("evict", evict),
                                FAST("last_error", last_error), FAST("setup", setup), {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kv_native", NULL, -1, methods, NULL, NULL,
                                    NULL, NULL};

PyMODINIT_FUNC PyInit__kv_native(void) {
  struct {
    PyObject **to;
    const char *name;
  } names[] = {{&s_nbytes, "nbytes"},         {&s_is_contiguous, "is_contiguous"},
               {&s_dtype, "dtype"},           {&s_get_device, "get_device"},
               {&s_data_ptr, "data_ptr"},     {&s_dim, "dim"},
               {&s_shape, "shape"},           {&s_stride, "stride"},
               {&s_cuda_stream, "cuda_stream"}};
  size_t i;
  for (i = 0; i < sizeof names / sizeof *names; ++i)
    if (!(*names[i].to = PyUnicode_InternFromString(names[i].name))) return NULL;
  return PyModule_Create(&module);
}
