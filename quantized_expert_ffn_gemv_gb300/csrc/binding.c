/*
 * The short path of the Python binding of include/moe_model.h.
 *
 * A decode step makes a handful of these calls a layer, and a ctypes call with
 * its tensors checked in Python costs 15 to 25 us of host time, several times
 * what the small kernels take.  These functions look at the tensors through
 * the CPython API (dtype, shape, stride, device, address), call the library,
 * and return what the Python functions of the same name return.  They answer
 * None to anything but the plain case (a mismatched tensor, another current
 * device), and the Python function then goes its own way, which names what is
 * wrong; a status other than 0 comes back as an int.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

#include "moe_model.h"

typedef moe_status_t (*norm_rope_fn)(const moe_norm_rope_t*, int32_t, int32_t, int32_t, int32_t, const moe_heads_t*,
                                     const moe_heads_t*, int32_t, const moe_heads_t*, const moe_heads_t*, const int32_t*, void*);
typedef moe_status_t (*append_fn)(const moe_kv_cache_t*, const moe_kv_batch_t*, int32_t, const moe_heads_t*, const moe_heads_t*,
                                  void*);
typedef moe_status_t (*append_norm_rope_fn)(const moe_kv_cache_t*, const moe_kv_batch_t*, const moe_norm_rope_t*, int32_t, int32_t,
                                            const moe_heads_t*, const moe_heads_t*, const moe_heads_t*, const moe_heads_t*,
                                            const int32_t*, void*);
typedef moe_status_t (*workspace_fn)(const moe_kv_cache_t*, const moe_kv_batch_t*, int32_t, int32_t, size_t*);
typedef moe_status_t (*attend_fn)(const moe_kv_cache_t*, const moe_kv_batch_t*, int32_t, int32_t, const moe_heads_t*,
                                  const moe_heads_t*, float*, float, int32_t, void*, size_t, void*);
typedef moe_status_t (*sample_fn)(const void*, int32_t, int32_t, int32_t, int64_t, const float*, const float*, const int32_t*,
                                  const float*, const float*, int32_t*, float*, void*);

static struct {
  norm_rope_fn norm_rope;
  append_fn append;
  append_norm_rope_fn append_norm_rope;
  append_fn read;
  workspace_fn workspace;
  attend_fn attend;
  sample_fn sample;
  PyObject *bf16, *fp16, *fp32, *int32, *uint8;
  PyObject *current_device, *raw_stream;
  PyObject *s_dtype, *s_shape, *s_stride, *s_data_ptr, *s_get_device, *s_device;
  PyObject *empty, *kw_empty;
  int ready;
} g;

/* What is known of a tensor; all checks that fail leave an error set or return 0. */
typedef struct {
  PyObject* dtype; /* borrowed from torch: dtypes are singletons that live as long as the module */
  int ndim;
  int64_t shape[3], stride[3];
  uintptr_t at;
  long dev;
} tensor_t;

static int read_ints(PyObject* tuple, int64_t* out) {
  if (!tuple || !PyTuple_Check(tuple)) return -1;
  const Py_ssize_t n = PyTuple_GET_SIZE(tuple);
  if (n > 3) return -1;
  for (Py_ssize_t i = 0; i < n; ++i) {
    out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(tuple, i));
    if (out[i] == -1 && PyErr_Occurred()) return -1;
  }
  return (int)n;
}

static int call_long(PyObject* t, PyObject* name, int64_t* out) {
  PyObject* r = PyObject_CallMethodNoArgs(t, name);
  if (!r) return 0;
  *out = PyLong_AsLongLong(r);
  Py_DECREF(r);
  return !(*out == -1 && PyErr_Occurred());
}

static int look(PyObject* t, tensor_t* o) {
  PyObject* r = PyObject_GetAttr(t, g.s_dtype);
  if (!r) return 0;
  o->dtype = r;
  Py_DECREF(r);
  r = PyObject_GetAttr(t, g.s_shape);
  o->ndim = read_ints(r, o->shape);
  Py_XDECREF(r);
  if (o->ndim < 0) return 0;
  r = PyObject_CallMethodNoArgs(t, g.s_stride);
  const int n = read_ints(r, o->stride);
  Py_XDECREF(r);
  if (n != o->ndim) return 0;
  int64_t v;
  r = PyObject_CallMethodNoArgs(t, g.s_data_ptr);
  if (!r) return 0;
  o->at = (uintptr_t)PyLong_AsUnsignedLongLong(r);
  Py_DECREF(r);
  if (o->at == (uintptr_t)-1 && PyErr_Occurred()) return 0;
  if (!call_long(t, g.s_get_device, &v)) return 0;
  o->dev = (long)v;
  return 1;
}

static int code_of(PyObject* dtype) { return dtype == g.bf16 ? MOE_BF16 : dtype == g.fp16 ? MOE_FP16 : dtype == g.fp32 ? MOE_FP32 : -1; }

/* [n0][n1][n2] rows of heads. */
static int as_rows(const tensor_t* t, PyObject* dtype, long dev, int64_t n0, int64_t n1, int64_t n2, int out, moe_heads_t* h) {
  if (t->ndim != 3 || t->dtype != dtype || t->dev != dev || t->shape[0] != n0 || t->shape[1] != n1 || t->shape[2] != n2) return 0;
  if (t->stride[2] != 1 || ((t->stride[0] | t->stride[1]) & 7) || (t->at & 15)) return 0;
  if (out && ((n0 > 1 && t->stride[0] < n2) || (n1 > 1 && t->stride[1] < n2))) return 0;
  if (out && n0 > 1 && n1 > 1 && t->stride[0] < (n1 - 1) * t->stride[1] + n2 && t->stride[1] < (n0 - 1) * t->stride[0] + n2) return 0;
  h->data = (void*)t->at;
  h->token_stride = t->stride[0];
  h->head_stride = t->stride[1];
  return 1;
}
static int rows(PyObject* o, PyObject* dtype, long dev, int64_t n0, int64_t n1, int64_t n2, int out, moe_heads_t* h) {
  tensor_t t;
  return look(o, &t) && as_rows(&t, dtype, dev, n0, n1, n2, out, h);
}
/* A contiguous [n] vector's address; None gives NULL. */
static int vector(PyObject* o, PyObject* dtype, long dev, int64_t n, void** at) {
  *at = NULL;
  if (o == Py_None) return 1;
  tensor_t t;
  if (!look(o, &t) || t.ndim != 1 || t.dtype != dtype || t.dev != dev || t.shape[0] != n || (n > 1 && t.stride[0] != 1)) return 0;
  *at = (void*)t.at;
  return 1;
}

/* The current stream of device dev, when dev is current. */
static int stream_of(long dev, void** out) {
  PyObject* r = PyObject_CallNoArgs(g.current_device);
  if (!r) return 0;
  const long cur = PyLong_AsLong(r);
  Py_DECREF(r);
  if (cur != dev) return 0;
  PyObject* arg = PyLong_FromLong(dev);
  if (!arg) return 0;
  r = PyObject_CallOneArg(g.raw_stream, arg);
  Py_DECREF(arg);
  if (!r) return 0;
  *out = (void*)(uintptr_t)PyLong_AsUnsignedLongLong(r);
  Py_DECREF(r);
  return !PyErr_Occurred();
}

/* torch.empty(size, dtype=, device= of `like`): less than half the host time of like.new_empty(size). */
static PyObject* empty(PyObject* size, PyObject* dtype, PyObject* like) {
  if (!size) return NULL;
  PyObject* dev = PyObject_GetAttr(like, g.s_device);
  PyObject* r = NULL;
  if (dev) {
    PyObject* args[4] = {NULL, size, dtype, dev};
    r = PyObject_Vectorcall(g.empty, args + 1, 1 | PY_VECTORCALL_ARGUMENTS_OFFSET, g.kw_empty);
    Py_DECREF(dev);
  }
  Py_DECREF(size);
  return r;
}
static PyObject* new_empty3(PyObject* like, int64_t a, int64_t b, int64_t c, PyObject* dtype) {
  return empty(Py_BuildValue("(LLL)", (long long)a, (long long)b, (long long)c), dtype, like);
}
static PyObject* new_empty1(PyObject* like, int64_t n, PyObject* dtype) { return empty(PyLong_FromLongLong(n), dtype, like); }

/* Not the plain case: the Python function takes over (and raises what is to be raised). */
static PyObject* decline(void) {
  PyErr_Clear();
  Py_RETURN_NONE;
}
static PyObject* failed(moe_status_t st) { return PyLong_FromLong((long)st); }

static int norm_desc(PyObject* const* a, PyObject* dtype, long dev, int64_t dim, moe_norm_rope_t* d) {
  /* a: table, q_weight, k_weight, eps, interleaved, weight_offset */
  void *qw, *kw;
  d->table = NULL;
  d->n_positions = d->rot_dim = 0;
  if (a[0] != Py_None) {
    tensor_t t;
    if (!look(a[0], &t) || t.ndim != 3 || t.dtype != g.fp32 || t.dev != dev || t.shape[2] != 2) return 0;
    if (t.stride[2] != 1 || t.stride[1] != 2 || (t.shape[0] > 1 && t.stride[0] != 2 * t.shape[1])) return 0;
    if (t.shape[0] > INT32_MAX || t.shape[1] > INT32_MAX / 2) return 0;
    d->table = (const float*)t.at;
    d->n_positions = (int32_t)t.shape[0];
    d->rot_dim = (int32_t)(2 * t.shape[1]);
  }
  if (!vector(a[1], dtype, dev, dim, &qw) || !vector(a[2], dtype, dev, dim, &kw)) return 0;
  d->q_weight = qw;
  d->k_weight = kw;
  d->eps = (float)PyFloat_AsDouble(a[3]);
  const int inter = PyObject_IsTrue(a[4]);
  d->interleaved = inter;
  d->weight_offset = (float)PyFloat_AsDouble(a[5]);
  return inter >= 0 && !PyErr_Occurred();
}

/* qk_norm_rope(q, k, positions, table, q_weight, k_weight, eps, interleaved, weight_offset, q_out, k_out) */
static PyObject* f_qk_norm_rope(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (!g.ready || n != 11) return decline();
  tensor_t q, k;
  if (!look(a[0], &q) || !look(a[1], &k) || q.ndim != 3 || k.ndim != 3) return decline();
  const int code = code_of(q.dtype);
  if ((code != MOE_BF16 && code != MOE_FP16) || q.dev < 0 || q.shape[0] > INT32_MAX || q.shape[1] > 65536 || k.shape[1] > 65536)
    return decline();
  if (a[3] != Py_None && a[2] == Py_None) return decline();
  const int64_t T = q.shape[0], nq = q.shape[1], nk = k.shape[1], dim = q.shape[2];
  moe_heads_t qh, kh, qo, ko;
  moe_norm_rope_t d;
  void *pos, *stream;
  if (!as_rows(&q, q.dtype, q.dev, T, nq, dim, 0, &qh) || !as_rows(&k, q.dtype, q.dev, T, nk, dim, 0, &kh) ||
      !norm_desc(a + 3, q.dtype, q.dev, dim, &d) || !vector(a[2], g.int32, q.dev, T, &pos) || !stream_of(q.dev, &stream))
    return decline();
  PyObject* oq = a[9] == Py_None ? new_empty3(a[0], T, nq, dim, q.dtype) : Py_NewRef(a[9]);
  PyObject* ok = a[10] == Py_None ? new_empty3(a[1], T, nk, dim, q.dtype) : Py_NewRef(a[10]);
  PyObject* r = NULL;
  if (oq && ok && rows(oq, q.dtype, q.dev, T, nq, dim, 1, &qo) && rows(ok, q.dtype, q.dev, T, nk, dim, 1, &ko)) {
    const moe_status_t st = g.norm_rope(&d, code, (int32_t)T, (int32_t)dim, (int32_t)nq, &qh, &qo, (int32_t)nk, &kh, &ko,
                                        (const int32_t*)pos, stream);
    r = st ? failed(st) : PyTuple_Pack(2, oq, ok);
  } else {
    r = decline();
  }
  Py_XDECREF(oq);
  Py_XDECREF(ok);
  return r;
}

/* The leading arguments of the cache's functions: addresses of the descriptors and the device, which the objects hold. */
static int descs(PyObject* const* a, const moe_kv_cache_t** c, const moe_kv_batch_t** b, long* dev) {
  *c = (const moe_kv_cache_t*)(uintptr_t)PyLong_AsUnsignedLongLong(a[0]);
  *b = (const moe_kv_batch_t*)(uintptr_t)PyLong_AsUnsignedLongLong(a[1]);
  *dev = PyLong_AsLong(a[2]);
  return !PyErr_Occurred() && *c && *b;
}

/* append(cache, batch, dev, k, v) -> 0 or a status */
static PyObject* f_append(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  const moe_kv_cache_t* c;
  const moe_kv_batch_t* b;
  long dev;
  tensor_t k;
  moe_heads_t kh, vh;
  void* stream;
  if (!g.ready || n != 5 || !descs(a, &c, &b, &dev) || !look(a[3], &k)) return decline();
  const int code = code_of(k.dtype);
  if ((code != MOE_BF16 && code != MOE_FP16) || !as_rows(&k, k.dtype, dev, b->n_tokens, c->n_kv_heads, c->head_dim, 0, &kh) ||
      !rows(a[4], k.dtype, dev, b->n_tokens, c->n_kv_heads, c->head_dim, 0, &vh) || !stream_of(dev, &stream))
    return decline();
  return failed(g.append(c, b, code, &kh, &vh, stream));
}

/* append_norm_rope(cache, batch, dev, q, k, v, table, q_weight, k_weight, eps, interleaved, weight_offset, positions, q_out) */
static PyObject* f_append_norm_rope(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  const moe_kv_cache_t* c;
  const moe_kv_batch_t* b;
  long dev;
  tensor_t q;
  moe_heads_t qh, kh, vh, qo;
  moe_norm_rope_t d;
  void *pos, *stream;
  if (!g.ready || n != 14 || !descs(a, &c, &b, &dev) || !look(a[3], &q) || q.ndim != 3 || q.shape[1] > 65536) return decline();
  const int code = code_of(q.dtype);
  const int64_t T = b->n_tokens, nq = q.shape[1], dim = c->head_dim;
  if ((code != MOE_BF16 && code != MOE_FP16) || !as_rows(&q, q.dtype, dev, T, nq, dim, 0, &qh) ||
      !rows(a[4], q.dtype, dev, T, c->n_kv_heads, dim, 0, &kh) || !rows(a[5], q.dtype, dev, T, c->n_kv_heads, dim, 0, &vh) ||
      !norm_desc(a + 6, q.dtype, dev, dim, &d) || !vector(a[12], g.int32, dev, T, &pos) || !stream_of(dev, &stream))
    return decline();
  PyObject* oq = a[13] == Py_None ? new_empty3(a[3], T, nq, dim, q.dtype) : Py_NewRef(a[13]);
  if (!oq) return decline();
  if (!rows(oq, q.dtype, dev, T, nq, dim, 1, &qo)) {
    Py_DECREF(oq);
    return decline();
  }
  const moe_status_t st = g.append_norm_rope(c, b, &d, code, (int32_t)nq, &qh, &qo, &kh, &vh, (const int32_t*)pos, stream);
  if (st) {
    Py_DECREF(oq);
    return failed(st);
  }
  return oq;
}

/* read(cache, batch, dev, data, dtype, k_out, v_out) */
static PyObject* f_read(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  const moe_kv_cache_t* c;
  const moe_kv_batch_t* b;
  long dev;
  moe_heads_t kh, vh;
  void* stream;
  if (!g.ready || n != 7 || !descs(a, &c, &b, &dev)) return decline();
  const int code = code_of(a[4]);
  if ((code != MOE_BF16 && code != MOE_FP16) || !stream_of(dev, &stream)) return decline();
  const int64_t T = b->n_tokens, heads = c->n_kv_heads, dim = c->head_dim;
  PyObject* k = a[5] == Py_None ? new_empty3(a[3], T, heads, dim, a[4]) : Py_NewRef(a[5]);
  PyObject* v = a[6] == Py_None ? new_empty3(a[3], T, heads, dim, a[4]) : Py_NewRef(a[6]);
  PyObject* r = NULL;
  if (k && v && rows(k, a[4], dev, T, heads, dim, 1, &kh) && rows(v, a[4], dev, T, heads, dim, 1, &vh)) {
    const moe_status_t st = g.read(c, b, code, &kh, &vh, stream);
    r = st ? failed(st) : PyTuple_Pack(2, k, v);
  } else {
    r = decline();
  }
  Py_XDECREF(k);
  Py_XDECREF(v);
  return r;
}

/* attend(cache, batch, dev, data, q, scale, out, lse, shared_tokens); scale None: D ** -0.5 */
static PyObject* f_attend(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  const moe_kv_cache_t* c;
  const moe_kv_batch_t* b;
  long dev;
  tensor_t q, l;
  moe_heads_t qh, oh;
  void *stream, *lse = NULL;
  if (!g.ready || n != 9 || !descs(a, &c, &b, &dev) || !look(a[4], &q) || q.ndim != 3 || q.shape[1] > 65536) return decline();
  const int code = code_of(q.dtype);
  const int64_t T = b->n_tokens, nq = q.shape[1], dim = c->head_dim;
  if ((code != MOE_BF16 && code != MOE_FP16) || !as_rows(&q, q.dtype, dev, T, nq, dim, 0, &qh)) return decline();
  if (a[7] != Py_None) {
    if (!look(a[7], &l) || l.ndim != 2 || l.dtype != g.fp32 || l.dev != dev || l.shape[0] != T || l.shape[1] != nq ||
        (nq > 1 && l.stride[1] != 1) || (T > 1 && l.stride[0] != nq))
      return decline();
    lse = (void*)l.at;
  }
  const double scale = a[5] == Py_None ? (dim == 64 ? 0.125 : dim == 256 ? 0.0625 : 0.08838834764831845) : PyFloat_AsDouble(a[5]);
  const long shared = PyLong_AsLong(a[8]);
  if (PyErr_Occurred() || shared < 0 || shared > INT32_MAX || !stream_of(dev, &stream)) return decline();
  size_t bytes = 0;
  moe_status_t st = g.workspace(c, b, (int32_t)nq, (int32_t)shared, &bytes);
  if (st) return failed(st);
  PyObject* out = a[6] == Py_None ? new_empty3(a[4], T, nq, dim, q.dtype) : Py_NewRef(a[6]);
  PyObject* work = new_empty1(a[3], (int64_t)bytes, g.uint8);
  PyObject* r = NULL;
  tensor_t w;
  if (out && work && rows(out, q.dtype, dev, T, nq, dim, 1, &oh) && look(work, &w)) {
    st = g.attend(c, b, code, (int32_t)nq, &qh, &oh, (float*)lse, (float)scale, (int32_t)shared, (void*)w.at, bytes, stream);
    r = st ? failed(st) : Py_NewRef(out);
  } else {
    r = decline();
  }
  Py_XDECREF(out);
  Py_XDECREF(work);
  return r;
}

/* sample(logits, u, temperature, top_k, top_p, min_p, tokens, probs) */
static PyObject* f_sample(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  tensor_t z;
  if (!g.ready || n != 8 || !look(a[0], &z) || z.ndim != 2 || a[1] == Py_None) return decline();
  const int code = code_of(z.dtype);
  const int64_t R = z.shape[0], V = z.shape[1], stride = R > 1 ? z.stride[0] : V;
  if (code < 0 || z.dev < 0 || V < 1 || (V > 1 && z.stride[1] != 1) || stride < V || R > INT32_MAX || V > INT32_MAX) return decline();
  void *u, *t, *k, *p, *m, *tok, *pr, *stream;
  if (!vector(a[1], g.fp32, z.dev, R, &u) || !vector(a[2], g.fp32, z.dev, R, &t) || !vector(a[3], g.int32, z.dev, R, &k) ||
      !vector(a[4], g.fp32, z.dev, R, &p) || !vector(a[5], g.fp32, z.dev, R, &m) || !stream_of(z.dev, &stream))
    return decline();
  PyObject* tokens = a[6] == Py_None ? new_empty1(a[1], R, g.int32) : Py_NewRef(a[6]);
  PyObject* probs = a[7] == Py_None ? new_empty1(a[1], R, g.fp32) : Py_NewRef(a[7]);
  PyObject* r = NULL;
  if (tokens && probs && vector(tokens, g.int32, z.dev, R, &tok) && vector(probs, g.fp32, z.dev, R, &pr)) {
    const moe_status_t st = g.sample((const void*)z.at, code, (int32_t)R, (int32_t)V, stride, u, t, k, p, m, tok, pr, stream);
    r = st ? failed(st) : PyTuple_Pack(2, tokens, probs);
  } else {
    r = decline();
  }
  Py_XDECREF(tokens);
  Py_XDECREF(probs);
  return r;
}

/* setup(addresses of the 7 library functions, (bf16, fp16, fp32, int32, uint8), current_device, raw_stream, torch.empty) */
static PyObject* f_setup(PyObject* self, PyObject* args) {
  (void)self;
  PyObject *fns, *types, *cur, *raw, *empty_fn;
  if (!PyArg_ParseTuple(args, "O!O!OOO", &PyTuple_Type, &fns, &PyTuple_Type, &types, &cur, &raw, &empty_fn)) return NULL;
  if (PyTuple_GET_SIZE(fns) != 7 || PyTuple_GET_SIZE(types) != 5) {
    PyErr_SetString(PyExc_ValueError, "7 functions and 5 types");
    return NULL;
  }
  uintptr_t at[7];
  for (int i = 0; i < 7; ++i) {
    at[i] = (uintptr_t)PyLong_AsUnsignedLongLong(PyTuple_GET_ITEM(fns, i));
    if (PyErr_Occurred()) return NULL;
  }
  g.norm_rope = (norm_rope_fn)at[0];
  g.append = (append_fn)at[1];
  g.append_norm_rope = (append_norm_rope_fn)at[2];
  g.read = (append_fn)at[3];
  g.workspace = (workspace_fn)at[4];
  g.attend = (attend_fn)at[5];
  g.sample = (sample_fn)at[6];
  g.bf16 = Py_NewRef(PyTuple_GET_ITEM(types, 0));
  g.fp16 = Py_NewRef(PyTuple_GET_ITEM(types, 1));
  g.fp32 = Py_NewRef(PyTuple_GET_ITEM(types, 2));
  g.int32 = Py_NewRef(PyTuple_GET_ITEM(types, 3));
  g.uint8 = Py_NewRef(PyTuple_GET_ITEM(types, 4));
  g.empty = Py_NewRef(empty_fn);
  g.current_device = Py_NewRef(cur);
  g.raw_stream = Py_NewRef(raw);
  g.ready = 1;
  Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"setup", f_setup, METH_VARARGS, NULL},
    {"qk_norm_rope", (PyCFunction)(void (*)(void))f_qk_norm_rope, METH_FASTCALL, NULL},
    {"append", (PyCFunction)(void (*)(void))f_append, METH_FASTCALL, NULL},
    {"append_norm_rope", (PyCFunction)(void (*)(void))f_append_norm_rope, METH_FASTCALL, NULL},
    {"read", (PyCFunction)(void (*)(void))f_read, METH_FASTCALL, NULL},
    {"attend", (PyCFunction)(void (*)(void))f_attend, METH_FASTCALL, NULL},
    {"sample", (PyCFunction)(void (*)(void))f_sample, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "moe_binding", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit_moe_binding(void) {
  g.s_dtype = PyUnicode_InternFromString("dtype");
  g.s_shape = PyUnicode_InternFromString("shape");
  g.s_stride = PyUnicode_InternFromString("stride");
  g.s_data_ptr = PyUnicode_InternFromString("data_ptr");
  g.s_get_device = PyUnicode_InternFromString("get_device");
  g.s_device = PyUnicode_InternFromString("device");
  g.kw_empty = Py_BuildValue("(ss)", "dtype", "device");
  if (!g.s_dtype || !g.s_shape || !g.s_stride || !g.s_data_ptr || !g.s_get_device || !g.s_device || !g.kw_empty)
    return NULL;
  return PyModule_Create(&module);
}
