/* The checks and the argument marshalling of kv.py's and sampling.py's calls, in C: at decode
 * sizes they cost more host time in Python than the launch itself.
 *
 * A tensor is read through its own attributes (is_cuda, dtype, shape, stride,
 * get_device, data_ptr), so nothing of torch is compiled in; the entry points
 * of libtern come as addresses (bind).  Every function returns the entry point's status;
 * what a tensor must be and is not raises ValueError, before the call. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "tern.h"

static PyObject *s_is_cuda, *s_dtype, *s_shape, *s_stride, *s_data_ptr, *s_get_device;
static PyObject *t_int32, *t_int64, *t_float32;   /* torch's types */
static PyObject* current_device;                   /* torch's, a callable; None: there is one device */

typedef tern_status (*plan_fn)(const int32_t*, const int32_t*, int64_t, int64_t, int32_t*, int64_t,
                               int64_t, const int32_t*, const int32_t*, int64_t, const int32_t*,
                               int32_t*, int64_t, int64_t*, int32_t*, int32_t*, int32_t*, int32_t*,
                               void*);
typedef tern_status (*write_fn)(const tern_kv_cache*, const void*, const void*, int64_t, int64_t,
                                int64_t, int64_t, const int64_t*, int64_t, void*);
typedef tern_status (*attn_fn)(const void*, int64_t, int64_t, const tern_kv_cache*, const int32_t*,
                               int64_t, int64_t, const int32_t*, const int32_t*, const uint64_t*,
                               int64_t, int64_t, int64_t, int64_t, int64_t, float, void*, float*,
                               void*, size_t, void*);
typedef tern_status (*commit_fn)(const tern_kv_cache*, int64_t, const int32_t*, int64_t, int64_t,
                                 const int32_t*, const int32_t*, int64_t, const int32_t*, int32_t*,
                                 int64_t, void*);
typedef tern_status (*rotate_fn)(const tern_kv_cache*, const tern_kv_cache8*, const tern_kv_rows*,
                                 void*);
typedef tern_status (*read_fn)(const tern_kv_cache8*, const int64_t*, int64_t, void*, void*, int32_t,
                               void*);
typedef tern_status (*attn8_fn)(const void*, int64_t, int64_t, int32_t, const tern_kv_cache8*,
                                const int32_t*, int64_t, int64_t, const int32_t*, const int32_t*,
                                const uint64_t*, int64_t, int64_t, int64_t, int64_t, int64_t, float,
                                void*, float*, void*, size_t, void*);
typedef tern_status (*commit8_fn)(const tern_kv_cache8*, int64_t, const int32_t*, int64_t, int64_t,
                                  const int32_t*, const int32_t*, int64_t, const int32_t*, int32_t*,
                                  int64_t, void*);
typedef tern_status (*sample_fn)(const void*, int64_t, int64_t, int64_t, int32_t, const float*,
                                 const float*, const int32_t*, const float*, const float*, int32_t*,
                                 void*);
typedef tern_status (*accept_fn)(const int32_t*, const int32_t*, const int32_t*, const int32_t*,
                                 int64_t, int64_t, int64_t, int32_t*, int32_t*, int32_t*, void*);
static plan_fn f_plan;
static write_fn f_write;
static attn_fn f_attn;
static commit_fn f_commit;
static rotate_fn f_rotate;
static read_fn f_read;
static commit8_fn f_commit8;
static attn8_fn f_attn8;
static sample_fn f_sample;
static accept_fn f_accept;

typedef struct {
  void* p;
  int64_t shape[3], stride[3];
  int ndim;
  long device;   /* -1: an argument that was not given, or there is one device */
} Tensor;

/* A dimension or stride tuple into out; its length, or -1. */
static int numbers(PyObject* tuple, int64_t* out) {
  if (tuple == NULL || !PyTuple_Check(tuple)) return -1;
  const Py_ssize_t n = PyTuple_GET_SIZE(tuple);
  if (n > 3) return 4;
  for (Py_ssize_t i = 0; i < n; ++i) {
    out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(tuple, i));
    if (out[i] == -1 && PyErr_Occurred()) return -1;
  }
  return (int)n;
}

/* Reads a CUDA tensor of the type and number of axes; 0 and an exception if
 * it is none. */
static int read_tensor(PyObject* o, PyObject* dtype, int ndim, const char* name, Tensor* t) {
  PyObject* x = PyObject_GetAttr(o, s_is_cuda);
  if (x == NULL) return 0;
  const int cuda = x == Py_True;
  Py_DECREF(x);
  x = PyObject_GetAttr(o, s_dtype);
  if (x == NULL) return 0;
  const int type = x == dtype;
  Py_DECREF(x);
  x = PyObject_GetAttr(o, s_shape);
  t->ndim = numbers(x, t->shape);
  Py_XDECREF(x);
  if (t->ndim < 0) return 0;
  if (!cuda || !type || t->ndim != ndim) {
    PyErr_Format(PyExc_ValueError, "%s: expected a %d-D CUDA tensor of %S", name, ndim, dtype);
    return 0;
  }
  x = PyObject_CallMethodNoArgs(o, s_stride);
  const int n = numbers(x, t->stride);
  Py_XDECREF(x);
  if (n < 0) return 0;
  t->device = -1;
  if (current_device != Py_None) {
    x = PyObject_CallMethodNoArgs(o, s_get_device);
    if (x == NULL) return 0;
    t->device = PyLong_AsLong(x);
    Py_DECREF(x);
    if (t->device < 0) {
      if (!PyErr_Occurred()) PyErr_Format(PyExc_ValueError, "%s: expected a device number", name);
      return 0;
    }
  }
  x = PyObject_CallMethodNoArgs(o, s_data_ptr);
  if (x == NULL) return 0;
  t->p = PyLong_AsVoidPtr(x);
  Py_DECREF(x);
  return !(t->p == NULL && PyErr_Occurred());
}

static int refuse(const char* what) {
  PyErr_SetString(PyExc_ValueError, what);
  return 0;
}

static int dense(const Tensor* t) {
  int64_t want = 1;
  for (int i = t->ndim - 1; i >= 0; --i) {
    if (t->shape[i] == 0) return 1;
    if (t->shape[i] != 1 && t->stride[i] != want) return 0;
    want *= t->shape[i];
  }
  return 1;
}

static int read_dense(PyObject* o, PyObject* dtype, int ndim, const char* name, Tensor* t) {
  if (!read_tensor(o, dtype, ndim, name, t)) return 0;
  if (!dense(t)) {
    PyErr_Format(PyExc_ValueError, "%s: expected a contiguous tensor", name);
    return 0;
  }
  return 1;
}

/* A block table of b rows; its row stride (rows may be longer than the part in use). */
static int read_table(PyObject* o, int64_t b, Tensor* t, int64_t* stride) {
  if (!read_tensor(o, t_int32, 2, "table", t)) return 0;
  const int64_t w = t->shape[1];
  if (t->shape[0] != b || (w > 1 && t->stride[1] != 1) || (b > 1 && t->stride[0] < w))
    return refuse("table: expected [requests, width] with dense rows");
  *stride = b > 1 ? t->stride[0] : (w > 1 ? w : 1);
  return 1;
}

/* [rows, heads, dim], dense along the last axis, e.g. a slice of the qkv
 * linear's output; its row and head strides (an axis of length one may have
 * any). */
static int read_heads(PyObject* o, PyObject* dtype, int64_t heads, int64_t dim, const char* name,
                      Tensor* t, int64_t* row, int64_t* head) {
  if (!read_tensor(o, dtype, 3, name, t)) return 0;
  if ((heads >= 0 && t->shape[1] != heads) || t->shape[2] != dim || t->stride[2] != 1) {
    PyErr_Format(PyExc_ValueError, "%s: expected [rows, heads, %lld], dense along the last axis",
                 name, (long long)dim);
    return 0;
  }
  *row = t->shape[0] > 1 ? t->stride[0] : t->shape[1] * dim;
  *head = t->shape[1] > 1 ? t->stride[1] : dim;
  return 1;
}

/* Returns an entry point's status as a number.  It runs without the interpreter's
 * lock: a launch waits where the stream's queue is full, e.g. behind a host
 * callback that needs the lock. */
#define RETURN_STATUS(call)          \
  do {                               \
    tern_status st_;                 \
    Py_BEGIN_ALLOW_THREADS           \
    st_ = (call);                    \
    Py_END_ALLOW_THREADS             \
    return PyLong_FromLong(st_);     \
  } while (0)

/* Whether all of them are on the current device, the one of the call's stream:
 * a pointer to another's memory could fault in a kernel. */
static int on_current_device(const Tensor* const* t, int n, long cache) {
  if (current_device == Py_None) return 1;
  PyObject* x = PyObject_CallNoArgs(current_device);
  if (x == NULL) return 0;
  const long now = PyLong_AsLong(x);
  Py_DECREF(x);
  if (now == -1 && PyErr_Occurred()) return 0;
  int ok = cache < 0 || cache == now;
  for (int i = 0; i < n; ++i) ok &= t[i]->device < 0 || t[i]->device == now;
  if (ok) return 1;
  PyErr_Format(PyExc_ValueError, "expected every tensor on the current device, cuda:%ld", now);
  return 0;
}
#define ON_CURRENT_DEVICE(cache, ...)                                  \
  on_current_device((const Tensor* const[]){__VA_ARGS__},              \
                    sizeof((const Tensor* const[]){__VA_ARGS__}) / sizeof(Tensor*), cache)

static int counted(Py_ssize_t got, Py_ssize_t want) {
  if (got == want) return 1;
  PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, got);
  return 0;
}

static int64_t integer(PyObject* o) { return PyLong_AsLongLong(o); }

/* bind(plan, write, attention, commit, int32, int64, float32, current device's callable or None) */
static PyObject* py_bind(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  if (!counted(n, 8)) return NULL;
  f_plan = (plan_fn)PyLong_AsVoidPtr(a[0]);
  f_write = (write_fn)PyLong_AsVoidPtr(a[1]);
  f_attn = (attn_fn)PyLong_AsVoidPtr(a[2]);
  f_commit = (commit_fn)PyLong_AsVoidPtr(a[3]);
  if (PyErr_Occurred()) return NULL;
  t_int32 = Py_NewRef(a[4]);
  t_int64 = Py_NewRef(a[5]);
  t_float32 = Py_NewRef(a[6]);
  current_device = Py_NewRef(a[7]);
  Py_RETURN_NONE;
}

/* plan(ctx_len, new_len, table, free_pages, free_head or None, page_size, capacity,
 *      row_start, slots, positions, request, info, held or None, held_out or None, stream) */
static PyObject* py_plan(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  Tensor ctx, new_len, table, free_pages, head, start, slots, pos, req, info, held, held_out;
  int64_t stride;
  if (!counted(n, 15) || !read_dense(a[0], t_int32, 1, "ctx_len", &ctx) ||
      !read_dense(a[1], t_int32, 1, "new_len", &new_len) ||
      !read_table(a[2], ctx.shape[0], &table, &stride) ||
      !read_dense(a[3], t_int32, 1, "free_pages", &free_pages) ||
      !read_dense(a[7], t_int32, 1, "row_start", &start) ||
      !read_dense(a[8], t_int64, 1, "slots", &slots) ||
      !read_dense(a[9], t_int32, 1, "positions", &pos) ||
      !read_dense(a[10], t_int32, 1, "request", &req) ||
      !read_dense(a[11], t_int32, 1, "info", &info))
    return NULL;
  const int64_t b = ctx.shape[0], page = integer(a[5]), capacity = integer(a[6]);
  head.p = NULL;
  head.device = -1;
  if (a[4] != Py_None) {
    if (!read_dense(a[4], t_int32, 1, "free_head", &head)) return NULL;
    if (head.shape[0] != 1) return refuse("free_head: expected one number"), NULL;
  }
  held.p = held_out.p = NULL;
  held.device = held_out.device = -1;
  if (a[12] != Py_None && !read_dense(a[12], t_int32, 1, "held", &held)) return NULL;
  if (a[13] != Py_None && !read_dense(a[13], t_int32, 1, "held_out", &held_out)) return NULL;
  void* stream = PyLong_AsVoidPtr(a[14]);
  if (PyErr_Occurred()) return NULL;
  if ((held.p != NULL && held.shape[0] != b) || (held_out.p != NULL && held_out.shape[0] != b))
    return refuse("held, held_out: expected as many requests as ctx_len"), NULL;
  if (new_len.shape[0] != b) return refuse("new_len: expected as many requests as ctx_len"), NULL;
  if (start.shape[0] != b + 1 || info.shape[0] != 4 || slots.shape[0] < capacity ||
      pos.shape[0] < capacity || req.shape[0] < capacity)
    return refuse("plan: buffers too small"), NULL;
  if (!ON_CURRENT_DEVICE(-1, &ctx, &new_len, &table, &free_pages, &head, &start, &slots, &pos, &req,
                         &info, &held, &held_out))
    return NULL;
  RETURN_STATUS(f_plan(ctx.p, new_len.p, b, page, table.p, stride, table.shape[1],
                       held.p, free_pages.p, free_pages.shape[0], head.p, start.p,
                       capacity, slots.p, pos.p, req.p, held_out.p, info.p, stream));
}

/* write(cache address, dtype, heads, dim, its device, k, v, slots, stream) */
static PyObject* py_write(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  Tensor k, v, slots;
  int64_t kr, kh, vr, vh;
  if (!counted(n, 9)) return NULL;
  const tern_kv_cache* cache = PyLong_AsVoidPtr(a[0]);
  const int64_t heads = integer(a[2]), dim = integer(a[3]);
  const long device = PyLong_AsLong(a[4]);
  void* stream = PyLong_AsVoidPtr(a[8]);
  if (PyErr_Occurred()) return NULL;
  if (!read_heads(a[5], a[1], heads, dim, "k", &k, &kr, &kh) ||
      !read_heads(a[6], a[1], heads, dim, "v", &v, &vr, &vh) ||
      !read_dense(a[7], t_int64, 1, "slots", &slots))
    return NULL;
  if (v.shape[0] != k.shape[0] || slots.shape[0] < k.shape[0])
    return refuse("v, slots: expected as many rows as k"), NULL;
  if (!ON_CURRENT_DEVICE(device, &k, &v, &slots)) return NULL;
  RETURN_STATUS(f_write(cache, k.p, v.p, kr, kh, vr, vh, slots.p, k.shape[0], stream));
}

/* attention(cache address, dtype, heads, dim, its device, q, table, ctx_len, row_start,
 *           max_new, mask or None, scale, out, lse or None, workspace address, its bytes, stream)
 * attention8: the same over an 8-bit cache, with the number of the rows' type behind */
static PyObject* attention(PyObject* const* a, Py_ssize_t n, int eight) {
  Tensor q, table, ctx, start, mask, out, lse;
  int64_t qr, qh, stride;
  if (!counted(n, eight ? 18 : 17)) return NULL;
  const void* cache = PyLong_AsVoidPtr(a[0]);
  const int32_t type = eight ? (int32_t)integer(a[17]) : 0;
  const int64_t heads = integer(a[2]), dim = integer(a[3]), max_new = integer(a[9]);
  const long device = PyLong_AsLong(a[4]);
  const double scale = PyFloat_AsDouble(a[11]);
  void* ws = PyLong_AsVoidPtr(a[14]);
  const size_t ws_bytes = PyLong_AsSize_t(a[15]);
  void* stream = PyLong_AsVoidPtr(a[16]);
  if (PyErr_Occurred()) return NULL;
  if (!read_heads(a[5], a[1], -1, dim, "q", &q, &qr, &qh) ||
      !read_dense(a[7], t_int32, 1, "ctx_len", &ctx) ||
      !read_table(a[6], ctx.shape[0], &table, &stride) ||
      !read_dense(a[8], t_int32, 1, "row_start", &start) ||
      !read_dense(a[12], a[1], 3, "out", &out))
    return NULL;
  const int64_t b = ctx.shape[0], t = q.shape[0], hq = q.shape[1];
  if (heads < 1 || hq < 1 || hq % heads != 0)
    return refuse("q: expected a multiple of the cache's heads"), NULL;
  if (start.shape[0] != b + 1)
    return refuse("row_start: expected one more entry than requests"), NULL;
  if (out.shape[0] != t || out.shape[1] != hq || out.shape[2] != dim)
    return refuse("out: expected [rows, query heads, dim]"), NULL;
  mask.p = NULL;
  mask.device = -1;
  mask.shape[1] = 0;
  if (a[10] != Py_None) {
    if (!read_dense(a[10], t_int64, 2, "mask", &mask)) return NULL;
    if (mask.shape[0] < t || mask.shape[1] < 1) return refuse("mask: expected [rows, words]"), NULL;
  }
  lse.p = NULL;
  lse.device = -1;
  if (a[13] != Py_None) {
    if (!read_dense(a[13], t_float32, 2, "lse", &lse)) return NULL;
    if (lse.shape[0] != t || lse.shape[1] != hq)
      return refuse("lse: expected [rows, query heads]"), NULL;
  }
  if (!ON_CURRENT_DEVICE(device, &q, &table, &ctx, &start, &out, &mask, &lse)) return NULL;
  if (eight)
    RETURN_STATUS(f_attn8(q.p, qr, qh, type, cache, table.p, stride, table.shape[1], ctx.p, start.p,
                          mask.p, mask.shape[1], b, t, hq, max_new, (float)scale, out.p, lse.p, ws,
                          ws_bytes, stream));
  RETURN_STATUS(f_attn(q.p, qr, qh, cache, table.p, stride, table.shape[1], ctx.p, start.p,
                       mask.p, mask.shape[1], b, t, hq, max_new, (float)scale, out.p,
                       lse.p, ws, ws_bytes, stream));
}

static PyObject* py_attention(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  return attention(a, n, 0);
}
static PyObject* py_attention8(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  return attention(a, n, 1);
}

/* commit(descriptions as bytes, layers, the caches' device, table, ctx_len, path, path_len, ctx_out, stream)
 * commit8: the same of 8-bit caches */
static PyObject* commit(PyObject* const* a, Py_ssize_t n, int eight) {
  Tensor table, ctx, path, len, out;
  int64_t stride;
  if (!counted(n, 9)) return NULL;
  const int64_t layers = integer(a[1]);
  const long device = PyLong_AsLong(a[2]);
  void* stream = PyLong_AsVoidPtr(a[8]);
  if (PyErr_Occurred()) return NULL;
  if (!PyBytes_Check(a[0]) ||
      PyBytes_GET_SIZE(a[0]) !=
          layers * (Py_ssize_t)(eight ? sizeof(tern_kv_cache8) : sizeof(tern_kv_cache)))
    return refuse("caches: expected a description each"), NULL;
  if (!read_dense(a[4], t_int32, 1, "ctx_len", &ctx) ||
      !read_table(a[3], ctx.shape[0], &table, &stride) ||
      !read_dense(a[5], t_int32, 2, "path", &path) ||
      !read_dense(a[6], t_int32, 1, "path_len", &len) ||
      !read_dense(a[7], t_int32, 1, "ctx_out", &out))
    return NULL;
  const int64_t b = ctx.shape[0];
  if (path.shape[0] != b || len.shape[0] != b || out.shape[0] != b)
    return refuse("path, path_len, ctx_out: expected a row each request"), NULL;
  if (!ON_CURRENT_DEVICE(device, &table, &ctx, &path, &len, &out)) return NULL;
  if (eight)
    RETURN_STATUS(f_commit8((const tern_kv_cache8*)PyBytes_AS_STRING(a[0]), layers, table.p, stride,
                            table.shape[1], ctx.p, path.p, path.shape[1], len.p, out.p, b, stream));
  RETURN_STATUS(f_commit((const tern_kv_cache*)PyBytes_AS_STRING(a[0]), layers, table.p,
                         stride, table.shape[1], ctx.p, path.p, path.shape[1], len.p,
                         out.p, b, stream));
}

static PyObject* py_commit(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  return commit(a, n, 0);
}
static PyObject* py_commit8(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  return commit(a, n, 1);
}

/* An argument that may be None: none of it, or a dense tensor. */
static int read_if(PyObject* o, PyObject* dtype, const char* name, Tensor* t) {
  t->p = NULL;
  t->device = -1;
  t->shape[0] = -1;
  return o == Py_None || read_dense(o, dtype, 1, name, t);
}

/* rotate(16-bit cache's address or 0, 8-bit cache's or 0, rows' dtype, its number, heads, dim, the
 *        cache's device, q or None, k, v, slots, positions or None, whether they have axes, turns or
 *        None, axis or None, neighbours, q_norm or None, k_norm or None, the norms' dtype, eps, out
 *        or None, stream) */
static PyObject* py_rotate(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  Tensor q, k, v, slots, pos, turns, axis, qn, kn, out;
  if (!counted(n, 22)) return NULL;
  const tern_kv_cache* cache = PyLong_AsVoidPtr(a[0]);
  const tern_kv_cache8* cache8 = PyLong_AsVoidPtr(a[1]);
  const int64_t heads = integer(a[4]), dim = integer(a[5]);
  const long device = PyLong_AsLong(a[6]);
  tern_kv_rows r = {0};
  r.dtype = (int32_t)integer(a[3]);
  const int axes = PyObject_IsTrue(a[12]);
  r.neighbours = PyObject_IsTrue(a[15]);
  r.norm_f32 = a[18] == t_float32;
  r.eps = (float)PyFloat_AsDouble(a[19]);
  void* stream = PyLong_AsVoidPtr(a[21]);
  if (PyErr_Occurred()) return NULL;
  if (!read_heads(a[8], a[2], heads, dim, "k", &k, &r.k_token_stride, &r.k_head_stride) ||
      !read_heads(a[9], a[2], heads, dim, "v", &v, &r.v_token_stride, &r.v_head_stride) ||
      !read_dense(a[10], t_int64, 1, "slots", &slots))
    return NULL;
  r.T = k.shape[0];
  if (v.shape[0] != r.T || slots.shape[0] < r.T)
    return refuse("v, slots: expected as many rows as k"), NULL;
  q.p = out.p = pos.p = NULL;
  q.device = out.device = pos.device = -1;
  if (a[7] != Py_None) {
    if (!read_heads(a[7], a[2], -1, dim, "q", &q, &r.q_token_stride, &r.q_head_stride) ||
        !read_dense(a[20], a[2], 3, "out", &out))
      return NULL;
    r.Hq = q.shape[1];
    if (q.shape[0] != r.T) return refuse("q: expected as many rows as k"), NULL;
    if (out.shape[0] != r.T || out.shape[1] != r.Hq || out.shape[2] != dim)
      return refuse("out: expected [rows, query heads, dim]"), NULL;
  }
  if (!read_if(a[13], t_int64, "turns", &turns) || !read_if(a[14], t_int32, "axis", &axis) ||
      !read_if(a[16], a[18], "q_norm", &qn) || !read_if(a[17], a[18], "k_norm", &kn))
    return NULL;
  if ((qn.p != NULL && qn.shape[0] != dim) || (kn.p != NULL && kn.shape[0] != dim))
    return refuse("q_norm, k_norm: expected a weight each element of a head"), NULL;
  if (turns.p != NULL) {
    r.rot = 2 * turns.shape[0];
    if (axis.p != NULL && axis.shape[0] != turns.shape[0])
      return refuse("axis: expected one each pair"), NULL;
    r.axes = 1;
    if (axes) {
      if (!read_tensor(a[11], t_int32, 2, "positions", &pos)) return NULL;
      r.axes = pos.shape[0];
      if (pos.shape[1] != r.T || (r.T > 1 && pos.stride[1] != 1))
        return refuse("positions: expected [axes, rows], dense along the rows"), NULL;
      r.position_stride = r.axes > 1 ? pos.stride[0] : r.T;
    } else {
      if (!read_dense(a[11], t_int32, 1, "positions", &pos)) return NULL;
      if (pos.shape[0] < r.T) return refuse("positions: expected one each row"), NULL;
    }
  }
  if (!ON_CURRENT_DEVICE(device, &q, &k, &v, &slots, &pos, &turns, &axis, &qn, &kn, &out)) return NULL;
  r.q = q.p;
  r.k = k.p;
  r.v = v.p;
  r.q_out = out.p;
  r.slots = slots.p;
  r.positions = pos.p;
  r.turns = turns.p;
  r.axis = axis.p;
  r.q_norm = qn.p;
  r.k_norm = kn.p;
  RETURN_STATUS(f_rotate(cache, cache8, &r, stream));
}

/* read(cache address, heads, dim, its device, slots, dtype, its number, k, v, stream) */
static PyObject* py_read(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  Tensor slots, k, v;
  if (!counted(n, 10)) return NULL;
  const tern_kv_cache8* cache = PyLong_AsVoidPtr(a[0]);
  const int64_t heads = integer(a[1]), dim = integer(a[2]);
  const long device = PyLong_AsLong(a[3]);
  const int32_t type = (int32_t)integer(a[6]);
  void* stream = PyLong_AsVoidPtr(a[9]);
  if (PyErr_Occurred()) return NULL;
  if (!read_dense(a[4], t_int64, 1, "slots", &slots) || !read_dense(a[7], a[5], 3, "k", &k) ||
      !read_dense(a[8], a[5], 3, "v", &v))
    return NULL;
  const int64_t t = k.shape[0];
  if (k.shape[1] != heads || k.shape[2] != dim || v.shape[0] != t || v.shape[1] != heads ||
      v.shape[2] != dim || slots.shape[0] < t)
    return refuse("k, v: expected [rows, heads, dim], a slot each row"), NULL;
  if (!ON_CURRENT_DEVICE(device, &slots, &k, &v)) return NULL;
  RETURN_STATUS(f_read(cache, slots.p, t, k.p, v.p, type, stream));
}

/* bind8(rotate_write, read, commit8, attention8), after bind */
static PyObject* py_bind8(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  if (!counted(n, 4)) return NULL;
  f_rotate = (rotate_fn)PyLong_AsVoidPtr(a[0]);
  f_read = (read_fn)PyLong_AsVoidPtr(a[1]);
  f_commit8 = (commit8_fn)PyLong_AsVoidPtr(a[2]);
  f_attn8 = (attn8_fn)PyLong_AsVoidPtr(a[3]);
  if (PyErr_Occurred()) return NULL;
  Py_RETURN_NONE;
}

/* sample(logits, dtype, its number, u, temperature or None, top_k or None, top_p or None, min_p or
 *        None, token, stream) */
static PyObject* py_sample(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  Tensor x, u, temperature, top_k, top_p, min_p, token;
  if (!counted(n, 10)) return NULL;
  const int32_t type = (int32_t)integer(a[2]);
  void* stream = PyLong_AsVoidPtr(a[9]);
  if (PyErr_Occurred()) return NULL;
  if (!read_tensor(a[0], a[1], 2, "logits", &x) || !read_dense(a[3], t_float32, 1, "u", &u) ||
      !read_if(a[4], t_float32, "temperature", &temperature) ||
      !read_if(a[5], t_int32, "top_k", &top_k) || !read_if(a[6], t_float32, "top_p", &top_p) ||
      !read_if(a[7], t_float32, "min_p", &min_p) || !read_dense(a[8], t_int32, 1, "token", &token))
    return NULL;
  const int64_t rows = x.shape[0], vocab = x.shape[1];
  if (rows > 0 && vocab > 1 && x.stride[1] != 1)
    return refuse("logits: expected to be dense along the last axis"), NULL;
  if (u.shape[0] != rows || token.shape[0] != rows ||
      (a[4] != Py_None && temperature.shape[0] != rows) || (a[5] != Py_None && top_k.shape[0] != rows) ||
      (a[6] != Py_None && top_p.shape[0] != rows) || (a[7] != Py_None && min_p.shape[0] != rows))
    return refuse("u, temperature, top_k, top_p, min_p, out: expected one number each row of logits"), NULL;
  if (!ON_CURRENT_DEVICE(-1, &x, &u, &temperature, &top_k, &top_p, &min_p, &token)) return NULL;
  RETURN_STATUS(f_sample(x.p, rows > 1 ? x.stride[0] : vocab, rows, vocab, type, u.p, temperature.p,
                         top_k.p, top_p.p, min_p.p, token.p, stream));
}

/* accept(tokens, target, parents, row_start, path, path_len, next, stream) */
static PyObject* py_accept(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  Tensor tokens, target, parent, start, path, len, next;
  if (!counted(n, 8)) return NULL;
  void* stream = PyLong_AsVoidPtr(a[7]);
  if (PyErr_Occurred()) return NULL;
  if (!read_dense(a[0], t_int32, 1, "tokens", &tokens) ||
      !read_dense(a[1], t_int32, 1, "target", &target) ||
      !read_dense(a[2], t_int32, 1, "parents", &parent) ||
      !read_dense(a[3], t_int32, 1, "row_start", &start) ||
      !read_dense(a[4], t_int32, 2, "path", &path) || !read_dense(a[5], t_int32, 1, "path_len", &len) ||
      !read_dense(a[6], t_int32, 1, "next", &next))
    return NULL;
  const int64_t t = tokens.shape[0], b = start.shape[0] - 1;
  if (b < 0) return refuse("row_start: expected one more entry than requests"), NULL;
  if (target.shape[0] != t || parent.shape[0] != t)
    return refuse("target, parents: expected one each token"), NULL;
  if (path.shape[0] != b || len.shape[0] != b || next.shape[0] != b)
    return refuse("path, path_len, next: expected a row each request"), NULL;
  if (!ON_CURRENT_DEVICE(-1, &tokens, &target, &parent, &start, &path, &len, &next)) return NULL;
  RETURN_STATUS(f_accept(tokens.p, target.p, parent.p, start.p, b, t, path.shape[1], path.p, len.p,
                         next.p, stream));
}

/* bind_tokens(sample, accept), after bind */
static PyObject* py_bind_tokens(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  if (!counted(n, 2)) return NULL;
  f_sample = (sample_fn)PyLong_AsVoidPtr(a[0]);
  f_accept = (accept_fn)PyLong_AsVoidPtr(a[1]);
  if (PyErr_Occurred()) return NULL;
  Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"bind", (PyCFunction)(void (*)(void))py_bind, METH_FASTCALL, NULL},
    {"plan", (PyCFunction)(void (*)(void))py_plan, METH_FASTCALL, NULL},
    {"write", (PyCFunction)(void (*)(void))py_write, METH_FASTCALL, NULL},
    {"attention", (PyCFunction)(void (*)(void))py_attention, METH_FASTCALL, NULL},
    {"commit", (PyCFunction)(void (*)(void))py_commit, METH_FASTCALL, NULL},
    {"bind8", (PyCFunction)(void (*)(void))py_bind8, METH_FASTCALL, NULL},
    {"rotate", (PyCFunction)(void (*)(void))py_rotate, METH_FASTCALL, NULL},
    {"read", (PyCFunction)(void (*)(void))py_read, METH_FASTCALL, NULL},
    {"attention8", (PyCFunction)(void (*)(void))py_attention8, METH_FASTCALL, NULL},
    {"commit8", (PyCFunction)(void (*)(void))py_commit8, METH_FASTCALL, NULL},
    {"bind_tokens", (PyCFunction)(void (*)(void))py_bind_tokens, METH_FASTCALL, NULL},
    {"sample", (PyCFunction)(void (*)(void))py_sample, METH_FASTCALL, NULL},
    {"accept", (PyCFunction)(void (*)(void))py_accept, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kvcall", NULL, -1, methods};

PyMODINIT_FUNC PyInit__kvcall(void) {
  s_is_cuda = PyUnicode_InternFromString("is_cuda");
  s_dtype = PyUnicode_InternFromString("dtype");
  s_shape = PyUnicode_InternFromString("shape");
  s_stride = PyUnicode_InternFromString("stride");
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  s_get_device = PyUnicode_InternFromString("get_device");
  if (!s_is_cuda || !s_dtype || !s_shape || !s_stride || !s_data_ptr || !s_get_device) return NULL;
  return PyModule_Create(&module);
}
