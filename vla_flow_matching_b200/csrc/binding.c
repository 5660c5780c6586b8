/*
 * Argument marshalling of the paged-cache calls for Python: tensors to pointers, sizes and
 * strides, their checks, and the call into libpi0x.  These calls take a few microseconds on
 * the GPU, less than a marshalling of their ten to fifteen arguments in Python itself
 * (measured, one token of one sample: 12.5 us a call through ctypes).  pi0x.py has the
 * functions a user calls and their documentation.
 *
 * Tensors are read through DLPack's C exchange interface, which the tensor type hands out, and
 * nothing of torch is linked.  (Their Python attributes one by one cost 0.7 to
 * 1.7 us a call more: 8.2 for an attention call against 7.5, 6.8 for a write against 5.2.)
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/dlpack.h>

#include "../../include/pi0x.h"

static const DLPackExchangeAPI *api;
static PyObject *s_new_empty;
static PyObject *t_tensor, *t_bf16, *t_f32, *t_u8;  /* torch's tensor type and dtypes */
static PyObject *f_empty_like, *f_device, *f_fail;  /* callables, see setup() */
static PyObject *kw_contiguous, *v_contiguous, *kw_dtype;

/* Element types by DLPack's code and bits. */
enum {
  kBf16 = kDLBfloat << 8 | 16,
  kF32 = kDLFloat << 8 | 32,
  kI32 = kDLInt << 8 | 32,
  kU8 = kDLUInt << 8 | 8,
  kBool = kDLBool << 8 | 8
};

typedef struct {
  char *data;
  int dtype, ndim;
  int64_t shape[5], stride[5];
  long device; /* -1: not a CUDA device */
} View;

static int as_int(PyObject *o) {
  const long v = PyLong_AsLong(o);
  if (v < INT32_MIN || v > INT32_MAX) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_OverflowError, "an integer argument of 2^31 or more");
    return -1;
  }
  return (int)v;
}

static int view(PyObject *t, View *v) {
  DLTensor d;
  if (!PyObject_TypeCheck(t, (PyTypeObject *)t_tensor)) {
    PyErr_Format(PyExc_AttributeError, "a tensor is expected, not %s", Py_TYPE(t)->tp_name);
    return -1;
  }
  if (api->dltensor_from_py_object_no_sync(t, &d)) return -1;
  if (d.ndim > 5) {
    PyErr_SetString(PyExc_ValueError, "tensors of at most 5 dimensions are taken");
    return -1;
  }
  v->data = (char *)d.data + d.byte_offset;
  v->dtype = d.dtype.code << 8 | d.dtype.bits;
  v->ndim = d.ndim;
  for (int i = 0; i < d.ndim; ++i) v->shape[i] = d.shape[i], v->stride[i] = d.strides[i];
  v->device = d.device.device_type == kDLCUDA ? d.device.device_id : -1;
  return 0;
}

static int contiguous(const View *v) {
  int64_t want = 1;
  for (int i = v->ndim - 1; i >= 0; --i) {
    if (v->shape[i] == 0) return 1;
    if (v->shape[i] != 1 && v->stride[i] != want) return 0;
    want *= v->shape[i];
  }
  return 1;
}

/* A view of `t`, on the device of the call (*device < 0: not known yet). */
static int take(const char *what, PyObject *t, View *v, long *device) {
  if (view(t, v)) return -1;
  if (v->device < 0) {
    PyErr_Format(PyExc_ValueError, "%s: every tensor must be on a CUDA device", what);
    return -1;
  }
  if (*device >= 0 && v->device != *device) {
    PyErr_Format(PyExc_ValueError, "%s: tensors on cuda:%ld and cuda:%ld", what, *device, v->device);
    return -1;
  }
  *device = v->device;
  return 0;
}

static int has_shape(const View *v, int n, const int64_t *shape) {
  if (v->ndim != n) return 0;
  for (int i = 0; i < n; ++i)
    if (v->shape[i] != shape[i]) return 0;
  return 1;
}

/* The stride of dimension i; 0 where its size is 1, since torch leaves such strides at any value
 * and the library wants whole 16 bytes. */
static int64_t stride_of(const View *v, int i) { return v->shape[i] > 1 ? v->stride[i] : 0; }

/* A view as (B, T, heads, D) rows of `dtype` with a contiguous last dimension. */
static int rows_of(const char *what, const char *name, const View *v, int64_t B, int64_t T, int64_t heads, int64_t D,
                   int dtype, pi0x_rows *r) {
  const int64_t shape[4] = {B, T, heads, D};
  if (!has_shape(v, 4, shape) || v->dtype != dtype || v->stride[3] != 1) {
    PyErr_Format(PyExc_ValueError,
                 "%s: %s must be (%lld, %lld, %lld, %lld) rows of the keys' or queries' type (%s) with a contiguous last "
                 "dimension",
                 what, name, (long long)B, (long long)T, (long long)heads, (long long)D,
                 dtype == kF32 ? "float32" : "bfloat16");
    return -1;
  }
  r->data = v->data;
  r->batch_stride = stride_of(v, 0);
  r->token_stride = stride_of(v, 1);
  r->head_stride = stride_of(v, 2);
  return 0;
}
static int take_rows(const char *what, const char *name, PyObject *t, int64_t B, int64_t T, int64_t heads, int64_t D,
                     int dtype, pi0x_rows *r, long *device) {
  View v;
  return take(what, t, &v, device) || rows_of(what, name, &v, B, T, heads, D, dtype, r) ? -1 : 0;
}

/* Contiguous int32 tensor of n dimensions, or None (*p = NULL). */
static int take_ints(const char *what, const char *name, PyObject *t, int n, const int64_t *shape, const int32_t **p,
                     long *device) {
  View v;
  *p = NULL;
  if (t == Py_None) return 0;
  if (take(what, t, &v, device)) return -1;
  if (v.dtype != kI32 || !has_shape(&v, n, shape) || !contiguous(&v)) {
    if (n == 1)
      PyErr_Format(PyExc_ValueError, "%s: %s must be a contiguous int32 tensor of shape (%lld,)", what, name,
                   (long long)shape[0]);
    else
      PyErr_Format(PyExc_ValueError, "%s: %s must be a contiguous int32 tensor of shape (%lld, %lld)", what, name,
                   (long long)shape[0], (long long)shape[1]);
    return -1;
  }
  *p = (const int32_t *)v.data;
  return 0;
}

static int take_gain(const char *what, PyObject *t, int64_t D, const float **p, long *device) {
  View v;
  *p = NULL;
  if (t == Py_None) return 0;
  if (take(what, t, &v, device)) return -1;
  if (v.dtype != kF32 || !has_shape(&v, 1, &D) || !contiguous(&v)) {
    PyErr_Format(PyExc_ValueError, "%s: a gain is a contiguous float32 tensor of shape (%lld,)", what, (long long)D);
    return -1;
  }
  *p = (const float *)v.data;
  return 0;
}

/* Page table (B, max_pages): *B < 0 takes the table's. */
static int take_table(const char *what, PyObject *t, int64_t *B, const int32_t **p, int *max_pages, long *device) {
  View v;
  if (take(what, t, &v, device)) return -1;
  if (v.dtype != kI32 || v.ndim != 2 || (*B >= 0 && v.shape[0] != *B) || v.shape[1] > INT32_MAX || !contiguous(&v)) {
    PyErr_Format(PyExc_ValueError, "%s: table must be a contiguous int32 tensor of shape (batch, max_pages)", what);
    return -1;
  }
  *B = v.shape[0];
  *p = (const int32_t *)v.data;
  *max_pages = (int)v.shape[1];
  return 0;
}

/* (B, length) uint8 or bool mask, length `least` or more, or None (NULL, 0). */
static int take_mask(const char *what, PyObject *t, int64_t B, int least, const uint8_t **p, int64_t *length, int *dtype,
                     long *device) {
  View v;
  *p = NULL;
  *length = 0;
  *dtype = 0;
  if (t == Py_None) return 0;
  if (take(what, t, &v, device)) return -1;
  if ((v.dtype != kU8 && v.dtype != kBool) || v.ndim != 2 || v.shape[0] != B || v.shape[1] < least ||
      v.shape[1] > INT32_MAX || !contiguous(&v)) {
    PyErr_Format(PyExc_ValueError, "%s: mask must be a contiguous uint8 or bool tensor of shape (%lld, %d or more)", what,
                 (long long)B, least);
    return -1;
  }
  *p = (const uint8_t *)v.data;
  *length = v.shape[1];
  *dtype = v.dtype;
  return 0;
}

static int fits(const char *what, int64_t a, int64_t b, int64_t c) {
  if (a <= INT32_MAX && b <= INT32_MAX && c <= INT32_MAX) return 0;
  PyErr_Format(PyExc_ValueError, "%s: a size of 2^31 or more", what);
  return -1;
}

/* bf16 or f32 rows: the library's code, or -1. */
static int row_type(const char *what, int dtype) {
  if (dtype == kBf16) return PI0X_DTYPE_BF16;
  if (dtype == kF32) return PI0X_DTYPE_F32;
  PyErr_Format(PyExc_ValueError, "%s: rows are bfloat16 or float32", what);
  return -1;
}

/* 1 if `device` is the current one, 0 if another is, -1 on error. */
static int is_current(long device) {
  PyObject *now = PyObject_CallNoArgs(f_device);
  if (!now) return -1;
  const long d = PyLong_AsLong(now);
  Py_DECREF(now);
  return d == -1 && PyErr_Occurred() ? -1 : d == device;
}

static int current_stream(long device, void **stream) {
  return api->current_work_stream(kDLCUDA, (int32_t)device, stream);
}

/* A new contiguous tensor like `t`, whose view is `v`. */
static PyObject *new_like(PyObject *t, const View *v) {
  if (contiguous(v)) return PyObject_CallOneArg(f_empty_like, t);
  PyObject *args[2] = {t, v_contiguous};
  return PyObject_Vectorcall(f_empty_like, args, 1, kw_contiguous);
}

static PyObject *tuple_of(int n, const int64_t *x) {
  PyObject *r = PyTuple_New(n);
  for (int i = 0; r && i < n; ++i) {
    PyObject *o = PyLong_FromLongLong(x[i]);
    if (o)
      PyTuple_SET_ITEM(r, i, o);
    else
      Py_CLEAR(r);
  }
  return r;
}
/* A new contiguous tensor of n dimensions (n <= 5) on the device of `on`
 * (on.new_empty_strided(): half a microsecond less host time than on.new_empty()). */
static PyObject *new_tensor(PyObject *on, int n, const int64_t *shape, PyObject *dtype) {
  int64_t stride[5], next = 1;
  for (int i = n - 1; i >= 0; --i) stride[i] = next, next *= shape[i] > 1 ? shape[i] : 1;
  PyObject *size = tuple_of(n, shape), *strides = size ? tuple_of(n, stride) : NULL, *r = NULL;
  if (strides) {
    PyObject *args[4] = {on, size, strides, dtype};
    r = PyObject_VectorcallMethod(s_new_empty, args, 3, kw_dtype);
  }
  Py_XDECREF(size);
  Py_XDECREF(strides);
  return r;
}

/* An output: `given`, or a new tensor like `like`; its rows. */
static PyObject *out_rows(const char *what, const char *name, PyObject *given, PyObject *like, const View *v, int64_t B,
                          int64_t T, int64_t heads, int64_t D, int dtype, pi0x_rows *r, long *device) {
  if (given != Py_None) return take_rows(what, name, given, B, T, heads, D, dtype, r, device) ? NULL : Py_NewRef(given);
  PyObject *t = new_like(like, v);
  View made;
  if (!t || view(t, &made)) {
    Py_XDECREF(t);
    return NULL;
  }
  r->data = made.data;
  r->batch_stride = T * heads * D;
  r->token_stride = heads * D;
  r->head_stride = D;
  return t;
}

static int done(int status, const char *what) {
  if (status == PI0X_OK) return 0;
  PyObject *r = PyObject_CallFunction(f_fail, "is", status, what);
  Py_XDECREF(r);
  if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, what);
  return -1;
}

static int arity(const char *what, Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return 0;
  PyErr_Format(PyExc_TypeError, "%s: %zd arguments, not %zd", what, n, want);
  return -1;
}

static int rotation(const char *what, PyObject *positions, PyObject *q_gain, PyObject *k_gain, PyObject *eps,
                    PyObject *base, int64_t B, int64_t T, int64_t D, pi0x_rotation *r, long *device) {
  const int64_t bt[2] = {B, T};
  if (take_gain(what, q_gain, D, &r->q_gain, device) || take_gain(what, k_gain, D, &r->k_gain, device) ||
      take_ints(what, "positions", positions, 2, bt, &r->positions, device))
    return -1;
  r->eps = (float)PyFloat_AsDouble(eps);
  r->rope_base = base == Py_None ? 0.0f : (float)PyFloat_AsDouble(base);
  return PyErr_Occurred() ? -1 : 0;
}

/* Every call below returns NotImplemented, before it has done anything, where another device
 * than the tensors' is current. */

/* qk_norm_rope(q, k, start, positions, q_gain, k_gain, eps, rope_base, q_out, k_out) -> (q_out, k_out) */
static PyObject *py_qk_norm_rope(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  static const char what[] = "qk_norm_rope";
  (void)self;
  if (arity(what, n, 10)) return NULL;
  long device = -1;
  View q, k;
  pi0x_rows rq, rk, rqo, rko;
  pi0x_rotation rot;
  const int32_t *start;
  const int has_k = a[1] != Py_None;
  if (take(what, a[0], &q, &device) || (has_k && take(what, a[1], &k, &device))) return NULL;
  const int dtype = row_type(what, q.dtype);
  if (dtype < 0) return NULL;
  if (q.ndim != 4 || (has_k && k.ndim != 4)) {
    PyErr_Format(PyExc_ValueError, "%s: q and k are (batch, tokens, heads, head_dim)", what);
    return NULL;
  }
  const int64_t B = q.shape[0], T = q.shape[1], heads = q.shape[2], D = q.shape[3], kv = has_k ? k.shape[2] : 0;
  if (fits(what, B, T, heads) || fits(what, kv, D, 0) ||
      rows_of(what, "q", &q, B, T, heads, D, q.dtype, &rq) ||
      (has_k && rows_of(what, "k", &k, B, T, kv, D, q.dtype, &rk)) ||
      take_ints(what, "start", a[2], 1, &B, &start, &device) ||
      rotation(what, a[3], a[4], a[5], a[6], a[7], B, T, D, &rot, &device))
    return NULL;
  const int here = is_current(device);
  if (here <= 0) return here < 0 ? NULL : Py_NewRef(Py_NotImplemented);
  PyObject *qo = out_rows(what, "q_out", a[8], a[0], &q, B, T, heads, D, q.dtype, &rqo, &device), *ko = NULL, *r = NULL;
  if (!qo) return NULL;
  ko = has_k ? out_rows(what, "k_out", a[9], a[1], &k, B, T, kv, D, q.dtype, &rko, &device) : Py_NewRef(Py_None);
  if (!ko) goto out;
  if (B != 0 && T != 0 && heads + kv != 0) {
    void *stream;
    int st;
    if (current_stream(device, &stream)) goto out;
    Py_BEGIN_ALLOW_THREADS
    st = pi0x_qk_norm_rope(dtype, (int)B, (int)T, (int)heads, (int)kv, (int)D, &rq, has_k ? &rk : NULL, start, &rot,
                           &rqo, has_k ? &rko : NULL, stream);
    Py_END_ALLOW_THREADS
    if (done(st, "pi0x_qk_norm_rope")) goto out;
  }
  r = PyTuple_Pack(2, qo, ko);
out:
  Py_DECREF(qo);
  Py_XDECREF(ko);
  return r;
}

static const pi0x_cache *cache_of(PyObject *address) { return (const pi0x_cache *)PyLong_AsVoidPtr(address); }

/* cache_write(cache, device, layer, k, v, table, start, count, q, q_out, positions, q_gain, k_gain, eps, rope_base) -> q_out */
static PyObject *py_cache_write(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  static const char what[] = "KVCache.write";
  (void)self;
  if (arity(what, n, 15)) return NULL;
  const pi0x_cache *c = cache_of(a[0]);
  long device = PyLong_AsLong(a[1]);
  const int layer = as_int(a[2]);
  if (PyErr_Occurred()) return NULL;
  View k, q;
  pi0x_rows rk, rv, rq, rqo;
  pi0x_rotation rot;
  const int32_t *table, *start, *count;
  int max_pages, rotate = 0;
  const int has_q = a[8] != Py_None;
  if (take(what, a[3], &k, &device) || (has_q && take(what, a[8], &q, &device))) return NULL;
  const int dtype = row_type(what, k.dtype);
  if (dtype < 0) return NULL;
  if (k.ndim != 4 || (has_q && q.ndim != 4) || a[6] == Py_None) {
    PyErr_Format(PyExc_ValueError, "%s: q, k and v are (batch, tokens, heads, head_dim), and start is required", what);
    return NULL;
  }
  int64_t B = k.shape[0];
  const int64_t T = k.shape[1], D = c->head_dim, heads = has_q ? q.shape[2] : 0;
  if (fits(what, B, T, heads) || rows_of(what, "k", &k, B, T, c->kv_heads, D, k.dtype, &rk) ||
      take_rows(what, "v", a[4], B, T, c->kv_heads, D, k.dtype, &rv, &device) ||
      (has_q && rows_of(what, "q", &q, B, T, heads, D, k.dtype, &rq)) ||
      take_table(what, a[5], &B, &table, &max_pages, &device) ||
      take_ints(what, "start", a[6], 1, &B, &start, &device) || take_ints(what, "count", a[7], 1, &B, &count, &device))
    return NULL;
  if (rotation(what, a[10], a[11], a[12], a[13], a[14], B, T, D, &rot, &device)) return NULL;
  rotate = has_q || rot.rope_base != 0.0f || rot.q_gain || rot.k_gain;
  const int here = is_current(device);
  if (here <= 0) return here < 0 ? NULL : Py_NewRef(Py_NotImplemented);
  PyObject *qo = has_q ? out_rows(what, "q_out", a[9], a[8], &q, B, T, heads, D, k.dtype, &rqo, &device) : Py_NewRef(Py_None);
  if (!qo) return NULL;
  if (B * T != 0) {
    void *stream;
    int st;
    if (current_stream(device, &stream)) goto fail;
    Py_BEGIN_ALLOW_THREADS
    st = pi0x_cache_write(c, layer, dtype, (int)B, (int)T, &rk, &rv, table, max_pages, start, count, rotate ? &rot : NULL,
                          (int)heads, has_q && heads ? &rq : NULL, has_q && heads ? &rqo : NULL, stream);
    Py_END_ALLOW_THREADS
    if (done(st, "pi0x_cache_write")) goto fail;
  }
  return qo;
fail:
  Py_DECREF(qo);
  return NULL;
}

/* An output of given shape and type: `given` if it is one, else new (`like` a contiguous tensor of
 * that shape and type, or NULL; `on` any tensor on the device); its memory in *p. */
static PyObject *out_tensor(const char *what, const char *name, PyObject *given, PyObject *like, PyObject *on, int n,
                            const int64_t *shape, int dtype, long *device, void **p) {
  View v;
  if (given == Py_None) {
    PyObject *t = like ? PyObject_CallOneArg(f_empty_like, like)
                       : new_tensor(on, n, shape, dtype == kBf16 ? t_bf16 : dtype == kF32 ? t_f32 : t_u8);
    if (!t || view(t, &v)) {
      Py_XDECREF(t);
      return NULL;
    }
    *p = v.data;
    return t;
  }
  if (take(what, given, &v, device)) return NULL;
  if (v.dtype != dtype || !has_shape(&v, n, shape) || !contiguous(&v)) {
    PyErr_Format(PyExc_ValueError, "%s: %s has another shape or type than the call's, or is not contiguous", what, name);
    return NULL;
  }
  *p = v.data;
  return Py_NewRef(given);
}

/* cache_read(cache, device, table, lens, length, mask, layer0, layers, dtype, k_out, v_out, mask_out) -> (k, v, mask) */
static PyObject *py_cache_read(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  static const char what[] = "KVCache.read";
  (void)self;
  if (arity(what, n, 12)) return NULL;
  const pi0x_cache *c = cache_of(a[0]);
  long device = PyLong_AsLong(a[1]);
  const int length = as_int(a[4]), layer0 = as_int(a[6]), layers = as_int(a[7]);
  if (PyErr_Occurred()) return NULL;
  int64_t B = -1, mask_len;
  const int32_t *table, *lens;
  const uint8_t *mask;
  int mask_type;
  int max_pages;
  const int type = a[8] == t_bf16 ? kBf16 : a[8] == t_f32 ? kF32 : 0, dtype = row_type(what, type);
  if (dtype < 0) return NULL;
  if (length < 0 || layers < 0) {
    PyErr_Format(PyExc_ValueError, "%s: %d layers of %d slots", what, layers, length);
    return NULL;
  }
  if (take_table(what, a[2], &B, &table, &max_pages, &device) || fits(what, B, 0, 0) ||
      take_ints(what, "lens", a[3], 1, &B, &lens, &device) || take_mask(what, a[5], B, 0, &mask, &mask_len, &mask_type, &device))
    return NULL;
  if (a[3] == Py_None || (a[5] != Py_None && mask_len != length)) {
    PyErr_Format(PyExc_ValueError, "%s: lens is required, and a mask covers the %d slots read", what, length);
    return NULL;
  }
  const int here = is_current(device);
  if (here <= 0) return here < 0 ? NULL : Py_NewRef(Py_NotImplemented);
  const int64_t shape[5] = {layers, B, c->kv_heads, length, c->head_dim}, mshape[2] = {B, length};
  void *pk, *pv, *pm;
  PyObject *k = out_tensor(what, "k_out", a[9], NULL, a[2], 5, shape, type, &device, &pk), *r = NULL;
  PyObject *v = k ? out_tensor(what, "v_out", a[10], k, a[2], 5, shape, type, &device, &pv) : NULL;
  PyObject *like = mask && mask_type == kU8 ? a[5] : NULL;
  PyObject *m = v ? out_tensor(what, "mask_out", a[11], like, a[2], 2, mshape, kU8, &device, &pm) : NULL;
  if (!m) goto out;
  if (B * length != 0) {
    void *stream;
    int st;
    if (current_stream(device, &stream)) goto out;
    Py_BEGIN_ALLOW_THREADS
    st = pi0x_cache_read(c, layer0, layers, (int)B, length, table, max_pages, lens, mask, dtype, pk, pv, (uint8_t *)pm,
                         stream);
    Py_END_ALLOW_THREADS
    if (done(st, "pi0x_cache_read")) goto out;
  }
  r = PyTuple_Pack(3, k, v, m);
out:
  Py_XDECREF(k);
  Py_XDECREF(v);
  Py_XDECREF(m);
  return r;
}

/* cache_attention(cache, device, layer, q, table, lens, mask, scale, out, lse) -> (out, lse) */
static PyObject *py_cache_attention(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  static const char what[] = "KVCache.attend";
  (void)self;
  if (arity(what, n, 10)) return NULL;
  const pi0x_cache *c = cache_of(a[0]);
  long device = PyLong_AsLong(a[1]);
  const int layer = as_int(a[2]);
  const double scale = PyFloat_AsDouble(a[7]);
  if (PyErr_Occurred()) return NULL;
  View q;
  const int32_t *table, *lens;
  const uint8_t *mask;
  int mask_type;
  int64_t mask_len;
  int max_pages;
  if (take(what, a[3], &q, &device)) return NULL;
  if (q.ndim != 3 || q.dtype != kBf16 || q.shape[2] != c->head_dim || q.stride[2] != 1) {
    PyErr_Format(PyExc_ValueError, "%s: q must be (batch, heads, %d) bfloat16 with a contiguous last dimension", what,
                 c->head_dim);
    return NULL;
  }
  int64_t B = q.shape[0];
  const int64_t heads = q.shape[1];
  if (fits(what, B, heads, 0) || take_table(what, a[4], &B, &table, &max_pages, &device) ||
      take_ints(what, "lens", a[5], 1, &B, &lens, &device) || take_mask(what, a[6], B, 1, &mask, &mask_len, &mask_type, &device))
    return NULL;
  if (a[5] == Py_None) {
    PyErr_Format(PyExc_ValueError, "%s: lens is required", what);
    return NULL;
  }
  const int here = is_current(device);
  if (here <= 0) return here < 0 ? NULL : Py_NewRef(Py_NotImplemented);
  void *po, *pl, *pw = NULL;
  PyObject *out = NULL, *lse = NULL, *work = NULL, *r = NULL;
  if (a[8] == Py_None) {
    pi0x_rows ro;
    out = out_rows(what, "out", a[8], a[3], &q, B, 1, heads, c->head_dim, kBf16, &ro, &device);
    po = ro.data;
  } else {
    out = out_tensor(what, "out", a[8], NULL, a[3], 3, q.shape, kBf16, &device, &po);
  }
  if (!out || !(lse = out_tensor(what, "lse", a[9], NULL, a[3], 2, q.shape, kF32, &device, &pl))) goto out;
  if (B * heads != 0) {
    /* a workspace of this call alone, from torch's allocator on the current stream */
    const size_t need = pi0x_cache_attention_workspace(c, (int)B, (int)heads, max_pages);
    const int64_t size = (int64_t)need;
    if (need && !(work = out_tensor(what, "workspace", Py_None, NULL, a[3], 1, &size, kU8, &device, &pw))) goto out;
    const pi0x_rows rq = {q.data, stride_of(&q, 0), 0, stride_of(&q, 1)};
    void *stream;
    int st;
    if (current_stream(device, &stream)) goto out;
    Py_BEGIN_ALLOW_THREADS
    st = pi0x_cache_attention(c, layer, (int)B, (int)heads, &rq, table, max_pages, lens, mask, (int)mask_len, (float)scale,
                              po, (float *)pl, pw, need, stream);
    Py_END_ALLOW_THREADS
    if (done(st, "pi0x_cache_attention")) goto out;
  }
  r = PyTuple_Pack(2, out, lse);
out:
  Py_XDECREF(out);
  Py_XDECREF(lse);
  Py_XDECREF(work);
  return r;
}

/* setup(torch, fail): what the calls above use of torch, and the function that raises for a status. */
static PyObject *py_setup(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  if (arity("setup", n, 2)) return NULL;
  PyObject *torch = a[0], *low = PyObject_GetAttrString(torch, "_C");
  if (!low) return NULL;
  f_fail = Py_NewRef(a[1]);
  t_tensor = PyObject_GetAttrString(torch, "Tensor");
  t_bf16 = PyObject_GetAttrString(torch, "bfloat16");
  t_f32 = PyObject_GetAttrString(torch, "float32");
  t_u8 = PyObject_GetAttrString(torch, "uint8");
  f_empty_like = PyObject_GetAttrString(torch, "empty_like");
  v_contiguous = PyObject_GetAttrString(torch, "contiguous_format");
  f_device = PyObject_GetAttrString(low, "_cuda_getDevice");
  kw_contiguous = Py_BuildValue("(s)", "memory_format");
  kw_dtype = Py_BuildValue("(s)", "dtype");
  Py_DECREF(low);
  PyObject *capsule = t_tensor ? PyObject_GetAttrString(t_tensor, "__dlpack_c_exchange_api__") : NULL;
  if (!capsule) {
    PyErr_SetString(PyExc_ImportError, "this torch does not hand out DLPack's C exchange interface (2.11 does)");
    return NULL;
  }
  api = PyCapsule_GetPointer(capsule, "dlpack_exchange_api"); /* lives as long as the process */
  Py_DECREF(capsule);
  if (api && (api->header.version.major != DLPACK_MAJOR_VERSION || !api->dltensor_from_py_object_no_sync ||
              !api->current_work_stream))
    PyErr_SetString(PyExc_ImportError, "this torch has another DLPack exchange interface than the one built against");
  if (PyErr_Occurred()) return NULL;
  Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"setup", (PyCFunction)(void (*)(void))py_setup, METH_FASTCALL, NULL},
    {"qk_norm_rope", (PyCFunction)(void (*)(void))py_qk_norm_rope, METH_FASTCALL, NULL},
    {"cache_write", (PyCFunction)(void (*)(void))py_cache_write, METH_FASTCALL, NULL},
    {"cache_read", (PyCFunction)(void (*)(void))py_cache_read, METH_FASTCALL, NULL},
    {"cache_attention", (PyCFunction)(void (*)(void))py_cache_attention, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__binding(void) {
  s_new_empty = PyUnicode_InternFromString("new_empty_strided");
  if (!s_new_empty) return NULL;
  return PyModule_Create(&module);
}
