/* Argument marshalling of the attention operators' Python calls: checks the
 * tensors, describes them to the C ABI (include/moe_attn.h) and calls it. Small
 * calls are bound by this work (an append of 64 tokens took 13 us of host time
 * through ctypes, 4 us of GPU time), so it is done here. Tensors are read
 * through their Python attributes; nothing of torch's own ABI is used. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <limits.h>
#include <math.h>

#include "../../include/moe_attn.h"

typedef int (*rope_fn)(const moe_attn_rows*, const moe_attn_rows*, const int32_t*, int32_t, int32_t,
                       int32_t, int32_t, const moe_attn_rotation*, void*);
typedef int (*append_fn)(moe_attn_handle*, const moe_attn_rows*, const moe_attn_rows*,
                         const moe_attn_rows*, const moe_attn_rows*, const int32_t*,
                         const int64_t*, int32_t, const moe_attn_rotation*, const moe_attn_cache*,
                         void*);
typedef int (*forward_fn)(moe_attn_handle*, const moe_attn_rows*, const moe_attn_rows*, float*,
                          const moe_attn_cache*, const moe_attn_batch*, const moe_attn_scores*,
                          void*);

static struct {
  rope_fn rope;
  append_fn append;
  forward_fn forward;
  PyObject *check;                       /* (status, what): raises */
  PyObject *empty, *raw_stream, *current_device;
  PyObject *grad_enabled, *inference_enabled; /* of the thread */
  PyObject *increment_version;           /* (tensors): they were written to */
  PyObject *bf16, *fp16, *f32, *i32, *i64;
  PyObject *shape, *stride, *dtype, *device, *get_device, *data_ptr, *is_contiguous,
      *requires_grad;
  PyObject *empty_names;                 /* ("dtype", "device") */
} G;

typedef struct {
  moe_attn_handle* handle;
  long long q_heads, kv_heads, dim, page;
  long index;
  PyObject *dtype, *device;
} layer_t;

#define MAX_DIMS 8

static int from_tuple(PyObject* t, long long* d) {
  if (!t) return -1;
  int n = -1;
  if (PyTuple_Check(t)) {
    n = (int)PyTuple_GET_SIZE(t);
    for (int i = 0; i < n && i < MAX_DIMS; ++i) d[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(t, i));
  } else {
    PyErr_SetString(PyExc_ValueError, "a tensor was expected");
  }
  Py_DECREF(t);
  return PyErr_Occurred() ? -1 : n;
}

static int shape_of(PyObject* t, long long* d) { return from_tuple(PyObject_GetAttr(t, G.shape), d); }

static PyObject* method(PyObject* t, PyObject* name) {
  return PyObject_VectorcallMethod(name, &t, 1 | PY_VECTORCALL_ARGUMENTS_OFFSET, NULL);
}

static int strides_of(PyObject* t, long long* d) { return from_tuple(method(t, G.stride), d); }

static int pointer_of(PyObject* t, void** p) {
  PyObject* v = method(t, G.data_ptr);
  if (!v) return -1;
  *p = PyLong_AsVoidPtr(v);
  Py_DECREF(v);
  return PyErr_Occurred() ? -1 : 0;
}

/* 1: the tensor has this type and lies on this device; 0: not; -1: an error */
static int placed(PyObject* t, PyObject* dtype, long index) {
  PyObject* d = PyObject_GetAttr(t, G.dtype);
  if (!d) return -1;
  const int same = d == dtype;
  Py_DECREF(d);
  if (!same) return 0;
  PyObject* v = method(t, G.get_device);
  if (!v) return -1;
  const long on = PyLong_AsLong(v);
  Py_DECREF(v);
  return PyErr_Occurred() ? -1 : on == index;
}

static int refuse_place(PyObject* t, const char* what, PyObject* dtype, long index) {
  if (PyErr_Occurred()) return -1;
  PyObject* d = PyObject_GetAttr(t, G.dtype);
  PyObject* on = PyObject_GetAttr(t, G.device);
  if (d && on)
    PyErr_Format(PyExc_ValueError, "%s must be %S on cuda:%ld, got %S on %S", what, dtype, index, d,
                 on);
  Py_XDECREF(d);
  Py_XDECREF(on);
  return -1;
}

/* t [tokens, heads, dim] -> r; the number of tokens, or -1 */
static long long rows_of(PyObject* t, long long heads, long long dim, PyObject* dtype, long index,
                         moe_attn_rows* r, const char* what) {
  long long d[MAX_DIMS], s[MAX_DIMS];
  const int n = shape_of(t, d);
  if (n < 0) return -1;
  if (n != 3 || d[1] != heads || d[2] != dim) {
    PyErr_Format(PyExc_ValueError, "%s must be [tokens, %lld, %lld]", what, heads, dim);
    return -1;
  }
  if (placed(t, dtype, index) != 1) return refuse_place(t, what, dtype, index);
  if (strides_of(t, s) != 3) return -1;
  if (s[2] != 1 && dim > 1) {
    PyErr_Format(PyExc_ValueError, "%s must be contiguous along head_dim", what);
    return -1;
  }
  if (d[0] > INT_MAX) {
    PyErr_Format(PyExc_ValueError, "%s has too many tokens", what);
    return -1;
  }
  /* the stride of a dimension of one element says nothing */
  r->head_stride = heads > 1 ? s[1] : dim;
  r->token_stride = d[0] > 1 ? s[0] : heads * r->head_stride;
  return pointer_of(t, &r->data) ? -1 : d[0];
}

/* t, a contiguous vector of n elements (n < 0: any number); its length or -1 */
static long long vector_of(PyObject* t, long long n, PyObject* dtype, long index, const void** p,
                           const char* what) {
  long long d[MAX_DIMS];
  const int dims = shape_of(t, d);
  if (dims < 0) return -1;
  if (placed(t, dtype, index) != 1) return refuse_place(t, what, dtype, index);
  int ok = dims == 1 && (n < 0 || d[0] == n);
  if (ok) {
    PyObject* v = method(t, G.is_contiguous);
    if (!v) return -1;
    ok = v == Py_True;
    Py_DECREF(v);
  }
  if (!ok) {
    if (n < 0)
      PyErr_Format(PyExc_ValueError, "%s must be a contiguous vector", what);
    else
      PyErr_Format(PyExc_ValueError, "%s must be a contiguous vector of %lld", what, n);
    return -1;
  }
  void* q;
  if (pointer_of(t, &q)) return -1;
  *p = q;
  return d[0];
}

static PyObject* new_tensor(PyObject* shape, PyObject* dtype, PyObject* device) {
  if (!shape) return NULL;
  PyObject* args[3] = {shape, dtype, device};
  PyObject* t = PyObject_Vectorcall(G.empty, args, 1, G.empty_names);
  Py_DECREF(shape);
  return t;
}

/* `given`, described in r, or where it is None a new tensor [tokens, heads, dim] */
static PyObject* output(PyObject* given, long long tokens, long long heads, long long dim,
                        PyObject* dtype, PyObject* device, long index, moe_attn_rows* r,
                        const char* what) {
  if (given != Py_None) {
    const long long n = rows_of(given, heads, dim, dtype, index, r, what);
    if (n < 0) return NULL;
    if (n != tokens) {
      PyErr_Format(PyExc_ValueError, "%s must have %lld tokens", what, tokens);
      return NULL;
    }
    return Py_NewRef(given);
  }
  PyObject* t = new_tensor(Py_BuildValue("(LLL)", tokens, heads, dim), dtype, device);
  if (!t) return NULL;
  r->head_stride = dim;
  r->token_stride = heads * dim;
  if (pointer_of(t, &r->data)) Py_CLEAR(t);
  return t;
}

static int stream_of(PyObject* given, long index, void** stream) {
  if (given != Py_None) {
    *stream = PyLong_AsVoidPtr(given);
    return PyErr_Occurred() ? -1 : 0;
  }
  PyObject* i = PyLong_FromLong(index);
  PyObject* v = i ? PyObject_CallOneArg(G.raw_stream, i) : NULL;
  Py_XDECREF(i);
  if (!v) return -1;
  *stream = PyLong_AsVoidPtr(v);
  Py_DECREF(v);
  return PyErr_Occurred() ? -1 : 0;
}

static int int32_of(PyObject* v, int32_t* out, const char* what) {
  const long x = PyLong_AsLong(v);
  if (x == -1 && PyErr_Occurred()) return -1;
  if (x < INT_MIN || x > INT_MAX) {
    PyErr_Format(PyExc_ValueError, "%s is out of range", what);
    return -1;
  }
  *out = (int32_t)x;
  return 0;
}

static int float_of(PyObject* v, float* out) {
  const double x = PyFloat_AsDouble(v);
  if (x == -1.0 && PyErr_Occurred()) return -1;
  *out = (float)x;
  return 0;
}

static int rotation_of(PyObject* freq, PyObject* layout, PyObject* magnitude, int inverse,
                       long index, moe_attn_rotation* r) {
  const void* p;
  const long long n = vector_of(freq, -1, G.i64, index, &p, "freq");
  if (n < 0) return -1;
  if (n > 65536) {
    PyErr_SetString(PyExc_ValueError, "freq is too long");
    return -1;
  }
  r->freq = p;
  r->rot_dim = (int32_t)(2 * n);
  r->inverse = inverse;
  return int32_of(layout, &r->layout, "layout") || float_of(magnitude, &r->magnitude) ? -1 : 0;
}

static int cache_of(const layer_t* l, PyObject* k, PyObject* v, moe_attn_cache* c) {
  long long d[MAX_DIMS], s[MAX_DIMS], d2[MAX_DIMS], s2[MAX_DIMS];
  const int n = shape_of(k, d), n2 = shape_of(v, d2);
  if (n < 0 || n2 < 0) return -1;
  if (n != 4 || d[1] != l->kv_heads || d[2] != l->page || d[3] != l->dim) {
    PyErr_Format(PyExc_ValueError, "k_pages must be [pages, %lld, %lld, %lld]", l->kv_heads,
                 l->page, l->dim);
    return -1;
  }
  if (strides_of(k, s) < 0 || strides_of(v, s2) < 0) return -1;
  int same = n2 == 4 && s[3] == 1;
  for (int i = 0; same && i < 4; ++i) same = d[i] == d2[i] && (s[i] == s2[i] || d[i] == 1);
  if (!same) {
    PyErr_SetString(PyExc_ValueError,
                    "k_pages and v_pages must have one shape and strides, head_dim contiguous");
    return -1;
  }
  if (placed(k, l->dtype, l->index) != 1) return refuse_place(k, "k_pages", l->dtype, l->index);
  if (placed(v, l->dtype, l->index) != 1) return refuse_place(v, "v_pages", l->dtype, l->index);
  c->num_pages = d[0];
  c->token_stride = s[2];
  /* the stride of a dimension of one element says nothing */
  c->head_stride = l->kv_heads > 1 ? s[1] : l->dim;
  c->page_stride = d[0] > 1 ? s[0] : l->page * l->kv_heads * l->dim;
  return pointer_of(k, &c->k) || pointer_of(v, &c->v) ? -1 : 0;
}

/* raises for a status other than 0 */
static int checked(int status, const char* what) {
  if (!status) return 0;
  PyObject* r = PyObject_CallFunction(G.check, "is", status, what);
  Py_XDECREF(r);
  if (r) PyErr_Format(PyExc_RuntimeError, "%s failed (%d)", what, status);
  return -1;
}

/* 1, 0, or -1 with an error */
static int asked(PyObject* what) {
  PyObject* v = PyObject_CallNoArgs(what);
  if (!v) return -1;
  Py_DECREF(v);
  return v == Py_True;
}

/* No gradient runs through these calls: refuses tensors that ask for one. */
static int no_gradient(PyObject* const* t, int n, const char* what) {
  const int on = asked(G.grad_enabled);
  for (int i = 0; i < n && on == 1; ++i) {
    if (t[i] == Py_None) continue;
    PyObject* v = PyObject_GetAttr(t[i], G.requires_grad);
    if (!v) return -1;
    Py_DECREF(v);
    if (v == Py_True) {
      PyErr_Format(PyExc_ValueError,
                   "%s has no autograd formula: call it under torch.no_grad(), or on detached "
                   "tensors (the gradient of rotary positions is moe_attn_rope with inverse=True)",
                   what);
      return -1;
    }
  }
  return on < 0 ? -1 : 0;
}

/* Tells autograd which of the outputs that the caller gave were written to, so that
 * a backward pass that kept one raises. Inference tensors keep no count. (Not the
 * cache's pages: 1.2 us more for each append, for tensors that are only ever read by
 * the calls here.) */
static int wrote(PyObject* const* t, int n) {
  PyObject* list = NULL;
  for (int i = 0; i < n; ++i) {
    if (t[i] == Py_None) continue;
    if (!list) {
      const int inference = asked(G.inference_enabled);
      if (inference) return inference < 0 ? -1 : 0;
      if (!(list = PyList_New(0))) return -1;
    }
    if (PyList_Append(list, t[i])) {
      Py_DECREF(list);
      return -1;
    }
  }
  if (!list) return 0;
  PyObject* r = PyObject_CallOneArg(G.increment_version, list);
  Py_DECREF(list);
  if (!r) {
    if (!PyErr_ExceptionMatches(PyExc_RuntimeError)) return -1;
    PyErr_Clear(); /* an inference tensor outside of inference mode */
  }
  Py_XDECREF(r);
  return 0;
}

static int arity(Py_ssize_t n, Py_ssize_t want, const char* what) {
  if (n == want) return 0;
  PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, got %zd", what, want, n);
  return -1;
}

/* rope(x, positions, freq, out, layout, magnitude, inverse, stream): out, or
 * NotImplemented where another device than x's is current */
static PyObject* rope(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (arity(n, 8, "rope")) return NULL;
  PyObject *x = a[0], *dtype = PyObject_GetAttr(x, G.dtype);
  if (!dtype) return NULL;
  Py_DECREF(dtype); /* torch keeps its types for good */
  const int32_t code = dtype == G.bf16 ? MOE_ATTN_BF16 : dtype == G.fp16 ? MOE_ATTN_FP16 : -1;
  long long d[MAX_DIMS];
  const int dims = shape_of(x, d);
  if (dims < 0) return NULL;
  PyObject* on = method(x, G.get_device);
  if (!on) return NULL;
  const long index = PyLong_AsLong(on);
  Py_DECREF(on);
  if (PyErr_Occurred()) return NULL;
  if (code < 0 || dims != 3 || index < 0) {
    PyErr_SetString(PyExc_ValueError,
                    "x must be a bf16 or fp16 CUDA tensor [tokens, heads, head_dim]");
    return NULL;
  }
  PyObject* current = PyObject_CallNoArgs(G.current_device);
  if (!current) return NULL;
  const long now = PyLong_AsLong(current);
  Py_DECREF(current);
  if (now != index) return PyErr_Occurred() ? NULL : Py_NewRef(Py_NotImplemented);
  if (d[1] > INT_MAX || d[2] > INT_MAX) {
    PyErr_SetString(PyExc_ValueError, "x is too large");
    return NULL;
  }
  moe_attn_rows xr, outr;
  moe_attn_rotation r;
  const void* pos;
  void* stream;
  const long long tokens = rows_of(x, d[1], d[2], dtype, index, &xr, "x");
  const int inverse = PyObject_IsTrue(a[6]);
  if (tokens < 0 || inverse < 0 || rotation_of(a[2], a[4], a[5], inverse, index, &r) ||
      vector_of(a[1], tokens, G.i32, index, &pos, "positions") < 0 ||
      stream_of(a[7], index, &stream))
    return NULL;
  PyObject* const tracked[2] = {x, a[3]};
  if (no_gradient(tracked, 2, "moe_attn_rope")) return NULL;
  PyObject* device = PyObject_GetAttr(x, G.device);
  if (!device) return NULL;
  PyObject* out = output(a[3], tokens, d[1], d[2], dtype, device, index, &outr, "out");
  Py_DECREF(device);
  if (!out) return NULL;
  int st;
  Py_BEGIN_ALLOW_THREADS;
  st = G.rope(&xr, &outr, pos, (int32_t)tokens, (int32_t)d[1], (int32_t)d[2], code, &r, stream);
  Py_END_ALLOW_THREADS;
  if (checked(st, "moe_attn_rope") || wrote(a + 3, 1)) Py_CLEAR(out);
  return out;
}

static void layer_free(PyObject* capsule) {
  layer_t* l = PyCapsule_GetPointer(capsule, "moe_attn_layer");
  Py_XDECREF(l->dtype);
  Py_XDECREF(l->device);
  PyMem_Free(l);
}

/* layer(handle, q_heads, kv_heads, head_dim, page_size, index, dtype, device) */
static PyObject* layer(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (arity(n, 8, "layer")) return NULL;
  layer_t* l = PyMem_Calloc(1, sizeof(*l));
  if (!l) return PyErr_NoMemory();
  l->handle = PyLong_AsVoidPtr(a[0]);
  l->q_heads = PyLong_AsLongLong(a[1]);
  l->kv_heads = PyLong_AsLongLong(a[2]);
  l->dim = PyLong_AsLongLong(a[3]);
  l->page = PyLong_AsLongLong(a[4]);
  l->index = PyLong_AsLong(a[5]);
  l->dtype = Py_NewRef(a[6]);
  l->device = Py_NewRef(a[7]);
  PyObject* c = PyErr_Occurred() ? NULL : PyCapsule_New(l, "moe_attn_layer", layer_free);
  if (!c) {
    Py_DECREF(l->dtype);
    Py_DECREF(l->device);
    PyMem_Free(l);
  }
  return c;
}

/* append(layer, q, k, v, positions, slots, k_pages, v_pages, freq, layout,
 * magnitude, q_out, stream): q_out, or None without q */
static PyObject* append(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (arity(n, 13, "append")) return NULL;
  const layer_t* l = PyCapsule_GetPointer(a[0], "moe_attn_layer");
  if (!l) return NULL;
  moe_attn_rows q, qo, k, v;
  moe_attn_rotation r;
  moe_attn_cache c;
  const void *pos, *slots;
  void* stream;
  const long long T = rows_of(a[2], l->kv_heads, l->dim, l->dtype, l->index, &k, "k");
  if (T < 0) return NULL;
  const long long Tv = rows_of(a[3], l->kv_heads, l->dim, l->dtype, l->index, &v, "v");
  if (Tv < 0) return NULL;
  const int with_q = a[1] != Py_None;
  long long Tq = T;
  if (with_q && (Tq = rows_of(a[1], l->q_heads, l->dim, l->dtype, l->index, &q, "q")) < 0)
    return NULL;
  if (Tv != T || Tq != T || (!with_q && a[11] != Py_None)) {
    PyErr_SetString(PyExc_ValueError, Tv != T || Tq != T ? "q, k and v differ in tokens"
                                                         : "q_out without q");
    return NULL;
  }
  if (rotation_of(a[8], a[9], a[10], 0, l->index, &r) ||
      vector_of(a[4], T, G.i32, l->index, &pos, "positions") < 0 ||
      vector_of(a[5], T, G.i64, l->index, &slots, "slots") < 0 || cache_of(l, a[6], a[7], &c) ||
      stream_of(a[12], l->index, &stream))
    return NULL;
  PyObject* const tracked[6] = {a[1], a[2], a[3], a[6], a[7], a[11]};
  if (no_gradient(tracked, 6, "PagedAttention.append")) return NULL;
  PyObject* out = with_q ? output(a[11], T, l->q_heads, l->dim, l->dtype, l->device, l->index, &qo,
                                  "q_out")
                         : Py_NewRef(Py_None);
  if (!out) return NULL;
  int st;
  Py_BEGIN_ALLOW_THREADS;
  st = G.append(l->handle, with_q ? &q : NULL, with_q ? &qo : NULL, &k, &v, pos, slots, (int32_t)T,
                &r, &c, stream);
  Py_END_ALLOW_THREADS;
  if (checked(st, "moe_attn_append") || wrote(a + 11, 1)) Py_CLEAR(out);
  return out;
}

/* forward(layer, q, k_pages, v_pages, page_table, cu_q, kv_len, max_q, scale,
 * softcap, window, slopes, prefix, out, lse, return_lse, stream): out, or (out, lse) */
static PyObject* forward(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (arity(n, 17, "forward")) return NULL;
  const layer_t* l = PyCapsule_GetPointer(a[0], "moe_attn_layer");
  if (!l) return NULL;
  moe_attn_rows q, o;
  moe_attn_cache c;
  moe_attn_batch b;
  moe_attn_scores s = {0};
  long long d[MAX_DIMS], st[MAX_DIMS];
  const void* p;
  void *stream, *lse_at = NULL, *table;
  const long long T = rows_of(a[1], l->q_heads, l->dim, l->dtype, l->index, &q, "q");
  if (T < 0) return NULL;
  const long long seqs = vector_of(a[6], -1, G.i32, l->index, &p, "kv_len");
  if (seqs < 0) return NULL;
  if (seqs >= INT_MAX) {
    PyErr_SetString(PyExc_ValueError, "too many sequences");
    return NULL;
  }
  b.kv_len = p;
  if (vector_of(a[5], seqs + 1, G.i32, l->index, &p, "cu_q") < 0) return NULL;
  b.cu_q = p;
  const int dims = shape_of(a[4], d);
  if (dims < 0 || strides_of(a[4], st) < 0) return NULL;
  if (placed(a[4], G.i32, l->index) != 1) {
    refuse_place(a[4], "page_table", G.i32, l->index);
    return NULL;
  }
  if (dims != 2 || d[0] != seqs || (st[1] != 1 && d[1] > 1) || d[1] > INT_MAX) {
    PyErr_Format(PyExc_ValueError,
                 "page_table must be [%lld, columns], contiguous along the columns", seqs);
    return NULL;
  }
  if (pointer_of(a[4], &table)) return NULL;
  b.page_table = table;
  b.columns = (int32_t)d[1];
  b.table_stride = seqs > 1 ? st[0] : d[1];
  b.num_seqs = (int32_t)seqs;
  b.num_tokens = (int32_t)T;
  if (int32_of(a[7], &b.max_q, "max_q") || cache_of(l, a[2], a[3], &c)) return NULL;
  if (a[8] == Py_None)
    s.scale = (float)(1.0 / sqrt((double)l->dim));
  else if (float_of(a[8], &s.scale))
    return NULL;
  if (float_of(a[9], &s.softcap) || int32_of(a[10], &s.window, "window")) return NULL;
  if (a[11] != Py_None) {
    if (vector_of(a[11], l->q_heads, G.f32, l->index, &p, "slopes") < 0) return NULL;
    s.slopes = p;
  }
  if (a[12] != Py_None) {
    if (vector_of(a[12], seqs, G.i32, l->index, &p, "prefix") < 0) return NULL;
    s.prefix = p;
  }
  const int with_lse = PyObject_IsTrue(a[15]);
  if (with_lse < 0 || stream_of(a[16], l->index, &stream)) return NULL;
  PyObject* const tracked[6] = {a[1], a[2], a[3], a[11], a[13], a[14]};
  if (no_gradient(tracked, 6, "PagedAttention.forward")) return NULL;
  PyObject* lse;
  if (a[14] != Py_None) {
    const int ld = shape_of(a[14], d);
    if (ld < 0) return NULL;
    if (placed(a[14], G.f32, l->index) != 1) {
      refuse_place(a[14], "lse", G.f32, l->index);
      return NULL;
    }
    PyObject* dense = method(a[14], G.is_contiguous);
    if (!dense) return NULL;
    const int ok = ld == 2 && d[0] == T && d[1] == l->q_heads && dense == Py_True;
    Py_DECREF(dense);
    if (!ok) {
      PyErr_Format(PyExc_ValueError, "lse must be contiguous [%lld, %lld]", T, l->q_heads);
      return NULL;
    }
    lse = Py_NewRef(a[14]);
  } else if (with_lse) {
    lse = new_tensor(Py_BuildValue("(LL)", T, l->q_heads), G.f32, l->device);
  } else {
    lse = Py_NewRef(Py_None);
  }
  if (!lse || (lse != Py_None && pointer_of(lse, &lse_at))) {
    Py_XDECREF(lse);
    return NULL;
  }
  PyObject* out = output(a[13], T, l->q_heads, l->dim, l->dtype, l->device, l->index, &o, "out");
  if (!out) {
    Py_DECREF(lse);
    return NULL;
  }
  int status;
  Py_BEGIN_ALLOW_THREADS;
  status = G.forward(l->handle, &q, &o, lse_at, &c, &b, &s, stream);
  Py_END_ALLOW_THREADS;
  PyObject* result = NULL;
  if (!checked(status, "moe_attn_forward") && !wrote(tracked + 4, 2))
    result = with_lse ? PyTuple_Pack(2, out, lse) : Py_NewRef(out);
  Py_DECREF(out);
  Py_DECREF(lse);
  return result;
}

/* setup(rope, append, forward, check, empty, raw_stream, current_device,
 * grad_enabled, inference_enabled, increment_version, bf16, fp16, f32, i32, i64): addresses of the library's functions, what raises for a
 * status, and of torch what is needed here. Once, before any other call. */
static PyObject* setup(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (arity(n, 15, "setup")) return NULL;
  G.rope = (rope_fn)PyLong_AsVoidPtr(a[0]);
  G.append = (append_fn)PyLong_AsVoidPtr(a[1]);
  G.forward = (forward_fn)PyLong_AsVoidPtr(a[2]);
  if (PyErr_Occurred()) return NULL;
  PyObject** to[] = {&G.check,        &G.empty,             &G.raw_stream,
                     &G.current_device, &G.grad_enabled,    &G.inference_enabled,
                     &G.increment_version, &G.bf16,         &G.fp16,
                     &G.f32,          &G.i32,               &G.i64};
  for (int i = 0; i < 12; ++i) Py_XSETREF(*to[i], Py_NewRef(a[3 + i]));
  Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"setup", (PyCFunction)(void (*)(void))setup, METH_FASTCALL, NULL},
    {"layer", (PyCFunction)(void (*)(void))layer, METH_FASTCALL, NULL},
    {"rope", (PyCFunction)(void (*)(void))rope, METH_FASTCALL, NULL},
    {"append", (PyCFunction)(void (*)(void))append, METH_FASTCALL, NULL},
    {"forward", (PyCFunction)(void (*)(void))forward, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_attn_binding", NULL, -1, methods,
                                    NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__attn_binding(void) {
  G.shape = PyUnicode_InternFromString("shape");
  G.stride = PyUnicode_InternFromString("stride");
  G.dtype = PyUnicode_InternFromString("dtype");
  G.device = PyUnicode_InternFromString("device");
  G.get_device = PyUnicode_InternFromString("get_device");
  G.data_ptr = PyUnicode_InternFromString("data_ptr");
  G.is_contiguous = PyUnicode_InternFromString("is_contiguous");
  G.requires_grad = PyUnicode_InternFromString("requires_grad");
  G.empty_names = Py_BuildValue("(ss)", "dtype", "device");
  if (!G.shape || !G.stride || !G.dtype || !G.device || !G.get_device || !G.data_ptr ||
      !G.is_contiguous || !G.requires_grad || !G.empty_names)
    return NULL;
  return PyModule_Create(&module);
}
