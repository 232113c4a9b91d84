/*
 * py_binding.c -- argument checks and calls of the small per-step operators for Python.
 *
 * A decode step's store, norm or read-back takes the GPU 2-4 us, and a ctypes call with a dozen tensors
 * took the host 7-15 us (about 0.35 us of checks per tensor and 3.6 us to convert 25 arguments), so the host
 * set their rate.  These functions make the same checks through the CPython API and call the library's
 * entry points by address: 2-3x less.  Types raise TypeError, everything else ValueError; the return value is
 * the library's status, or -1 if the tensors' device is not the current one (the caller switches and retries).
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>
#include <stdlib.h>

#include "../../include/ra.h"

static PyObject *s_dtype, *s_device, *s_shape, *s_stride, *s_is_contiguous, *s_data_ptr, *s_type, *s_index,
    *s_cuda_stream;
static PyObject *t_bf16, *t_i32, *t_f32, *t_u8;         /* torch dtypes */
static PyObject *f_raw_stream, *f_current_device;       /* current raw stream of a device; current device */

static ra_status (*p_kv8_store)(void*, int64_t, int32_t, int32_t, const void*, const void*, const int32_t*, int64_t,
                                uint32_t*, ra_stream_t);
static ra_status (*p_kv8_load)(const void*, int64_t, int32_t, int32_t, const int32_t*, void*, void*, int64_t,
                               uint32_t*, ra_stream_t);
static size_t (*p_kv8_slot_bytes)(int32_t, int32_t);
static ra_status (*p_kv8_decode)(const void*, int64_t, int32_t, int32_t, const void*, void*, int32_t, float,
                                 const int32_t*, int64_t, int64_t, const int32_t*, const int32_t*, int32_t, int32_t,
                                 void*, size_t, uint32_t*, ra_stream_t);
static ra_status (*p_norm_rope)(const void*, int64_t, const void*, int64_t, const void*, int64_t, int32_t, int32_t,
                                int32_t, const void*, const void*, float, const int32_t*, const float*, int64_t,
                                int32_t, int32_t, void*, int64_t, void*, void*, int64_t, const int32_t*, int64_t,
                                uint32_t*, ra_stream_t);
static ra_status (*p_norm_rope_kv8)(const void*, int64_t, const void*, int64_t, const void*, int64_t, int32_t, int32_t,
                                    int32_t, const void*, const void*, float, const int32_t*, const float*, int64_t,
                                    int32_t, int32_t, void*, int64_t, void*, int64_t, const int32_t*, int64_t,
                                    uint32_t*, ra_stream_t);
static ra_status (*p_tree)(const void*, const void*, int64_t, int32_t, int32_t, const void*, void*, int32_t, float,
                           const int32_t*, int64_t, int64_t, const int32_t*, const int32_t*, const int32_t*,
                           const int32_t*, const uint32_t*, int32_t, int32_t, int64_t, int32_t, int32_t, void*, size_t,
                           uint32_t*, ra_stream_t);

/* init(dtypes (bf16, i32, f32, u8), raw_stream, current_device, addresses in the order above) */
static PyObject* init(PyObject* self, PyObject* args) {
  unsigned long long a[7];
  PyObject *bf, *i, *f, *u, *rs, *cd;
  (void)self;
  if (!PyArg_ParseTuple(args, "OOOOOOKKKKKKK", &bf, &i, &f, &u, &rs, &cd, a, a + 1, a + 2, a + 3, a + 4, a + 5, a + 6))
    return NULL;
  t_bf16 = Py_NewRef(bf), t_i32 = Py_NewRef(i), t_f32 = Py_NewRef(f), t_u8 = Py_NewRef(u);
  f_raw_stream = Py_NewRef(rs), f_current_device = Py_NewRef(cd);
  *(void**)&p_kv8_store = (void*)(uintptr_t)a[0];
  *(void**)&p_kv8_load = (void*)(uintptr_t)a[1];
  *(void**)&p_kv8_slot_bytes = (void*)(uintptr_t)a[2];
  *(void**)&p_kv8_decode = (void*)(uintptr_t)a[3];
  *(void**)&p_norm_rope = (void*)(uintptr_t)a[4];
  *(void**)&p_norm_rope_kv8 = (void*)(uintptr_t)a[5];
  *(void**)&p_tree = (void*)(uintptr_t)a[6];
  Py_RETURN_NONE;
}

/* dims sizes of a tensor; -1 with an exception if it has another number of dimensions */
static int sizes(PyObject* t, const char* name, int dims, int64_t* out) {
  PyObject* shape = PyObject_GetAttr(t, s_shape);
  if (!shape) return -1;
  if (!PyTuple_Check(shape) || PyTuple_GET_SIZE(shape) != dims) {
    PyErr_Format(PyExc_ValueError, "%s: expected %d dimensions, got shape %R", name, dims, shape);
    Py_DECREF(shape);
    return -1;
  }
  for (int i = 0; i < dims; ++i) out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, i));
  Py_DECREF(shape);
  return PyErr_Occurred() ? -1 : 0;
}

static int wrong_shape(const char* name, const char* expected) {
  PyErr_Format(PyExc_ValueError, "%s: expected shape %s", name, expected);
  return -1;
}

/* dtype and device; -1 with an exception */
static int typed(PyObject* t, PyObject* dtype, PyObject* device, const char* name) {
  PyObject* x = PyObject_GetAttr(t, s_dtype);
  if (!x) return -1;
  if (x != dtype) {
    PyErr_Format(PyExc_TypeError, "%s: expected %R, got %R", name, dtype, x);
    Py_DECREF(x);
    return -1;
  }
  Py_DECREF(x);
  x = PyObject_GetAttr(t, s_device);
  if (!x) return -1;
  const int same = x == device ? 1 : PyObject_RichCompareBool(x, device, Py_EQ);
  if (same == 0) PyErr_Format(PyExc_ValueError, "%s: expected device %S, got %S", name, device, x);
  Py_DECREF(x);
  return same == 1 ? 0 : -1;
}

static int address(PyObject* t, void** out) {
  PyObject* x = PyObject_CallMethodNoArgs(t, s_data_ptr);
  if (!x) return -1;
  *out = PyLong_AsVoidPtr(x);
  Py_DECREF(x);
  return PyErr_Occurred() ? -1 : 0;
}

/* address of a contiguous tensor of this dtype on this device; None gives NULL where `optional` */
static int tensor(PyObject* t, PyObject* dtype, PyObject* device, const char* name, int optional, void** out) {
  *out = NULL;
  if (optional && t == Py_None) return 0;
  if (typed(t, dtype, device, name)) return -1;
  PyObject* x = PyObject_CallMethodNoArgs(t, s_is_contiguous);
  if (!x) return -1;
  const int contiguous = x == Py_True;
  Py_DECREF(x);
  if (!contiguous) {
    PyErr_Format(PyExc_ValueError, "%s: must be contiguous", name);
    return -1;
  }
  return address(t, out);
}

/* bf16 head rows [n, h, d]: a token's rows contiguous, tokens at any stride */
static int head_rows(PyObject* t, PyObject* device, const char* name, const int64_t* want, void** out, int64_t* stride) {
  int64_t s[3];
  if (typed(t, t_bf16, device, name) || sizes(t, name, 3, s)) return -1;
  if (s[0] != want[0] || s[1] != want[1] || s[2] != want[2]) return wrong_shape(name, "[num_tokens, H, D] like its peers");
  PyObject* st = PyObject_CallMethodNoArgs(t, s_stride);
  if (!st) return -1;
  int64_t v[3] = {0, 0, 0};
  for (int i = 0; i < 3 && PyTuple_Check(st) && PyTuple_GET_SIZE(st) == 3; ++i)
    v[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(st, i));
  Py_DECREF(st);
  if (PyErr_Occurred()) return -1;
  if ((v[2] != 1 && s[2] > 1) || (v[1] != s[2] && s[1] > 1)) {
    PyErr_Format(PyExc_ValueError, "%s: a token's head rows must be contiguous", name);
    return -1;
  }
  *stride = s[0] > 1 ? v[0] : s[1] * s[2];
  return address(t, out);
}

/* 0: the call may go ahead on *out; 1: another device is current; -1: exception */
static int stream_of(PyObject* device, PyObject* stream, ra_stream_t* out) {
  PyObject* type = PyObject_GetAttr(device, s_type);
  if (!type) return -1;
  const int cuda = PyUnicode_Check(type) && PyUnicode_CompareWithASCIIString(type, "cuda") == 0;
  Py_DECREF(type);
  if (!cuda) {
    PyErr_Format(PyExc_ValueError, "expected CUDA tensors, got %S", device);
    return -1;
  }
  PyObject* index = PyObject_GetAttr(device, s_index);
  if (!index) return -1;
  PyObject* current = PyObject_CallNoArgs(f_current_device);
  if (!current) {
    Py_DECREF(index);
    return -1;
  }
  const long long i = PyLong_AsLongLong(index), c = PyLong_AsLongLong(current);
  Py_DECREF(current);
  if (PyErr_Occurred() || i != c) {
    Py_DECREF(index);
    return PyErr_Occurred() ? -1 : 1;
  }
  PyObject* s = stream == Py_None ? PyObject_CallOneArg(f_raw_stream, index) : PyObject_GetAttr(stream, s_cuda_stream);
  Py_DECREF(index);
  if (!s) return -1;
  *out = (ra_stream_t)PyLong_AsVoidPtr(s);
  Py_DECREF(s);
  return PyErr_Occurred() ? -1 : 0;
}

/* pool of records: its address and slots */
static int kv8_pool(PyObject* t, PyObject* device, int64_t hkv, int64_t d, void** out, int64_t* slots) {
  int64_t s[2];
  if (sizes(t, "kv8_pool", 2, s)) return -1;
  const size_t want = hkv > 0 && hkv <= INT32_MAX && d <= INT32_MAX ? p_kv8_slot_bytes((int32_t)hkv, (int32_t)d) : 0;
  if (want == 0 || s[1] != (int64_t)want) {
    PyErr_Format(PyExc_ValueError, "kv8_pool: expected [num_slots, %zu] for %lld kv heads of %lld, got [%lld, %lld]", want,
                 (long long)hkv, (long long)d, (long long)s[0], (long long)s[1]);
    return -1;
  }
  *slots = s[0];
  return tensor(t, t_u8, device, "kv8_pool", 0, out);
}

static int arity(const char* name, Py_ssize_t got, Py_ssize_t want) {
  if (got == want) return 0;
  PyErr_Format(PyExc_TypeError, "%s: expected %zd arguments, got %zd", name, want, got);
  return -1;
}

#define FAIL_IF(x) \
  do {             \
    if (x) {       \
      Py_DECREF(device); \
      return NULL; \
    }              \
  } while (0)

/* the call itself, without the interpreter lock: a launch may wait for room in the stream's queue */
#define CALL(expr)               \
  do {                           \
    ra_status status;            \
    Py_BEGIN_ALLOW_THREADS;      \
    status = (expr);             \
    Py_END_ALLOW_THREADS;        \
    return PyLong_FromLong(status); \
  } while (0)

/* Python int -> int32 range-checked */
static int as_i32(PyObject* o, int32_t* out) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) return -1;
  if (v < INT32_MIN || v > INT32_MAX) {
    PyErr_Format(PyExc_ValueError, "%lld does not fit in 32 bits", v);
    return -1;
  }
  *out = (int32_t)v;
  return 0;
}

static int workspace_of(PyObject* t, PyObject* device, void** out, size_t* bytes) {
  int64_t s[1];
  if (sizes(t, "workspace", 1, s) || tensor(t, t_u8, device, "workspace", 0, out)) return -1;
  *bytes = (size_t)s[0];
  return 0;
}

/* (pool, k, v, loc, err, stream), store; (pool, slots, k, v, err, stream), load */
static PyObject* kv8_move(PyObject* const* a, Py_ssize_t n, int load) {
  if (arity(load ? "kv8_load" : "kv8_store", n, 6)) return NULL;
  PyObject *ko = a[load ? 2 : 1], *vo = a[load ? 3 : 2], *so = a[load ? 1 : 3];
  PyObject* device = PyObject_GetAttr(a[0], s_device);
  if (!device) return NULL;
  int64_t ks[3], vs[3], ls[1], slots;
  void *pool, *k, *v, *loc, *err;
  ra_stream_t stream;
  FAIL_IF(sizes(ko, "K rows", 3, ks) || sizes(vo, "V rows", 3, vs) || sizes(so, "slots", 1, ls));
  FAIL_IF((ks[0] != vs[0] || ks[1] != vs[1] || ks[2] != vs[2] || ls[0] != ks[0]) &&
          wrong_shape("K and V rows", "[num_tokens, Hkv, D], slots [num_tokens]"));
  FAIL_IF(kv8_pool(a[0], device, ks[1], ks[2], &pool, &slots) || tensor(ko, t_bf16, device, "K rows", 0, &k) ||
          tensor(vo, t_bf16, device, "V rows", 0, &v) || tensor(so, t_i32, device, "slots", 0, &loc) ||
          tensor(a[4], t_i32, device, "device_error", 1, &err));
  const int ready = stream_of(device, a[5], &stream);
  FAIL_IF(ready < 0);
  Py_DECREF(device);
  if (ready) return PyLong_FromLong(-1);
  CALL(load ? p_kv8_load(pool, slots, (int32_t)ks[1], (int32_t)ks[2], loc, k, v, ks[0], err, stream)
            : p_kv8_store(pool, slots, (int32_t)ks[1], (int32_t)ks[2], k, v, loc, ks[0], err, stream));
}

static PyObject* kv8_store(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  return kv8_move(a, n, 0);
}
static PyObject* kv8_load(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  return kv8_move(a, n, 1);
}

/* (pool, q, o, table, rpi, lens, num_kv_heads, max_seq_len, sm_scale, workspace, err, stream) */
static PyObject* kv8_decode(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (arity("kv8_decode_attention", n, 12)) return NULL;
  PyObject* device = PyObject_GetAttr(a[0], s_device);
  if (!device) return NULL;
  int64_t qs[3], os[3], ts[2], rs[1], ls[1], slots;
  int32_t hkv, max_len;
  void *pool, *q, *o, *table, *rpi, *lens, *ws, *err;
  size_t ws_bytes;
  ra_stream_t stream;
  FAIL_IF(sizes(a[1], "q", 3, qs) || sizes(a[2], "o", 3, os) || sizes(a[3], "req_to_token", 2, ts) ||
          sizes(a[4], "req_pool_indices", 1, rs) || sizes(a[5], "seq_lens", 1, ls));
  FAIL_IF((qs[0] != os[0] || qs[1] != os[1] || qs[2] != os[2]) && wrong_shape("o", "that of q"));
  FAIL_IF((rs[0] != qs[0] || ls[0] != qs[0]) && wrong_shape("req_pool_indices and seq_lens", "[batch]"));
  FAIL_IF(as_i32(a[6], &hkv) || as_i32(a[7], &max_len));
  const double scale = PyFloat_AsDouble(a[8]);
  FAIL_IF(scale == -1.0 && PyErr_Occurred());
  FAIL_IF(kv8_pool(a[0], device, hkv, qs[2], &pool, &slots) || tensor(a[1], t_bf16, device, "q", 0, &q) ||
          tensor(a[2], t_bf16, device, "o", 0, &o) || tensor(a[3], t_i32, device, "req_to_token", 0, &table) ||
          tensor(a[4], t_i32, device, "req_pool_indices", 0, &rpi) || tensor(a[5], t_i32, device, "seq_lens", 0, &lens) ||
          workspace_of(a[9], device, &ws, &ws_bytes) || tensor(a[10], t_i32, device, "device_error", 1, &err));
  FAIL_IF((qs[0] > INT32_MAX || qs[1] > INT32_MAX) && wrong_shape("q", "within 32 bits"));
  const int ready = stream_of(device, a[11], &stream);
  FAIL_IF(ready < 0);
  Py_DECREF(device);
  if (ready) return PyLong_FromLong(-1);
  CALL(p_kv8_decode(pool, slots, hkv, (int32_t)qs[2], q, o, (int32_t)qs[1], (float)scale, table, ts[1], ts[0],
                    rpi, lens, (int32_t)qs[0], max_len, ws, ws_bytes, err, stream));
}

/* (q, k, v, q_weight, k_weight, positions, cos_sin, q_out, pools..., loc, eps, interleaved, err, stream) */
static PyObject* norm_rope_call(PyObject* const* a, Py_ssize_t n, int kv8) {
  if (arity("qk_norm_rope_store", n, kv8 ? 14 : 15)) return NULL;
  PyObject* const* b = a + (kv8 ? 9 : 10); /* loc, eps, interleaved, err, stream */
  PyObject* device = PyObject_GetAttr(a[8], s_device);
  if (!device) return NULL;
  int64_t qs[3], ks[3], ps[1], cs[2], ls[1], w[1], slots, stride[4];
  void *q, *k, *v, *qw, *kw, *pos, *cos_sin, *qo, *pool, *v_pool = NULL, *loc, *err;
  ra_stream_t stream;
  FAIL_IF(sizes(a[0], "q", 3, qs) || sizes(a[1], "k", 3, ks) || sizes(a[5], "positions", 1, ps) ||
          sizes(a[6], "cos_sin", 2, cs) || sizes(b[0], "out_cache_loc", 1, ls));
  FAIL_IF((ks[0] != qs[0] || ks[2] != qs[2]) && wrong_shape("k and v", "[num_tokens, Hkv, D]"));
  FAIL_IF((ps[0] != qs[0] || ls[0] != qs[0]) && wrong_shape("positions and out_cache_loc", "[num_tokens]"));
  for (int i = 3; i < 5; ++i)
    if (a[i] != Py_None) FAIL_IF(sizes(a[i], "weights", 1, w) || (w[0] != qs[2] && wrong_shape("weights", "[D]")));
  FAIL_IF(head_rows(a[0], device, "q", qs, &q, stride) || head_rows(a[1], device, "k", ks, &k, stride + 1) ||
          head_rows(a[2], device, "v", ks, &v, stride + 2) || head_rows(a[7], device, "q_out", qs, &qo, stride + 3) ||
          tensor(a[3], t_bf16, device, "q_weight", 1, &qw) || tensor(a[4], t_bf16, device, "k_weight", 1, &kw) ||
          tensor(a[5], t_i32, device, "positions", 0, &pos) || tensor(a[6], t_f32, device, "cos_sin", 0, &cos_sin) ||
          tensor(b[0], t_i32, device, "out_cache_loc", 0, &loc) || tensor(b[3], t_i32, device, "device_error", 1, &err));
  if (kv8) {
    FAIL_IF(kv8_pool(a[8], device, ks[1], ks[2], &pool, &slots));
  } else {
    int64_t s[3], t[3];
    FAIL_IF(sizes(a[8], "k_pool", 3, s) || sizes(a[9], "v_pool", 3, t));
    FAIL_IF((s[1] != ks[1] || s[2] != ks[2] || t[0] != s[0] || t[1] != s[1] || t[2] != s[2]) &&
            wrong_shape("pools", "[num_slots, Hkv, D]"));
    FAIL_IF(tensor(a[8], t_bf16, device, "k_pool", 0, &pool) || tensor(a[9], t_bf16, device, "v_pool", 0, &v_pool));
    slots = s[0];
  }
  FAIL_IF((qs[1] > INT32_MAX || ks[1] > INT32_MAX || qs[2] > INT32_MAX || cs[1] > INT32_MAX) &&
          wrong_shape("q, k, v and cos_sin", "within 32 bits"));
  const double eps = PyFloat_AsDouble(b[1]);
  FAIL_IF(eps == -1.0 && PyErr_Occurred());
  const int inter = PyObject_IsTrue(b[2]);
  FAIL_IF(inter < 0);
  const int ready = stream_of(device, b[4], &stream);
  FAIL_IF(ready < 0);
  Py_DECREF(device);
  if (ready) return PyLong_FromLong(-1);
  CALL(kv8 ? p_norm_rope_kv8(q, stride[0], k, stride[1], v, stride[2], (int32_t)qs[1], (int32_t)ks[1], (int32_t)qs[2], qw,
                            kw, (float)eps, pos, cos_sin, cs[0], (int32_t)cs[1], inter, qo, stride[3], pool, slots, loc,
                            qs[0], err, stream)
          : p_norm_rope(q, stride[0], k, stride[1], v, stride[2], (int32_t)qs[1], (int32_t)ks[1], (int32_t)qs[2], qw, kw,
                        (float)eps, pos, cos_sin, cs[0], (int32_t)cs[1], inter, qo, stride[3], pool, v_pool, slots, loc,
                        qs[0], err, stream));
}

static PyObject* norm_rope_store(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  return norm_rope_call(a, n, 0);
}
static PyObject* norm_rope_kv8_store(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  return norm_rope_call(a, n, 1);
}

/* (k_pool, v_pool, q, o, table, rpi, prefix_lens, draft_lens, qo_indptr, tree_mask, max_draft_len, max_prefix_len,
 *  sm_scale, workspace, err, stream) */
static PyObject* tree(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (arity("tree_attention", n, 16)) return NULL;
  PyObject* device = PyObject_GetAttr(a[0], s_device);
  if (!device) return NULL;
  int64_t s[3], t[3], qs[3], os[3], ts[2], rs[1], ps[1], ds[1], is[1], ms[2];
  int32_t max_draft, max_prefix;
  void *k, *v, *q, *o, *table, *rpi, *pl, *dl, *qo, *mask, *ws, *err;
  size_t ws_bytes;
  ra_stream_t stream;
  FAIL_IF(sizes(a[0], "k_pool", 3, s) || sizes(a[1], "v_pool", 3, t) || sizes(a[2], "q", 3, qs) ||
          sizes(a[3], "o", 3, os) || sizes(a[4], "req_to_token", 2, ts) || sizes(a[5], "req_pool_indices", 1, rs) ||
          sizes(a[6], "prefix_lens", 1, ps) || sizes(a[7], "draft_lens", 1, ds) || sizes(a[8], "qo_indptr", 1, is) ||
          sizes(a[9], "tree_mask", 2, ms));
  FAIL_IF((s[0] != t[0] || s[1] != t[1] || s[2] != t[2]) && wrong_shape("v_pool", "that of k_pool"));
  FAIL_IF((qs[2] != s[2] || qs[0] != os[0] || qs[1] != os[1] || qs[2] != os[2]) &&
          wrong_shape("q and o", "[total_q, Hq, D]"));
  FAIL_IF((ps[0] != rs[0] || ds[0] != rs[0] || is[0] != rs[0] + 1) &&
          wrong_shape("prefix_lens, draft_lens and qo_indptr", "[batch], [batch] and [batch + 1]"));
  FAIL_IF(ms[0] != qs[0] && wrong_shape("tree_mask", "[total_q, words]"));
  FAIL_IF((rs[0] > INT32_MAX || qs[1] > INT32_MAX || s[1] > INT32_MAX || s[2] > INT32_MAX || ms[1] > INT32_MAX) &&
          wrong_shape("q, the pools, the mask and the batch", "within 32 bits"));
  FAIL_IF(as_i32(a[10], &max_draft) || as_i32(a[11], &max_prefix));
  const double scale = PyFloat_AsDouble(a[12]);
  FAIL_IF(scale == -1.0 && PyErr_Occurred());
  FAIL_IF(tensor(a[0], t_bf16, device, "k_pool", 0, &k) || tensor(a[1], t_bf16, device, "v_pool", 0, &v) ||
          tensor(a[2], t_bf16, device, "q", 0, &q) || tensor(a[3], t_bf16, device, "o", 0, &o) ||
          tensor(a[4], t_i32, device, "req_to_token", 0, &table) ||
          tensor(a[5], t_i32, device, "req_pool_indices", 0, &rpi) || tensor(a[6], t_i32, device, "prefix_lens", 0, &pl) ||
          tensor(a[7], t_i32, device, "draft_lens", 0, &dl) || tensor(a[8], t_i32, device, "qo_indptr", 0, &qo) ||
          tensor(a[9], t_i32, device, "tree_mask", 0, &mask) || workspace_of(a[13], device, &ws, &ws_bytes) ||
          tensor(a[14], t_i32, device, "device_error", 1, &err));
  const int ready = stream_of(device, a[15], &stream);
  FAIL_IF(ready < 0);
  Py_DECREF(device);
  if (ready) return PyLong_FromLong(-1);
  CALL(p_tree(k, v, s[0], (int32_t)s[1], (int32_t)s[2], q, o, (int32_t)qs[1], (float)scale, table, ts[1],
                                ts[0], rpi, pl, dl, qo, mask, (int32_t)ms[1], (int32_t)rs[0], qs[0], max_draft, max_prefix,
                                ws, ws_bytes, err, stream));
}

static PyMethodDef methods[] = {
    {"init", init, METH_VARARGS, "dtypes, stream and device functions, entry points"},
    {"kv8_store", (PyCFunction)(void (*)(void))kv8_store, METH_FASTCALL, NULL},
    {"kv8_load", (PyCFunction)(void (*)(void))kv8_load, METH_FASTCALL, NULL},
    {"kv8_decode", (PyCFunction)(void (*)(void))kv8_decode, METH_FASTCALL, NULL},
    {"norm_rope_store", (PyCFunction)(void (*)(void))norm_rope_store, METH_FASTCALL, NULL},
    {"norm_rope_kv8_store", (PyCFunction)(void (*)(void))norm_rope_kv8_store, METH_FASTCALL, NULL},
    {"tree", (PyCFunction)(void (*)(void))tree, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_ra_binding", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__ra_binding(void) {
  if (!(s_dtype = PyUnicode_InternFromString("dtype")) || !(s_device = PyUnicode_InternFromString("device")) ||
      !(s_shape = PyUnicode_InternFromString("shape")) || !(s_stride = PyUnicode_InternFromString("stride")) ||
      !(s_is_contiguous = PyUnicode_InternFromString("is_contiguous")) ||
      !(s_data_ptr = PyUnicode_InternFromString("data_ptr")) || !(s_type = PyUnicode_InternFromString("type")) ||
      !(s_index = PyUnicode_InternFromString("index")) || !(s_cuda_stream = PyUnicode_InternFromString("cuda_stream")))
    return NULL;
  return PyModule_Create(&module);
}
