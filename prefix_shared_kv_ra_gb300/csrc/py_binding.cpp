// py_binding.cpp -- argument checks and calls of the small per-step operators for Python.
//
// A decode step's store, norm or read-back takes the GPU 2-4 us, and a ctypes call with a dozen tensors took
// the host 7-15 us (about 0.35 us of checks per tensor and 3.6 us to convert 25 arguments), so the host set
// their rate.  These functions make the same checks on the tensors' C++ objects and call the library's entry
// points by address.  A wrong type raises TypeError, everything else ValueError; the return value is the
// library's status.  The tensors' device is made current for the call (the library asks for the current
// device's properties), and the interpreter lock is released (a launch may wait for room in its queue).
#include <Python.h>
#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <cstdint>
#include <exception>
#include <limits>

#include "../../include/ra.h"

namespace {

decltype(&ra_kv8_store) p_kv8_store;
decltype(&ra_kv8_load) p_kv8_load;
decltype(&ra_kv8_slot_bytes) p_kv8_slot_bytes;
decltype(&ra_kv8_decode_attention) p_kv8_decode;
decltype(&ra_qk_norm_rope_store) p_norm_rope;
decltype(&ra_qk_norm_rope_kv8_store) p_norm_rope_kv8;
decltype(&ra_tree_attention) p_tree;
decltype(&ra_step_slots) p_step_slots;
decltype(&ra_tree_verify) p_tree_verify;
decltype(&ra_tree_verify_greedy) p_tree_verify_greedy;
decltype(&ra_tree_commit) p_tree_commit;
decltype(&ra_extend_attention_mod) p_extend_mod;
decltype(&ra_decode_attention_mod) p_decode_mod;

PyObject* s_cuda_stream;

// A failed check: the Python exception is set.
struct Failed {};

[[noreturn]] void wrong(PyObject* type, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  PyErr_FormatV(type, fmt, ap);
  va_end(ap);
  throw Failed{};
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) wrong(PyExc_TypeError, "%s: expected a tensor, got %s", name, Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}

const at::Tensor& tensor(PyObject* o, const char* name, int64_t dims) {
  const at::Tensor& t = tensor(o, name);
  if (t.dim() != dims)
    wrong(PyExc_ValueError, "%s: expected %lld dimensions, got %lld", name, (long long)dims, (long long)t.dim());
  return t;
}

void typed(const at::Tensor& t, const char* name, at::ScalarType dtype, const at::Device& device) {
  if (t.scalar_type() != dtype)
    wrong(PyExc_TypeError, "%s: expected torch.%s, got torch.%s", name, c10::toString(dtype), c10::toString(t.scalar_type()));
  if (t.device() != device)
    wrong(PyExc_ValueError, "%s: expected device %s, got %s", name, device.str().c_str(), t.device().str().c_str());
}

// Address of a contiguous tensor of this type on this device.
template <typename T>
T* data(const at::Tensor& t, const char* name, at::ScalarType dtype, const at::Device& device) {
  typed(t, name, dtype, device);
  if (!t.is_contiguous()) wrong(PyExc_ValueError, "%s: must be contiguous", name);
  return static_cast<T*>(t.data_ptr());
}

// The same of an argument that may be None.
template <typename T>
T* optional_data(PyObject* o, const char* name, at::ScalarType dtype, const at::Device& device) {
  return o == Py_None ? nullptr : data<T>(tensor(o, name), name, dtype, device);
}

void same_shape(const at::Tensor& t, const at::Tensor& like, const char* name, const char* expected) {
  if (t.sizes() != like.sizes()) wrong(PyExc_ValueError, "%s: expected shape %s", name, expected);
}

void length(const at::Tensor& t, int64_t n, const char* name, const char* expected) {
  if (t.size(0) != n) wrong(PyExc_ValueError, "%s: expected shape %s", name, expected);
}

int32_t narrow(int64_t v, const char* name) {
  if (v < std::numeric_limits<int32_t>::min() || v > std::numeric_limits<int32_t>::max())
    wrong(PyExc_ValueError, "%s: %lld does not fit in 32 bits", name, (long long)v);
  return static_cast<int32_t>(v);
}

int32_t int_of(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Failed{};
  return narrow(v, name);
}

double float_of(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Failed{};
  return v;
}

// bf16 head rows [n, h, d]: a token's rows contiguous, tokens at any stride (a slice of a fused projection).
void* head_rows(const at::Tensor& t, const char* name, const at::Device& device, int64_t* stride) {
  typed(t, name, at::kBFloat16, device);
  const int64_t n = t.size(0), h = t.size(1), d = t.size(2);
  if ((t.stride(2) != 1 && d > 1) || (t.stride(1) != d && h > 1))
    wrong(PyExc_ValueError, "%s: a token's head rows must be contiguous", name);
  *stride = n > 1 ? t.stride(0) : h * d;
  return t.data_ptr();
}

// A pool of records for these heads, uint8 [num_slots, ra_kv8_slot_bytes(hkv, d)].
void* kv8_pool(const at::Tensor& t, int32_t hkv, int32_t d, const at::Device& device) {
  const size_t want = hkv > 0 ? p_kv8_slot_bytes(hkv, d) : 0;
  if (want == 0 || t.size(1) != static_cast<int64_t>(want))
    wrong(PyExc_ValueError, "kv8_pool: expected [num_slots, %zu] for %d kv heads of %d, got [%lld, %lld]", want, hkv, d,
          (long long)t.size(0), (long long)t.size(1));
  return data<void>(t, "kv8_pool", at::kByte, device);
}

// Run `call(stream)` on the device and the stream given (None: the device's current one).
template <typename Call>
PyObject* launch(const at::Device& device, PyObject* stream, Call call) {
  if (!device.is_cuda()) wrong(PyExc_ValueError, "expected CUDA tensors, got %s", device.str().c_str());
  c10::cuda::CUDAGuard guard(device);
  ra_stream_t s;
  if (stream == Py_None) {
    s = reinterpret_cast<ra_stream_t>(c10::cuda::getCurrentCUDAStream(device.index()).stream());
  } else {
    PyObject* raw = PyObject_GetAttr(stream, s_cuda_stream);
    if (!raw) throw Failed{};
    s = static_cast<ra_stream_t>(PyLong_AsVoidPtr(raw));
    Py_DECREF(raw);
    if (PyErr_Occurred()) throw Failed{};
  }
  ra_status status;
  Py_BEGIN_ALLOW_THREADS;
  status = call(s);
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(status);
}

// A method: its body with the checks' failures and C++ exceptions turned into Python ones.
template <typename Body>
PyObject* method(const char* name, Py_ssize_t got, Py_ssize_t want, Body body) {
  try {
    if (got != want) wrong(PyExc_TypeError, "%s: expected %zd arguments, got %zd", name, want, got);
    return body();
  } catch (const Failed&) {
  } catch (const std::exception& e) {
    PyErr_Format(PyExc_ValueError, "%s: %s", name, e.what());
  }
  return nullptr;
}

// store: (pool, k, v, loc, err, stream); load: (pool, slots, k, v, err, stream)
PyObject* kv8_move(PyObject* const* a, Py_ssize_t n, bool load) {
  return method(load ? "ra_kv8_load" : "ra_kv8_store", n, 6, [&] {
    const at::Tensor &pool = tensor(a[0], "kv8_pool", 2), &k = tensor(a[load ? 2 : 1], "K rows", 3),
                     &v = tensor(a[load ? 3 : 2], "V rows", 3), &loc = tensor(a[load ? 1 : 3], "slots", 1);
    const at::Device device = pool.device();
    same_shape(v, k, "V rows", "[num_tokens, Hkv, D], that of the K rows");
    length(loc, k.size(0), "slots", "[num_tokens]");
    const int32_t hkv = narrow(k.size(1), "Hkv"), d = narrow(k.size(2), "D");
    void* rec = kv8_pool(pool, hkv, d, device);
    void *kp = data<void>(k, "K rows", at::kBFloat16, device), *vp = data<void>(v, "V rows", at::kBFloat16, device);
    const int32_t* lp = data<int32_t>(loc, "slots", at::kInt, device);
    uint32_t* err = optional_data<uint32_t>(a[4], "device_error", at::kInt, device);
    const int64_t slots = pool.size(0), tokens = k.size(0);
    return launch(device, a[5], [&](ra_stream_t s) {
      return load ? p_kv8_load(rec, slots, hkv, d, lp, kp, vp, tokens, err, s)
                  : p_kv8_store(rec, slots, hkv, d, kp, vp, lp, tokens, err, s);
    });
  });
}

PyObject* kv8_store(PyObject*, PyObject* const* a, Py_ssize_t n) { return kv8_move(a, n, false); }
PyObject* kv8_load(PyObject*, PyObject* const* a, Py_ssize_t n) { return kv8_move(a, n, true); }

struct Workspace {
  void* at;
  size_t bytes;
};
Workspace workspace_of(PyObject* o, const at::Device& device) {
  const at::Tensor& t = tensor(o, "workspace");
  if (t.scalar_type() != at::kByte || t.device() != device || !t.is_contiguous())
    wrong(PyExc_ValueError, "workspace must be a contiguous uint8 tensor on the pool's device");
  return {t.data_ptr(), static_cast<size_t>(t.numel())};
}

// (pool, q, o, table, rpi, lens, num_kv_heads, max_seq_len, sm_scale, workspace, err, stream)
PyObject* kv8_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return method("ra_kv8_decode_attention", n, 12, [&] {
    const at::Tensor &pool = tensor(a[0], "kv8_pool", 2), &q = tensor(a[1], "q", 3), &o = tensor(a[2], "o", 3),
                     &table = tensor(a[3], "req_to_token", 2), &rpi = tensor(a[4], "req_pool_indices", 1),
                     &lens = tensor(a[5], "seq_lens", 1);
    const at::Device device = pool.device();
    const int32_t batch = narrow(q.size(0), "batch"), hq = narrow(q.size(1), "Hq"), d = narrow(q.size(2), "D");
    same_shape(o, q, "o", "that of q");
    length(rpi, batch, "req_pool_indices", "[batch]");
    length(lens, batch, "seq_lens", "[batch]");
    const int32_t hkv = int_of(a[6], "num_kv_heads"), max_len = int_of(a[7], "max_seq_len");
    const float scale = static_cast<float>(float_of(a[8]));
    void* rec = kv8_pool(pool, hkv, d, device);
    void *qp = data<void>(q, "q", at::kBFloat16, device), *op = data<void>(o, "o", at::kBFloat16, device);
    const int32_t *tp = data<int32_t>(table, "req_to_token", at::kInt, device),
                  *rp = data<int32_t>(rpi, "req_pool_indices", at::kInt, device),
                  *lp = data<int32_t>(lens, "seq_lens", at::kInt, device);
    const Workspace ws = workspace_of(a[9], device);
    uint32_t* err = optional_data<uint32_t>(a[10], "device_error", at::kInt, device);
    return launch(device, a[11], [&](ra_stream_t s) {
      return p_kv8_decode(rec, pool.size(0), hkv, d, qp, op, hq, scale, tp, table.size(1), table.size(0), rp, lp, batch,
                          max_len, ws.at, ws.bytes, err, s);
    });
  });
}

// (q, k, v, q_weight, k_weight, positions, cos_sin, q_out, pool or k_pool and v_pool, loc, eps, interleaved, err, stream)
PyObject* norm_rope(PyObject* const* a, Py_ssize_t n, bool kv8) {
  return method(kv8 ? "ra_qk_norm_rope_kv8_store" : "ra_qk_norm_rope_store", n, kv8 ? 14 : 15, [&] {
    PyObject* const* b = a + (kv8 ? 9 : 10);  // loc, eps, interleaved, err, stream
    const at::Tensor &q = tensor(a[0], "q", 3), &k = tensor(a[1], "k", 3), &v = tensor(a[2], "v", 3),
                     &positions = tensor(a[5], "positions", 1), &cos_sin = tensor(a[6], "cos_sin", 2),
                     &q_out = tensor(a[7], "q_out", 3), &pool = tensor(a[8], kv8 ? "kv8_pool" : "k_pool", kv8 ? 2 : 3),
                     &loc = tensor(b[0], "out_cache_loc", 1);
    const at::Device device = pool.device();
    const int64_t tokens = q.size(0);
    const int32_t hq = narrow(q.size(1), "Hq"), d = narrow(q.size(2), "D"), hkv = narrow(k.size(1), "Hkv");
    if (k.size(0) != tokens || k.size(2) != d) wrong(PyExc_ValueError, "k: expected shape [num_tokens, Hkv, D]");
    same_shape(v, k, "v", "that of k");
    same_shape(q_out, q, "q_out", "that of q");
    length(positions, tokens, "positions", "[num_tokens]");
    length(loc, tokens, "out_cache_loc", "[num_tokens]");
    for (int i = 3; i < 5; ++i)
      if (a[i] != Py_None) length(tensor(a[i], "weights", 1), d, "weights", "[D]");
    int64_t qs, ks, vs, qos;
    void *qp = head_rows(q, "q", device, &qs), *kp = head_rows(k, "k", device, &ks), *vp = head_rows(v, "v", device, &vs),
         *qop = head_rows(q_out, "q_out", device, &qos);
    void *qw = optional_data<void>(a[3], "q_weight", at::kBFloat16, device),
         *kw = optional_data<void>(a[4], "k_weight", at::kBFloat16, device);
    const int32_t *pp = data<int32_t>(positions, "positions", at::kInt, device),
                  *lp = data<int32_t>(loc, "out_cache_loc", at::kInt, device);
    const float* cs = data<float>(cos_sin, "cos_sin", at::kFloat, device);
    const int32_t rot = narrow(cos_sin.size(1), "rotary_dim");
    void *kpool, *vpool = nullptr;
    if (kv8) {
      kpool = kv8_pool(pool, hkv, d, device);
    } else {
      const at::Tensor& v_pool = tensor(a[9], "v_pool", 3);
      if (pool.size(1) != hkv || pool.size(2) != d) wrong(PyExc_ValueError, "k_pool: expected shape [num_slots, Hkv, D]");
      same_shape(v_pool, pool, "v_pool", "that of k_pool");
      kpool = data<void>(pool, "k_pool", at::kBFloat16, device);
      vpool = data<void>(v_pool, "v_pool", at::kBFloat16, device);
    }
    const float eps = static_cast<float>(float_of(b[1]));
    const int interleaved = PyObject_IsTrue(b[2]);
    if (interleaved < 0) throw Failed{};
    uint32_t* err = optional_data<uint32_t>(b[3], "device_error", at::kInt, device);
    return launch(device, b[4], [&](ra_stream_t s) {
      return kv8 ? p_norm_rope_kv8(qp, qs, kp, ks, vp, vs, hq, hkv, d, qw, kw, eps, pp, cs, cos_sin.size(0), rot, interleaved,
                                   qop, qos, kpool, pool.size(0), lp, tokens, err, s)
                 : p_norm_rope(qp, qs, kp, ks, vp, vs, hq, hkv, d, qw, kw, eps, pp, cs, cos_sin.size(0), rot, interleaved,
                               qop, qos, kpool, vpool, pool.size(0), lp, tokens, err, s);
    });
  });
}

PyObject* norm_rope_store(PyObject*, PyObject* const* a, Py_ssize_t n) { return norm_rope(a, n, false); }
PyObject* norm_rope_kv8_store(PyObject*, PyObject* const* a, Py_ssize_t n) { return norm_rope(a, n, true); }

// (k_pool, v_pool, q, o, table, rpi, prefix_lens, draft_lens, qo_indptr, tree_mask, max_draft_len, max_prefix_len,
//  sm_scale, workspace, err, stream)
PyObject* tree(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return method("ra_tree_attention", n, 16, [&] {
    const at::Tensor &k = tensor(a[0], "k_pool", 3), &v = tensor(a[1], "v_pool", 3), &q = tensor(a[2], "q", 3),
                     &o = tensor(a[3], "o", 3), &table = tensor(a[4], "req_to_token", 2),
                     &rpi = tensor(a[5], "req_pool_indices", 1), &prefix = tensor(a[6], "prefix_lens", 1),
                     &draft = tensor(a[7], "draft_lens", 1), &qo = tensor(a[8], "qo_indptr", 1),
                     &mask = tensor(a[9], "tree_mask", 2);
    const at::Device device = k.device();
    const int32_t hkv = narrow(k.size(1), "Hkv"), d = narrow(k.size(2), "D"), hq = narrow(q.size(1), "Hq"),
                  batch = narrow(rpi.size(0), "batch"), words = narrow(mask.size(1), "mask words");
    same_shape(v, k, "v_pool", "that of k_pool");
    if (q.size(2) != d) wrong(PyExc_ValueError, "q: expected shape [total_q, Hq, D]");
    same_shape(o, q, "o", "that of q");
    length(prefix, batch, "prefix_lens", "[batch]");
    length(draft, batch, "draft_lens", "[batch]");
    length(qo, static_cast<int64_t>(batch) + 1, "qo_indptr", "[batch + 1]");
    length(mask, q.size(0), "tree_mask", "[total_q, words]");
    const int32_t max_draft = int_of(a[10], "max_draft_len"), max_prefix = int_of(a[11], "max_prefix_len");
    const float scale = static_cast<float>(float_of(a[12]));
    void *kp = data<void>(k, "k_pool", at::kBFloat16, device), *vp = data<void>(v, "v_pool", at::kBFloat16, device),
         *qp = data<void>(q, "q", at::kBFloat16, device), *op = data<void>(o, "o", at::kBFloat16, device);
    const int32_t *tp = data<int32_t>(table, "req_to_token", at::kInt, device),
                  *rp = data<int32_t>(rpi, "req_pool_indices", at::kInt, device),
                  *pp = data<int32_t>(prefix, "prefix_lens", at::kInt, device),
                  *dp = data<int32_t>(draft, "draft_lens", at::kInt, device),
                  *ip = data<int32_t>(qo, "qo_indptr", at::kInt, device);
    const uint32_t* mp = data<uint32_t>(mask, "tree_mask", at::kInt, device);
    const Workspace ws = workspace_of(a[13], device);
    uint32_t* err = optional_data<uint32_t>(a[14], "device_error", at::kInt, device);
    return launch(device, a[15], [&](ra_stream_t s) {
      return p_tree(kp, vp, k.size(0), hkv, d, qp, op, hq, scale, tp, table.size(1), table.size(0), rp, pp, dp, ip, mp, words,
                    batch, q.size(0), max_draft, max_prefix, ws.at, ws.bytes, err, s);
    });
  });
}

// extend: (k_pool, v_pool, q, o, table, rpi, prefix_lens, extend_lens, qo_indptr, max_extend_len, max_prefix_len, sm_scale,
//  workspace, score_cap, window, slopes, first_key, full_lens, err, stream)
// decode: (k_pool, v_pool, q, o, table, rpi, seq_lens, max_seq_len, sm_scale, workspace, score_cap, window, slopes,
//  first_key, err, stream)
PyObject* attention_mod(PyObject* const* a, Py_ssize_t n, bool extend) {
  return method(extend ? "ra_extend_attention_mod" : "ra_decode_attention_mod", n, extend ? 20 : 16, [&] {
    const at::Tensor &k = tensor(a[0], "k_pool", 3), &v = tensor(a[1], "v_pool", 3), &q = tensor(a[2], "q", 3),
                     &o = tensor(a[3], "o", 3), &table = tensor(a[4], "req_to_token", 2),
                     &rpi = tensor(a[5], "req_pool_indices", 1),
                     &lens = tensor(a[6], extend ? "prefix_lens" : "seq_lens", 1);
    const at::Device device = k.device();
    const int32_t hkv = narrow(k.size(1), "Hkv"), d = narrow(k.size(2), "D"), hq = narrow(q.size(1), "Hq"),
                  batch = narrow(rpi.size(0), "batch");
    same_shape(v, k, "v_pool", "that of k_pool");
    if (q.size(2) != d) wrong(PyExc_ValueError, "q: expected shape [%s, Hq, D]", extend ? "total_q" : "batch");
    same_shape(o, q, "o", "that of q");
    length(lens, batch, extend ? "prefix_lens" : "seq_lens", "[batch]");
    if (!extend) length(q, batch, "q", "[batch, Hq, D]");
    auto i32 = [&](const at::Tensor& t, const char* name) { return data<int32_t>(t, name, at::kInt, device); };
    void *kp = data<void>(k, "k_pool", at::kBFloat16, device), *vp = data<void>(v, "v_pool", at::kBFloat16, device),
         *qp = data<void>(q, "q", at::kBFloat16, device), *op = data<void>(o, "o", at::kBFloat16, device);
    const int32_t *tp = i32(table, "req_to_token"), *rp = i32(rpi, "req_pool_indices"),
                  *lp = i32(lens, extend ? "prefix_lens" : "seq_lens");
    PyObject* const* b = a + (extend ? 9 : 7);  // max_extend_len, max_prefix_len or max_seq_len
    PyObject* const* c = b + (extend ? 2 : 1);  // sm_scale, workspace, score_cap, window, slopes, first_key
    const int32_t longest = int_of(b[0], extend ? "max_extend_len" : "max_seq_len"),
                  prefix = extend ? int_of(b[1], "max_prefix_len") : 0;
    const float scale = static_cast<float>(float_of(c[0])), cap = static_cast<float>(float_of(c[2]));
    const Workspace ws = workspace_of(c[1], device);
    const int32_t window = int_of(c[3], "window");
    if (c[4] != Py_None) length(tensor(c[4], "slopes", 1), hq, "slopes", "[Hq]");
    if (c[5] != Py_None)
      length(tensor(c[5], "first_key", 1), q.size(0), "first_key", extend ? "[total_q]" : "[batch]");
    const float* slopes = optional_data<float>(c[4], "slopes", at::kFloat, device);
    const int32_t* first = optional_data<int32_t>(c[5], "first_key", at::kInt, device);
    if (!extend) {
      uint32_t* err = optional_data<uint32_t>(c[6], "device_error", at::kInt, device);
      return launch(device, c[7], [&](ra_stream_t s) {
        return p_decode_mod(kp, vp, k.size(0), hkv, d, qp, op, hq, scale, cap, window, slopes, first, tp, table.size(1),
                            table.size(0), rp, lp, batch, longest, ws.at, ws.bytes, err, s);
      });
    }
    const at::Tensor &news = tensor(a[7], "extend_lens", 1), &qo = tensor(a[8], "qo_indptr", 1);
    length(news, batch, "extend_lens", "[batch]");
    length(qo, static_cast<int64_t>(batch) + 1, "qo_indptr", "[batch + 1]");
    if (c[6] != Py_None) length(tensor(c[6], "full_lens", 1), batch, "full_lens", "[batch]");
    const int32_t *np = i32(news, "extend_lens"), *ip = i32(qo, "qo_indptr"),
                  *full = optional_data<int32_t>(c[6], "full_lens", at::kInt, device);
    uint32_t* err = optional_data<uint32_t>(c[7], "device_error", at::kInt, device);
    return launch(device, c[8], [&](ra_stream_t s) {
      return p_extend_mod(kp, vp, k.size(0), hkv, d, qp, op, hq, scale, cap, window, slopes, first, full, tp, table.size(1),
                          table.size(0), rp, lp, np, ip, batch, q.size(0), longest, prefix, ws.at, ws.bytes, err, s);
    });
  });
}

PyObject* extend_mod(PyObject*, PyObject* const* a, Py_ssize_t n) { return attention_mod(a, n, true); }
PyObject* decode_mod(PyObject*, PyObject* const* a, Py_ssize_t n) { return attention_mod(a, n, false); }

// (table, rpi, seq_lens, new_lens, free_pages, free_count, out_cache_loc, positions, qo_indptr, seq_lens_out, page_size,
//  free_count_out or None, err, stream)
PyObject* step_slots(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return method("ra_step_slots", n, 14, [&] {
    const at::Tensor &table = tensor(a[0], "req_to_token", 2), &rpi = tensor(a[1], "req_pool_indices", 1),
                     &lens = tensor(a[2], "seq_lens", 1), &news = tensor(a[3], "new_lens", 1),
                     &pages = tensor(a[4], "free_pages", 1), &count = tensor(a[5], "free_count", 1),
                     &loc = tensor(a[6], "out_cache_loc", 1), &positions = tensor(a[7], "positions", 1),
                     &qo = tensor(a[8], "qo_indptr", 1), &out = tensor(a[9], "seq_lens_out", 1);
    const at::Tensor& left = a[11] == Py_None ? count : tensor(a[11], "free_count_out", 1);
    const at::Device device = table.device();
    const int32_t batch = narrow(rpi.size(0), "batch");
    length(lens, batch, "seq_lens", "[batch]");
    length(news, batch, "new_lens", "[batch]");
    length(out, batch, "seq_lens_out", "[batch]");
    length(qo, static_cast<int64_t>(batch) + 1, "qo_indptr", "[batch + 1]");
    length(positions, loc.size(0), "positions", "[num_tokens]");
    length(count, 1, "free_count", "[1]");
    length(left, 1, "free_count_out", "[1]");
    const int32_t page = int_of(a[10], "page_size");
    auto i32 = [&](const at::Tensor& t, const char* name) { return data<int32_t>(t, name, at::kInt, device); };
    int32_t *tp = i32(table, "req_to_token"), *lp = i32(loc, "out_cache_loc"), *pp = i32(positions, "positions"),
            *qp = i32(qo, "qo_indptr"), *op = i32(out, "seq_lens_out"), *fo = i32(left, "free_count_out");
    const int32_t *rp = i32(rpi, "req_pool_indices"), *sp = i32(lens, "seq_lens"), *np = i32(news, "new_lens"),
                  *fp = i32(pages, "free_pages"), *fc = i32(count, "free_count");
    uint32_t* err = optional_data<uint32_t>(a[12], "device_error", at::kInt, device);
    return launch(device, a[13], [&](ra_stream_t s) {
      return p_step_slots(tp, table.size(1), table.size(0), rp, sp, np, batch, fp, pages.size(0), fc, fo, page, lp, pp,
                          loc.size(0), qp, op, err, s);
    });
  });
}

// Rows [n, vocab] of one of two types, the values of a row contiguous, rows at any stride (>= vocab).
const void* vocab_rows(const at::Tensor& t, const char* name, const at::Device& device, int64_t* stride) {
  if (t.device() != device)
    wrong(PyExc_ValueError, "%s: expected device %s, got %s", name, device.str().c_str(), t.device().str().c_str());
  const int64_t n = t.size(0), vocab = t.size(1);
  if (vocab > 1 && t.stride(1) != 1) wrong(PyExc_ValueError, "%s: a row's values must be contiguous", name);
  *stride = n > 1 ? t.stride(0) : vocab;
  if (*stride < vocab) wrong(PyExc_ValueError, "%s: rows must not overlap", name);
  return t.data_ptr();
}

// target, [draft_probs], tokens, parents, draft_lens, qo_indptr, [accept_uniforms, final_uniforms], path, accept_lens,
// next_tokens, max_draft_len, err, stream; in brackets: not for the greedy form
PyObject* verify(PyObject* const* a, Py_ssize_t n, bool greedy) {
  return method(greedy ? "ra_tree_verify_greedy" : "ra_tree_verify", n, greedy ? 11 : 14, [&] {
    PyObject* const* tree = a + (greedy ? 1 : 2);
    PyObject* const* out = tree + (greedy ? 4 : 6);
    const at::Tensor &target = tensor(a[0], greedy ? "target_logits" : "target_probs", 2),
                     &tokens = tensor(tree[0], "draft_tokens", 1), &parents = tensor(tree[1], "parents", 1),
                     &drafts = tensor(tree[2], "draft_lens", 1), &qo = tensor(tree[3], "qo_indptr", 1),
                     &path = tensor(out[0], "path", 2), &accepted = tensor(out[1], "accept_lens", 1),
                     &next = tensor(out[2], "next_tokens", 1);
    const at::Device device = target.device();
    const int64_t total = target.size(0);
    const int32_t batch = narrow(drafts.size(0), "batch"), vocab = narrow(target.size(1), "vocab");
    const int32_t max_draft = int_of(out[3], "max_draft_len");
    length(tokens, total, "draft_tokens", "[total_q]");
    length(parents, total, "parents", "[total_q]");
    length(qo, static_cast<int64_t>(batch) + 1, "qo_indptr", "[batch + 1]");
    length(accepted, batch, "accept_lens", "[batch]");
    length(next, batch, "next_tokens", "[batch]");
    if (path.size(0) != batch || path.size(1) != max_draft)
      wrong(PyExc_ValueError, "path: expected shape [batch, max_draft_len]");
    int64_t stride, draft_stride = 0;
    const void* tp = vocab_rows(target, greedy ? "target_logits" : "target_probs", device, &stride);
    auto i32 = [&](const at::Tensor& t, const char* name) { return data<int32_t>(t, name, at::kInt, device); };
    const int32_t *kp = i32(tokens, "draft_tokens"), *pp = i32(parents, "parents"), *dp = i32(drafts, "draft_lens"),
                  *qp = i32(qo, "qo_indptr");
    int32_t *wp = i32(path, "path"), *ap = i32(accepted, "accept_lens"), *np = i32(next, "next_tokens");
    uint32_t* err = optional_data<uint32_t>(out[4], "device_error", at::kInt, device);
    if (greedy) {
      const bool fp32 = target.scalar_type() == at::kFloat;
      if (!fp32) typed(target, "target_logits", at::kBFloat16, device);
      return launch(device, out[5], [&](ra_stream_t s) {
        return p_tree_verify_greedy(tp, fp32, stride, vocab, kp, pp, dp, qp, batch, total, max_draft, wp, ap, np, err, s);
      });
    }
    typed(target, "target_probs", at::kFloat, device);
    const void* draft = nullptr;
    if (a[1] != Py_None) {
      const at::Tensor& q = tensor(a[1], "draft_probs", 2);
      typed(q, "draft_probs", at::kFloat, device);
      same_shape(q, target, "draft_probs", "that of target_probs");
      draft = vocab_rows(q, "draft_probs", device, &draft_stride);
    }
    const at::Tensor &ua = tensor(tree[4], "accept_uniforms", 1), &uf = tensor(tree[5], "final_uniforms", 1);
    length(ua, total, "accept_uniforms", "[total_q]");
    length(uf, batch, "final_uniforms", "[batch]");
    const float *uap = data<float>(ua, "accept_uniforms", at::kFloat, device),
                *ufp = data<float>(uf, "final_uniforms", at::kFloat, device);
    return launch(device, out[5], [&](ra_stream_t s) {
      return p_tree_verify(static_cast<const float*>(tp), stride, static_cast<const float*>(draft), draft_stride, vocab, kp,
                           pp, dp, qp, uap, ufp, batch, total, max_draft, wp, ap, np, err, s);
    });
  });
}

PyObject* tree_verify(PyObject*, PyObject* const* a, Py_ssize_t n) { return verify(a, n, false); }
PyObject* tree_verify_greedy(PyObject*, PyObject* const* a, Py_ssize_t n) { return verify(a, n, true); }

// (table, rpi, prefix_lens, draft_lens, qo_indptr, out_cache_loc, path, accept_lens, seq_lens_out, free_list, free_count,
//  free_count_out or None, err, stream)
PyObject* tree_commit(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return method("ra_tree_commit", n, 14, [&] {
    const at::Tensor &table = tensor(a[0], "req_to_token", 2), &rpi = tensor(a[1], "req_pool_indices", 1),
                     &prefix = tensor(a[2], "prefix_lens", 1), &drafts = tensor(a[3], "draft_lens", 1),
                     &qo = tensor(a[4], "qo_indptr", 1), &loc = tensor(a[5], "out_cache_loc", 1),
                     &path = tensor(a[6], "path", 2), &accepted = tensor(a[7], "accept_lens", 1),
                     &out = tensor(a[8], "seq_lens_out", 1), &list = tensor(a[9], "free_list", 1),
                     &count = tensor(a[10], "free_count", 1);
    const at::Tensor& left = a[11] == Py_None ? count : tensor(a[11], "free_count_out", 1);
    const at::Device device = table.device();
    const int32_t batch = narrow(rpi.size(0), "batch");
    length(prefix, batch, "prefix_lens", "[batch]");
    length(drafts, batch, "draft_lens", "[batch]");
    length(qo, static_cast<int64_t>(batch) + 1, "qo_indptr", "[batch + 1]");
    length(path, batch, "path", "[batch, max_draft_len]");
    length(accepted, batch, "accept_lens", "[batch]");
    length(out, batch, "seq_lens_out", "[batch]");
    length(count, 1, "free_count", "[1]");
    length(left, 1, "free_count_out", "[1]");
    auto i32 = [&](const at::Tensor& t, const char* name) { return data<int32_t>(t, name, at::kInt, device); };
    int32_t *tp = i32(table, "req_to_token"), *op = i32(out, "seq_lens_out"), *fp = i32(list, "free_list"),
            *fo = i32(left, "free_count_out");
    const int32_t *rp = i32(rpi, "req_pool_indices"), *pp = i32(prefix, "prefix_lens"), *dp = i32(drafts, "draft_lens"),
                  *qp = i32(qo, "qo_indptr"), *lp = i32(loc, "out_cache_loc"), *wp = i32(path, "path"),
                  *ap = i32(accepted, "accept_lens"), *fc = i32(count, "free_count");
    const int32_t stride = narrow(path.size(1), "max_draft_len");
    uint32_t* err = optional_data<uint32_t>(a[12], "device_error", at::kInt, device);
    return launch(device, a[13], [&](ra_stream_t s) {
      return p_tree_commit(tp, table.size(1), table.size(0), rp, pp, dp, qp, batch, lp, loc.size(0), wp, stride, ap, op, fp,
                           list.size(0), fc, fo, err, s);
    });
  });
}

// init(addresses of the entry points in the order of the declarations above)
PyObject* init(PyObject*, PyObject* args) {
  unsigned long long a[13];
  if (!PyArg_ParseTuple(args, "KKKKKKKKKKKKK", a, a + 1, a + 2, a + 3, a + 4, a + 5, a + 6, a + 7, a + 8, a + 9, a + 10,
                        a + 11, a + 12))
    return nullptr;
  p_kv8_store = reinterpret_cast<decltype(p_kv8_store)>(a[0]);
  p_kv8_load = reinterpret_cast<decltype(p_kv8_load)>(a[1]);
  p_kv8_slot_bytes = reinterpret_cast<decltype(p_kv8_slot_bytes)>(a[2]);
  p_kv8_decode = reinterpret_cast<decltype(p_kv8_decode)>(a[3]);
  p_norm_rope = reinterpret_cast<decltype(p_norm_rope)>(a[4]);
  p_norm_rope_kv8 = reinterpret_cast<decltype(p_norm_rope_kv8)>(a[5]);
  p_tree = reinterpret_cast<decltype(p_tree)>(a[6]);
  p_step_slots = reinterpret_cast<decltype(p_step_slots)>(a[7]);
  p_tree_verify = reinterpret_cast<decltype(p_tree_verify)>(a[8]);
  p_tree_verify_greedy = reinterpret_cast<decltype(p_tree_verify_greedy)>(a[9]);
  p_tree_commit = reinterpret_cast<decltype(p_tree_commit)>(a[10]);
  p_extend_mod = reinterpret_cast<decltype(p_extend_mod)>(a[11]);
  p_decode_mod = reinterpret_cast<decltype(p_decode_mod)>(a[12]);
  Py_RETURN_NONE;
}

PyCFunction fast(PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {{"init", init, METH_VARARGS, "entry points of the library"},
                         {"kv8_store", fast(kv8_store), METH_FASTCALL, nullptr},
                         {"kv8_load", fast(kv8_load), METH_FASTCALL, nullptr},
                         {"kv8_decode", fast(kv8_decode), METH_FASTCALL, nullptr},
                         {"norm_rope_store", fast(norm_rope_store), METH_FASTCALL, nullptr},
                         {"norm_rope_kv8_store", fast(norm_rope_kv8_store), METH_FASTCALL, nullptr},
                         {"tree", fast(tree), METH_FASTCALL, nullptr},
                         {"step_slots", fast(step_slots), METH_FASTCALL, nullptr},
                         {"tree_verify", fast(tree_verify), METH_FASTCALL, nullptr},
                         {"tree_verify_greedy", fast(tree_verify_greedy), METH_FASTCALL, nullptr},
                         {"tree_commit", fast(tree_commit), METH_FASTCALL, nullptr},
                         {"extend_mod", fast(extend_mod), METH_FASTCALL, nullptr},
                         {"decode_mod", fast(decode_mod), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_ra_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ra_binding() {
  s_cuda_stream = PyUnicode_InternFromString("cuda_stream");
  return s_cuda_stream ? PyModule_Create(&module) : nullptr;
}
