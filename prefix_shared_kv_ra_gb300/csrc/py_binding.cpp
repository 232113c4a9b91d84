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

// init(addresses of the entry points in the order of the declarations above)
PyObject* init(PyObject*, PyObject* args) {
  unsigned long long a[7];
  if (!PyArg_ParseTuple(args, "KKKKKKK", a, a + 1, a + 2, a + 3, a + 4, a + 5, a + 6)) return nullptr;
  p_kv8_store = reinterpret_cast<decltype(p_kv8_store)>(a[0]);
  p_kv8_load = reinterpret_cast<decltype(p_kv8_load)>(a[1]);
  p_kv8_slot_bytes = reinterpret_cast<decltype(p_kv8_slot_bytes)>(a[2]);
  p_kv8_decode = reinterpret_cast<decltype(p_kv8_decode)>(a[3]);
  p_norm_rope = reinterpret_cast<decltype(p_norm_rope)>(a[4]);
  p_norm_rope_kv8 = reinterpret_cast<decltype(p_norm_rope_kv8)>(a[5]);
  p_tree = reinterpret_cast<decltype(p_tree)>(a[6]);
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
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_ra_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ra_binding() {
  s_cuda_stream = PyUnicode_InternFromString("cuda_stream");
  return s_cuda_stream ? PyModule_Create(&module) : nullptr;
}
