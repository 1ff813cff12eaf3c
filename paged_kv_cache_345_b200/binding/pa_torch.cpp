// Argument marshalling of the cache writes and of the calls of a decode step with
// drafted tokens, in C++: from torch tensors straight to the C ABI (include/pa.h).
// The Python functions of the package carry the signatures and documentation and
// pass their arguments on in order; what they check is checked here, with the same
// exceptions (ValueError, TypeError, PagedAttentionError). Small calls are bound by
// this: the rows of a step of 8 sequences took 15.3 us a call with the checks in
// Python and take 3.5 us here, writing and moving their accepted rows (two calls)
// 17.8 us and 5.6 us.
//
// The C functions are bound by address from the library that the package has
// loaded, so there is one library, one device error word and one last error.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <cstdint>

#include "pa.h"

namespace {

struct Bound {
  decltype(&::pa_kv_append) kv_append;
  decltype(&::pa_kv_append_fp8) kv_append_fp8;
  decltype(&::pa_qk_norm_rope_append) qk_norm_rope_append;
  decltype(&::pa_decode_tree) decode_tree;
  decltype(&::pa_verify_draft) verify_draft;
  decltype(&::pa_kv_accept) kv_accept;
  decltype(&::pa_last_error) last_error;
} lib = {};
PyObject* error_class = nullptr;

struct Raised {};  // a Python exception is set

[[noreturn]] void raise(PyObject* type, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  PyErr_FormatV(type, fmt, ap);
  va_end(ap);
  throw Raised{};
}

const char* type_name(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return "torch.float32";
    case at::kBFloat16: return "torch.bfloat16";
    case at::kInt: return "torch.int32";
    case at::kLong: return "torch.int64";
    case at::kByte: return "torch.uint8";
    case at::kFloat8_e4m3fn: return "torch.float8_e4m3fn";
    default: return c10::toString(t);
  }
}

constexpr at::ScalarType kAny = at::ScalarType::Undefined;
bool is_codes(at::ScalarType t) { return t == at::kByte || t == at::kFloat8_e4m3fn; }

// The tensors of one call: each checked as it is taken, all on one device.
class Call {
 public:
  const at::Tensor* optional(PyObject* o, const char* name, at::ScalarType type = kAny) {
    return o == Py_None ? nullptr : &tensor(o, name, type, true);
  }
  const at::Tensor& tensor(PyObject* o, const char* name, at::ScalarType type = kAny,
                           bool contiguous = true) {
    if (!THPVariable_Check(o)) raise(PyExc_TypeError, "%s must be a tensor", name);
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda()) raise(PyExc_ValueError, "%s must be a CUDA tensor", name);
    if (contiguous && !t.is_contiguous()) raise(PyExc_ValueError, "%s must be contiguous", name);
    if (type != kAny && t.scalar_type() != type)
      raise(PyExc_TypeError, "%s must be %s, got %s", name, type_name(type), type_name(t.scalar_type()));
    const int d = t.get_device();
    if (device_ < 0) device_ = d;
    if (d != device_)
      raise(PyExc_ValueError, "tensors of one call are on several devices: cuda:%d, cuda:%d", device_, d);
    return t;
  }
  // [N, heads, d] with dense heads, tokens any stride apart: the elements between them.
  int64_t rows(const at::Tensor& t, const char* name) {
    const int64_t n = t.size(0), h = t.size(1), d = t.size(2);
    if (t.numel() != 0 && ((d > 1 && t.stride(2) != 1) || (h > 1 && t.stride(1) != d)))
      raise(PyExc_ValueError, "%s must be [N, heads, head_dim] with dense heads", name);
    return n > 1 ? t.stride(0) : h * d;
  }
  // An explicit stream must belong to the tensors' device; None is torch's current one there.
  pa_stream_t stream(PyObject* o) {
    if (o == Py_None) return reinterpret_cast<pa_stream_t>(c10::cuda::getCurrentCUDAStream(device_).stream());
    PyObject* dev = attribute(o, "device");
    PyObject* index = PyObject_GetAttrString(dev, "index");
    Py_DECREF(dev);
    if (!index) throw Raised{};
    const long on = index == Py_None ? -1 : PyLong_AsLong(index);
    Py_DECREF(index);
    if (PyErr_Occurred()) throw Raised{};
    if (on != device_) raise(PyExc_ValueError, "stream is on cuda:%ld, the tensors on cuda:%d", on, device_);
    PyObject* raw = attribute(o, "cuda_stream");
    const unsigned long long handle = PyLong_AsUnsignedLongLong(raw);
    Py_DECREF(raw);
    if (PyErr_Occurred()) throw Raised{};
    return reinterpret_cast<pa_stream_t>(static_cast<uintptr_t>(handle));
  }
  int device() const { return device_; }

 private:
  static PyObject* attribute(PyObject* o, const char* name) {
    PyObject* v = PyObject_GetAttrString(o, name);
    if (!v) throw Raised{};
    return v;
  }
  int device_ = -1;
};

void* at_(const at::Tensor* t) { return t ? t->data_ptr() : nullptr; }
void* at_(const at::Tensor& t) { return t.data_ptr(); }
template <typename T>
T* to(const at::Tensor& t) { return static_cast<T*>(t.data_ptr()); }
template <typename T>
T* to(const at::Tensor* t) { return t ? static_cast<T*>(t->data_ptr()) : nullptr; }

bool shaped(const at::Tensor& t, std::initializer_list<int64_t> s) {
  return t.sizes() == c10::IntArrayRef(s.begin(), s.size());
}

// Sizes reach the C ABI as int.
int narrow(int64_t x, const char* what) {
  if (x < INT32_MIN || x > INT32_MAX) raise(PyExc_ValueError, "%s %lld does not fit 32 bits", what, static_cast<long long>(x));
  return static_cast<int>(x);
}
double number(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw Raised{};
  return x;
}
int64_t whole(PyObject* o) {
  PyObject* i = PyNumber_Index(o);
  if (!i) throw Raised{};
  const int64_t x = PyLong_AsLongLong(i);
  Py_DECREF(i);
  if (x == -1 && PyErr_Occurred()) throw Raised{};
  return x;
}

pa_dtype cache_type(const at::Tensor& t) {
  if (t.scalar_type() == at::kBFloat16) return PA_BF16;
  if (t.scalar_type() == at::kFloat) return PA_F32;
  if (is_codes(t.scalar_type())) return PA_FP8_E4M3;
  raise(PyExc_TypeError, "unsupported dtype %s (float32, bfloat16, or uint8 E4M3 codes)", type_name(t.scalar_type()));
}

struct Cache {
  const at::Tensor &k, &v;
  int nb, bs, hkv, d;
  pa_dtype type;
};
Cache caches(Call& c, PyObject* ko, PyObject* vo) {
  const at::Tensor& k = c.tensor(ko, "k_cache");
  const pa_dtype type = cache_type(k);
  // (E4M3 codes: uint8 and float8_e4m3fn are the same bytes, and K and V may differ in it)
  const at::Tensor& v = c.tensor(vo, "v_cache");
  if (v.scalar_type() != k.scalar_type() && !(is_codes(k.scalar_type()) && is_codes(v.scalar_type())))
    raise(PyExc_TypeError, "v_cache must be %s, got %s", type_name(k.scalar_type()), type_name(v.scalar_type()));
  if (k.dim() != 4) raise(PyExc_ValueError, "k_cache must be [num_blocks, block_size, num_kv_heads, head_dim]");
  if (v.sizes() != k.sizes()) raise(PyExc_ValueError, "cache shape mismatch");
  return Cache{k, v, narrow(k.size(0), "num_blocks"), narrow(k.size(1), "block_size"),
               narrow(k.size(2), "num_kv_heads"), narrow(k.size(3), "head_dim"), type};
}

// One C call, other Python threads free to run meanwhile (a launch waits when the
// stream's queue is full).
template <typename... P, typename... A>
void call(int (*fn)(P...), A... args) {
  PyThreadState* held = PyEval_SaveThread();
  const int status = fn(args...);
  PyEval_RestoreThread(held);
  if (status == PA_OK) return;
  PyObject* e = PyObject_CallFunction(error_class, "is", status, lib.last_error());
  if (e) {
    PyErr_SetObject(error_class, e);
    Py_DECREF(e);
  }
  throw Raised{};
}

// Runs `f` for one Python call of n arguments; other exceptions become RuntimeError.
template <typename F>
PyObject* guarded(const char* name, Py_ssize_t got, Py_ssize_t want, F&& f) {
  if (got != want) {
    PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, got %zd", name, want, got);
    return nullptr;
  }
  try {
    f();
  } catch (const Raised&) {
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
  Py_RETURN_NONE;
}

// k_new, v_new, slot_mapping, k_cache, v_cache, stream
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("kv_append", n, 6, [&] {
    Call c;
    const Cache kv = caches(c, a[3], a[4]);
    const at::ScalarType dt = kv.k.scalar_type();
    c.tensor(a[4], "v_cache", dt);
    const at::Tensor& k = c.tensor(a[0], "k_new", dt);
    const at::Tensor& v = c.tensor(a[1], "v_new", dt);
    const at::Tensor& slots = c.tensor(a[2], "slot_mapping", at::kLong);
    if (k.dim() != 3 || k.size(1) != kv.hkv || k.size(2) != kv.d || v.sizes() != k.sizes())
      raise(PyExc_ValueError, "k_new/v_new must be [N, num_kv_heads, head_dim] matching the cache");
    if (!shaped(slots, {k.size(0)})) raise(PyExc_ValueError, "cache or slot_mapping shape mismatch");
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(c.device()));
    call(lib.kv_append, at_(k), at_(v), to<int64_t>(slots), narrow(k.size(0), "num_tokens"), at_(kv.k), at_(kv.v),
         kv.nb, kv.bs, kv.hkv, kv.d, kv.type, c.stream(a[5]));
  });
}

// k_new, v_new, slot_mapping, k_cache, v_cache, k_scale, v_scale, stream
PyObject* kv_append_fp8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("kv_append_fp8", n, 8, [&] {
    Call c;
    const Cache kv = caches(c, a[3], a[4]);
    if (kv.type != PA_FP8_E4M3) raise(PyExc_TypeError, "caches must hold E4M3 codes (uint8 or float8_e4m3fn)");
    const at::Tensor& k = c.tensor(a[0], "k_new", at::kBFloat16);
    const at::Tensor& v = c.tensor(a[1], "v_new", at::kBFloat16);
    const at::Tensor& slots = c.tensor(a[2], "slot_mapping", at::kLong);
    if (k.dim() != 3 || k.size(1) != kv.hkv || k.size(2) != kv.d || v.sizes() != k.sizes())
      raise(PyExc_ValueError, "k_new/v_new must be [N, num_kv_heads, head_dim] matching the cache");
    if (!shaped(slots, {k.size(0)})) raise(PyExc_ValueError, "cache or slot_mapping shape mismatch");
    const at::Tensor& ks = c.tensor(a[5], "k_scale", at::kFloat);
    const at::Tensor& vs = c.tensor(a[6], "v_scale", at::kFloat);
    if (!shaped(ks, {kv.hkv}) || !shaped(vs, {kv.hkv}))
      raise(PyExc_ValueError, "k_scale/v_scale must be [num_kv_heads]");
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(c.device()));
    call(lib.kv_append_fp8, at_(k), at_(v), to<int64_t>(slots), narrow(k.size(0), "num_tokens"), at_(kv.k),
         at_(kv.v), to<float>(ks), to<float>(vs), kv.nb, kv.bs, kv.hkv, kv.d, c.stream(a[7]));
  });
}

// q_out, q, k, v, positions, slot_mapping, k_cache, v_cache, cos_sin, q_weight, k_weight,
// eps, interleaved, k_scale, v_scale, stream
PyObject* qk_norm_rope_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("qk_norm_rope_append", n, 16, [&] {
    Call c;
    const Cache kv = caches(c, a[6], a[7]);
    const bool fp8 = kv.type == PA_FP8_E4M3;
    const at::ScalarType dt = fp8 ? at::kBFloat16 : kv.k.scalar_type();
    const at::Tensor& out = c.tensor(a[0], "q_out", dt, false);
    const at::Tensor& q = c.tensor(a[1], "q", dt, false);
    const at::Tensor& k = c.tensor(a[2], "k", dt, false);
    const at::Tensor& v = c.tensor(a[3], "v", dt, false);
    if (q.dim() != 3 || k.dim() != 3 || q.size(2) != kv.d || k.size(2) != kv.d || k.size(1) != kv.hkv ||
        out.sizes() != q.sizes() || v.sizes() != k.sizes() || k.size(0) != q.size(0))
      raise(PyExc_ValueError, "q/q_out must be [N, num_heads, head_dim], k/v [N, num_kv_heads, head_dim]");
    const at::Tensor& pos = c.tensor(a[4], "positions", at::kInt);
    const at::Tensor& slots = c.tensor(a[5], "slot_mapping", at::kLong);
    if (!shaped(pos, {q.size(0)}) || !shaped(slots, {q.size(0)}))
      raise(PyExc_ValueError, "cache, positions or slot_mapping shape mismatch");
    const at::Tensor& cs = c.tensor(a[8], "cos_sin", at::kFloat);
    if (cs.dim() != 2) raise(PyExc_ValueError, "cos_sin must be [max_position, rotary_dim]");
    const at::Tensor* qw = c.optional(a[9], "q_weight", dt);
    const at::Tensor* kw = c.optional(a[10], "k_weight", dt);
    if (qw && !shaped(*qw, {kv.d})) raise(PyExc_ValueError, "q_weight must be [head_dim]");
    if (kw && !shaped(*kw, {kv.d})) raise(PyExc_ValueError, "k_weight must be [head_dim]");
    if (fp8 != (a[13] != Py_None) || fp8 != (a[14] != Py_None))
      raise(PyExc_ValueError, "k_scale and v_scale go with (and only with) E4M3 caches");
    const at::Tensor* ks = c.optional(a[13], "k_scale", at::kFloat);
    const at::Tensor* vs = c.optional(a[14], "v_scale", at::kFloat);
    if (fp8 && (!shaped(*ks, {kv.hkv}) || !shaped(*vs, {kv.hkv})))
      raise(PyExc_ValueError, "k_scale/v_scale must be [num_kv_heads]");
    const int interleaved = PyObject_IsTrue(a[12]);
    if (interleaved < 0) throw Raised{};
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(c.device()));
    call(lib.qk_norm_rope_append, at_(out), at_(q), at_(k), at_(v), c.rows(out, "q_out"), c.rows(q, "q"),
         c.rows(k, "k"), c.rows(v, "v"),
         to<int32_t>(pos), to<int64_t>(slots), narrow(q.size(0), "num_tokens"), to<float>(cs),
         narrow(cs.size(0), "max_position"), narrow(cs.size(1), "rotary_dim"), interleaved, at_(qw), at_(kw),
         static_cast<float>(number(a[11])), at_(kv.k), at_(kv.v), to<float>(ks), to<float>(vs), kv.nb, kv.bs,
         narrow(q.size(1), "num_heads"), kv.hkv, kv.d, kv.type, c.stream(a[15]));
  });
}

// out, q, k_cache, v_cache, block_tables, context_lens, query_start, parents,
// max_query_len, scale, workspace, stream
PyObject* decode_tree(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("decode_tree", n, 12, [&] {
    Call c;
    const Cache kv = caches(c, a[2], a[3]);
    const at::ScalarType dt = kv.k.scalar_type();
    const at::Tensor& out = c.tensor(a[0], "out", dt);
    const at::Tensor& q = c.tensor(a[1], "q", dt);
    if (q.dim() != 3 || q.size(2) != kv.d || out.sizes() != q.sizes())
      raise(PyExc_ValueError, "q/out/cache shape mismatch");
    const at::Tensor& tables = c.tensor(a[4], "block_tables", at::kInt);
    const at::Tensor& lens = c.tensor(a[5], "context_lens", at::kInt);
    const at::Tensor& start = c.tensor(a[6], "query_start", at::kInt);
    if (lens.dim() != 1 || tables.dim() != 2 || tables.size(0) != lens.size(0) || !shaped(start, {lens.size(0) + 1}))
      raise(PyExc_ValueError, "block_tables must be [S, max_blocks], query_start [S + 1]");
    const at::Tensor* parents = c.optional(a[7], "parents", at::kInt);
    if (parents && !shaped(*parents, {q.size(0)})) raise(PyExc_ValueError, "parents must be [total_q]");
    if (a[10] == Py_None) raise(PyExc_ValueError, "pa_decode_tree needs a workspace");
    const at::Tensor& ws = c.tensor(a[10], "workspace");
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(c.device()));
    call(lib.decode_tree, at_(out), at_(q), at_(kv.k), at_(kv.v), to<int32_t>(tables), to<int32_t>(lens),
         to<int32_t>(start), to<int32_t>(parents), narrow(lens.size(0), "num_seqs"),
         narrow(q.size(0), "total_q"), narrow(q.size(1), "num_heads"), kv.hkv, kv.d, kv.bs, kv.nb,
         narrow(tables.size(1), "max_blocks_per_seq"), narrow(whole(a[8]), "max_query_len"),
         static_cast<float>(number(a[9])), at_(ws), ws.nbytes(), kv.type, c.stream(a[11]));
  });
}

// out_tokens, out_path, out_len, target_probs, draft_probs, draft_tokens, parents,
// query_start, u_accept, u_sample, stream
PyObject* verify_draft(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("verify_draft", n, 11, [&] {
    Call c;
    const at::Tensor& out = c.tensor(a[0], "out_tokens", at::kInt);
    const at::Tensor& path = c.tensor(a[1], "out_path", at::kInt);
    if (out.dim() != 2 || path.sizes() != out.sizes())
      raise(PyExc_ValueError, "out_tokens and out_path must be [S, max_query_len]");
    const int64_t s = out.size(0);
    const at::Tensor& len = c.tensor(a[2], "out_len", at::kInt);
    const at::Tensor& target = c.tensor(a[3], "target_probs", at::kFloat, false);
    if (target.dim() != 2) raise(PyExc_ValueError, "target_probs must be [total_q, vocab_size]");
    const int64_t rows = target.size(0), vocab = target.size(1);
    const at::Tensor& start = c.tensor(a[7], "query_start", at::kInt);
    const at::Tensor& us = c.tensor(a[9], "u_sample", at::kFloat);
    if (!shaped(len, {s}) || !shaped(start, {s + 1}) || !shaped(us, {s}))
      raise(PyExc_ValueError, "out_len and u_sample must be [S], query_start [S + 1]");
    const at::Tensor& tokens = c.tensor(a[5], "draft_tokens", at::kInt);
    const at::Tensor& ua = c.tensor(a[8], "u_accept", at::kFloat);
    const at::Tensor* parents = c.optional(a[6], "parents", at::kInt);
    if (!shaped(tokens, {rows})) raise(PyExc_ValueError, "draft_tokens must be [total_q]");
    if (!shaped(ua, {rows})) raise(PyExc_ValueError, "u_accept must be [total_q]");
    if (parents && !shaped(*parents, {rows})) raise(PyExc_ValueError, "parents must be [total_q]");
    auto stride = [&](const at::Tensor& t, const char* name) {
      if (!shaped(t, {rows, vocab}) || (vocab > 1 && t.numel() != 0 && t.stride(1) != 1))
        raise(PyExc_ValueError, "%s must be [total_q, vocab_size] with dense rows", name);
      return rows > 1 ? t.stride(0) : vocab;
    };
    const at::Tensor* draft = a[4] == Py_None ? nullptr : &c.tensor(a[4], "draft_probs", at::kFloat, false);
    const int64_t ts = stride(target, "target_probs"), ds = draft ? stride(*draft, "draft_probs") : 0;
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(c.device()));
    call(lib.verify_draft, to<int32_t>(out), to<int32_t>(path), to<int32_t>(len), to<float>(target), ts,
         to<float>(draft), ds, to<int32_t>(tokens), to<int32_t>(parents), to<int32_t>(start),
         to<float>(ua), to<float>(us), narrow(s, "num_seqs"), narrow(rows, "total_q"),
         narrow(vocab, "vocab_size"), narrow(out.size(1), "max_query_len"), c.stream(a[10]));
  });
}

// k_cache, v_cache, block_tables, context_lens, query_start, path, path_len, stream
PyObject* kv_accept(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("kv_accept", n, 8, [&] {
    Call c;
    const Cache kv = caches(c, a[0], a[1]);
    const at::Tensor& tables = c.tensor(a[2], "block_tables", at::kInt);
    const at::Tensor& lens = c.tensor(a[3], "context_lens", at::kInt);
    const at::Tensor& start = c.tensor(a[4], "query_start", at::kInt);
    if (lens.dim() != 1 || tables.dim() != 2 || tables.size(0) != lens.size(0) || !shaped(start, {lens.size(0) + 1}))
      raise(PyExc_ValueError, "block_tables must be [S, max_blocks], query_start [S + 1]");
    const at::Tensor& path = c.tensor(a[5], "path", at::kInt);
    const at::Tensor& len = c.tensor(a[6], "path_len", at::kInt);
    if (path.dim() != 2 || path.size(0) != lens.size(0) || !shaped(len, {lens.size(0)}))
      raise(PyExc_ValueError, "path must be [S, max_path_len], path_len [S]");
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(c.device()));
    call(lib.kv_accept, at_(kv.k), at_(kv.v), to<int32_t>(tables), to<int32_t>(lens), to<int32_t>(start),
         to<int32_t>(path), to<int32_t>(len), narrow(lens.size(0), "num_seqs"),
         narrow(path.size(1), "max_path_len"), kv.nb, kv.bs,
         narrow(tables.size(1), "max_blocks_per_seq"), kv.hkv, kv.d, kv.type, c.stream(a[7]));
  });
}

// bind(addresses by C name, PagedAttentionError)
PyObject* bind(PyObject*, PyObject* args) {
  PyObject *table, *cls;
  if (!PyArg_ParseTuple(args, "O!O", &PyDict_Type, &table, &cls)) return nullptr;
  auto take = [&](const char* name, auto& fn) {
    PyObject* v = PyDict_GetItemString(table, name);
    if (!v) {
      PyErr_Format(PyExc_KeyError, "%s", name);
      return false;
    }
    const unsigned long long at = PyLong_AsUnsignedLongLong(v);
    if (PyErr_Occurred()) return false;
    fn = reinterpret_cast<std::remove_reference_t<decltype(fn)>>(static_cast<uintptr_t>(at));
    return true;
  };
  if (!take("pa_kv_append", lib.kv_append) || !take("pa_kv_append_fp8", lib.kv_append_fp8) ||
      !take("pa_qk_norm_rope_append", lib.qk_norm_rope_append) || !take("pa_decode_tree", lib.decode_tree) ||
      !take("pa_verify_draft", lib.verify_draft) || !take("pa_kv_accept", lib.kv_accept) ||
      !take("pa_last_error", lib.last_error))
    return nullptr;
  Py_INCREF(cls);
  Py_XSETREF(error_class, cls);
  Py_RETURN_NONE;
}

template <typename F>
PyCFunction method(F f) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)); }

PyMethodDef methods[] = {
    {"bind", bind, METH_VARARGS, nullptr},
    {"kv_append", method(kv_append), METH_FASTCALL, nullptr},
    {"kv_append_fp8", method(kv_append_fp8), METH_FASTCALL, nullptr},
    {"qk_norm_rope_append", method(qk_norm_rope_append), METH_FASTCALL, nullptr},
    {"decode_tree", method(decode_tree), METH_FASTCALL, nullptr},
    {"verify_draft", method(verify_draft), METH_FASTCALL, nullptr},
    {"kv_accept", method(kv_accept), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pa_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// (built_for: the torch and Python that this was built for, which the package checks)
PyMODINIT_FUNC PyInit__pa_torch(void) {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "built_for", PA_BUILT_FOR) != 0) Py_CLEAR(m);
  return m;
}
