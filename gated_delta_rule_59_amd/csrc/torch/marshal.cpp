// Tensor marshalling of the calls beside KDA (kda_kv_append and those declared after it) for binding.py:
// checks the tensors, fills the argument structs of include/kda.h, allocates what the caller left out, and
// calls the library on the tensors' device. No computation. It is C++ because these calls can be
// shorter than their own marshalling: a decode step's append runs 5 us on the GPU, and the same
// checks written in Python took 17 us of the host.
//
// bind() takes the addresses of the functions that binding.py has loaded from libkda.so, so this
// module links against torch only.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/core/DeviceGuard.h>
#include <c10/core/StreamGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <optional>
#include <type_traits>

#include "kda.h"

namespace {

struct Library {
  decltype(&kda_kv_append) append;
  decltype(&kda_paged_decode) decode;
  decltype(&kda_paged_decode_workspace_bytes) decode_bytes;
  decltype(&kda_verify_drafts) verify;
  decltype(&kda_verify_drafts_workspace_bytes) verify_bytes;
  decltype(&kda_lin_chunk_fwd) lin_chunk;
  decltype(&kda_lin_chunk_fwd_workspace_bytes) lin_chunk_bytes;
  decltype(&kda_lin_decode_step) lin_step;
  decltype(&kda_lin_decode_multi) lin_multi;
  decltype(&kda_page_plan) plan;
  decltype(&kda_adjust_logits) logits;
  decltype(&kda_adjust_logits_workspace_bytes) logits_bytes;
  decltype(&kda_last_error) last_error;
  PyObject* error;  // binding.KDAError
} lib{};

[[noreturn]] void raise(PyObject* type, const char* fmt, va_list ap) {
  char buf[512];
  std::vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  PyErr_SetString(type, buf);
  throw python_error();
}
[[noreturn]] __attribute__((format(printf, 1, 2))) void type_error(const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  raise(PyExc_TypeError, fmt, ap);
}
[[noreturn]] __attribute__((format(printf, 1, 2))) void value_error(const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  raise(PyExc_ValueError, fmt, ap);
}

typedef at::Tensor const* Opt;  // nullptr: None

Opt optional(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) type_error("%s must be a torch.Tensor", name);
  return &THPVariable_Unpack(o);
}
const at::Tensor& tensor(PyObject* o, const char* name) {
  Opt t = optional(o, name);
  if (!t) type_error("%s must be a torch.Tensor", name);
  return *t;
}

// The device of a call: its first tensor's, a GPU, and every other tensor's.
struct On {
  c10::Device device;
  explicit On(const at::Tensor& t) : device(t.device()) {
    if (!device.is_cuda()) value_error("tensors must be on the GPU");
  }
  void also(const char* name, Opt t) const {
    if (t && t->device() != device)
      value_error("%s must be on %s", name, device.str().c_str());
  }
};

void of_type(const char* name, const at::Tensor& t, at::ScalarType type) {
  if (t.scalar_type() != type) type_error("%s must be %s", name, c10::toString(type));
}

// Given (nullptr is skipped), a tensor is contiguous and of this device, type and shape.
void plain(const On& on, const char* name, Opt t, at::ScalarType type, at::IntArrayRef shape) {
  if (!t) return;
  on.also(name, t);
  of_type(name, *t, type);
  if (t->sizes() != shape || !t->is_contiguous())
    value_error("%s must be contiguous of shape %s", name, c10::str(shape).c_str());
}

int to_int(const char* name, int64_t x) {
  if (x > INT32_MAX || x < INT32_MIN) value_error("%s is too large", name);
  return (int)x;
}

kda_dtype act_type(const at::Tensor& t, const char* name) {
  if (t.scalar_type() == at::kFloat) return KDA_F32;
  if (t.scalar_type() == at::kBFloat16) return KDA_BF16;
  type_error("%s must be float32 or bfloat16", name);
}

at::ScalarType out_type(Opt given, PyObject* dtype) {
  if (!given && !THPDtype_Check(dtype)) type_error("out_dtype must be a torch.dtype");
  const at::ScalarType t = given ? given->scalar_type() : reinterpret_cast<THPDtype*>(dtype)->scalar_type;
  if (t != at::kFloat && t != at::kBFloat16) type_error("the output must be float32 or bfloat16");
  return t;
}

// Token and head strides of a [lead0, lead1, heads, d] view whose tokens lie evenly apart, or of a [lead0,
// heads, d] one (dim 3).
void heads(const On& on, const char* name, const at::Tensor& t, at::ScalarType type, int64_t lead0,
           int64_t lead1, int64_t d, int64_t* token, int64_t* head, int dim = 4) {
  on.also(name, &t);
  of_type(name, t, type);
  if (t.dim() != dim || t.size(0) != lead0 || (dim == 4 && t.size(1) != lead1) || t.size(dim - 1) != d) {
    if (dim == 3) value_error("%s must be of shape [%lld, heads, %lld]", name, (long long)lead0, (long long)d);
    value_error("%s must be of shape [%lld, %lld, heads, %lld]", name, (long long)lead0,
                            (long long)lead1, (long long)d);
  }
  if (dim == 3) lead1 = 1;
  const int64_t H = t.size(dim - 2);
  *token = H * d;
  *head = d;
  if (t.numel() == 0) return;
  const auto s = t.strides();
  if ((s[dim - 1] != 1 && d > 1) || (lead0 > 1 && lead1 > 1 && s[0] != lead1 * s[1]))
    value_error("%s must have contiguous channels and evenly spaced tokens", name);
  if (lead1 > 1) *token = s[1];
  else if (lead0 > 1) *token = s[0];
  if (H > 1) *head = s[dim - 2];
}

void page_cache(const On& on, const at::Tensor& k, const at::Tensor& v, const at::Tensor& table, Opt k_scale,
                Opt v_scale, int64_t n_seq, int64_t Hkv, int64_t d, kda_page_cache* c) {
  on.also("k_cache", &k);
  on.also("v_cache", &v);
  const auto type = k.scalar_type();
  if (v.scalar_type() != type || (type != at::kFloat && type != at::kBFloat16 && type != at::kFloat8_e4m3fn))
    type_error("k_cache and v_cache must both be float32, bfloat16 or float8_e4m3fn");
  if (k.dim() != 4 || v.sizes() != k.sizes() || k.size(2) != Hkv || k.size(3) != d)
    value_error("k_cache and v_cache must be of shape [pages, page_size, %lld, %lld]",
                            (long long)Hkv, (long long)d);
  const auto ks = k.strides(), vs = v.strides();
  if (ks[3] != 1 || vs[3] != 1)
    value_error("k_cache and v_cache must have contiguous channels");
  on.also("block_table", &table);
  of_type("block_table", table, at::kInt);
  if (table.dim() != 2 || table.size(0) != n_seq || (table.size(1) > 1 && table.stride(1) != 1))
    value_error("block_table must be of shape [%lld, max_pages], pages side by side",
                            (long long)n_seq);
  plain(on, "k_scale", k_scale, at::kFloat, {Hkv});
  plain(on, "v_scale", v_scale, at::kFloat, {Hkv});
  c->k = k.data_ptr();
  c->v = v.data_ptr();
  c->dtype = type == at::kFloat ? KDA_F32 : type == at::kBFloat16 ? KDA_BF16 : KDA_F8E4M3;
  c->num_pages = to_int("k_cache", k.size(0));
  c->page_size = to_int("k_cache", k.size(1));
  c->k_page_stride = ks[0], c->k_token_stride = ks[1], c->k_head_stride = ks[2];
  c->v_page_stride = vs[0], c->v_token_stride = vs[1], c->v_head_stride = vs[2];
  c->block_table = static_cast<const int32_t*>(table.data_ptr());
  c->table_stride = table.stride(0);
  c->max_pages = to_int("block_table", table.size(1));
  c->k_scale = k_scale ? static_cast<const float*>(k_scale->data_ptr()) : nullptr;
  c->v_scale = v_scale ? static_cast<const float*>(v_scale->data_ptr()) : nullptr;
}

// The stream of a call: the one given (a torch.cuda.Stream), or the device's current one. What is
// allocated here for a given stream comes from that stream's memory: memory of the current stream may
// have been freed while work queued there still uses it, and only that stream waits for that work.
// The other way round, a result's memory is not handed out again before the current stream, where
// the caller is, is done with it.
struct Stream {
  std::optional<c10::Stream> given, current;
  void* raw;
  Stream(PyObject* o, const On& on) {
    const c10::hip::HIPStream now = c10::hip::getCurrentHIPStream(on.device.index());
    raw = now.stream();
    if (o == Py_None) return;
    if (attribute(o, "device_index") != on.device.index())
      value_error("the stream must be of %s", on.device.str().c_str());
    void* const own = reinterpret_cast<void*>(attribute(o, "cuda_stream"));
    if (own == raw) return;
    raw = own;
    given = c10::Stream(c10::Stream::UNSAFE, on.device, attribute(o, "stream_id"));
    current = c10::Stream(c10::Stream::UNSAFE, on.device, now.id());
  }
  static int64_t attribute(PyObject* o, const char* name) {
    PyObject* a = PyObject_GetAttrString(o, name);
    if (!a) throw python_error();
    const int64_t x = PyLong_AsLongLong(a);
    Py_DECREF(a);
    if (x == -1 && PyErr_Occurred()) throw python_error();
    return x;
  }
  at::Tensor scratch(at::IntArrayRef shape, at::ScalarType type, const On& on) const {
    const c10::OptionalStreamGuard guard(given);
    return at::empty(shape, at::TensorOptions().dtype(type).device(on.device));
  }
  at::Tensor empty(at::IntArrayRef shape, at::ScalarType type, const On& on) const {
    at::Tensor t = scratch(shape, type, on);
    if (given && t.numel()) t.record_stream(*current);
    return t;
  }
};

// The caller's workspace, or a new one of the size that the library asks for (kept in `own`).
template <typename Args>
void workspace(Args* a, Opt given, size_t (*bytes)(const Args*), const Stream& s, const On& on,
               at::Tensor* own) {
  if (given) {
    on.also("workspace", given);
    if (!given->is_contiguous()) value_error("workspace must be contiguous");
    a->workspace = given->data_ptr();
    a->workspace_bytes = given->numel() * given->element_size();
    return;
  }
  const size_t n = bytes(a);
  if (n == 0 || n == SIZE_MAX) return;  // if invalid, the call itself says what is wrong
  *own = s.scratch({(int64_t)n}, at::kByte, on);
  a->workspace = own->data_ptr();
  a->workspace_bytes = n;
}

void check(kda_status s) {
  if (s == KDA_OK) return;
  PyObject* e = PyObject_CallFunction(lib.error, "is", (int)s, lib.last_error());
  if (e) {
    PyErr_SetObject(lib.error, e);
    Py_DECREF(e);
  }
  throw python_error();
}

const int32_t* ints(Opt t) { return t ? static_cast<const int32_t*>(t->data_ptr()) : nullptr; }
int32_t* out_ints(const at::Tensor& t) { return static_cast<int32_t*>(t.data_ptr()); }

void arguments(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) type_error("%d arguments expected", (int)want);
}
bool truth(PyObject* o) {
  const int x = PyObject_IsTrue(o);
  if (x < 0) throw python_error();
  return x;
}
int number(PyObject* o, const char* name) {
  const long long x = PyLong_AsLongLong(o);
  if (x == -1 && PyErr_Occurred()) throw python_error();
  return to_int(name, x);
}

// bind(addresses of the library's functions ..., KDAError)
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  constexpr int F = 13;  // functions of Library
  arguments(n, F + 1);
  void* p[F];
  for (int i = 0; i < F; ++i) {
    p[i] = PyLong_AsVoidPtr(args[i]);
    if (!p[i] && PyErr_Occurred()) throw python_error();
  }
  Py_INCREF(args[F]);
  Py_XDECREF(lib.error);
  int i = 0;
  const auto next = [&](auto& f) { f = reinterpret_cast<std::remove_reference_t<decltype(f)>>(p[i++]); };
  next(lib.append), next(lib.decode), next(lib.decode_bytes), next(lib.verify), next(lib.verify_bytes);
  next(lib.lin_chunk), next(lib.lin_chunk_bytes), next(lib.lin_step), next(lib.lin_multi);
  next(lib.plan), next(lib.logits), next(lib.logits_bytes), next(lib.last_error);
  lib.error = args[F];
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// kv_append(k, v, k_cache, v_cache, block_table, start, q, q_out, inv_freq, interleaved, cu_seqlens,
//           k_scale, v_scale, stream) -> q_out or None
PyObject* kv_append(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  arguments(nargs, 14);
  const at::Tensor &k = tensor(args[0], "k"), &v = tensor(args[1], "v"), &k_cache = tensor(args[2], "k_cache"),
                   &v_cache = tensor(args[3], "v_cache"), &table = tensor(args[4], "block_table"),
                   &start = tensor(args[5], "start");
  Opt q = optional(args[6], "q"), q_out = optional(args[7], "q_out"), inv_freq = optional(args[8], "inv_freq"),
      cu = optional(args[10], "cu_seqlens"), k_scale = optional(args[11], "k_scale"),
      v_scale = optional(args[12], "v_scale");
  const On on(k);
  if (k.dim() != 4 || v.sizes() != k.sizes())
    value_error("k and v must both be of shape [B, T, Hkv, d]");
  const int64_t B = k.size(0), T = k.size(1), Hkv = k.size(2), d = k.size(3);
  const int64_t n_seq = cu ? cu->numel() - 1 : B, rot = inv_freq ? 2 * inv_freq->numel() : 0;
  kda_kv_append_args a{};
  a.B = to_int("B", B), a.T = to_int("T", T), a.Hkv = to_int("Hkv", Hkv), a.d = to_int("d", d);
  a.act_dtype = act_type(k, "k");
  heads(on, "k", k, k.scalar_type(), B, T, d, &a.k_token_stride, &a.k_head_stride);
  heads(on, "v", v, k.scalar_type(), B, T, d, &a.v_token_stride, &a.v_head_stride);
  plain(on, "start", &start, at::kInt, {n_seq});
  plain(on, "cu_seqlens", cu, at::kInt, {n_seq + 1});
  plain(on, "inv_freq", inv_freq, at::kFloat, {rot / 2});
  page_cache(on, k_cache, v_cache, table, k_scale, v_scale, n_seq, Hkv, d, &a.cache);
  a.k = k.data_ptr();
  a.v = v.data_ptr();
  a.start = ints(&start);
  a.inv_freq = rot ? static_cast<const float*>(inv_freq->data_ptr()) : nullptr;
  a.rot = to_int("rot", rot);
  a.flags = truth(args[9]) ? KDA_APPEND_PAIRS : 0;
  a.cu_seqlens = ints(cu);
  a.N = cu ? to_int("N", n_seq) : 0;
  const Stream stream(args[13], on);
  at::Tensor own;
  if (q) {
    heads(on, "q", *q, k.scalar_type(), B, T, d, &a.q_token_stride, &a.q_head_stride);
    a.Hq = to_int("Hq", q->size(2));
    if (q_out) {
      plain(on, "q_out", q_out, q->scalar_type(), q->sizes());
    } else {
      own = stream.empty(q->sizes(), q->scalar_type(), on);
      q_out = &own;
    }
    a.q = q->data_ptr();
    a.q_out = q_out->data_ptr();
  } else if (q_out) {
    value_error("q_out needs q");
  }
  const c10::DeviceGuard guard(on.device);
  check(lib.append(&a, stream.raw));
  if (!q) Py_RETURN_NONE;
  return own.defined() ? THPVariable_Wrap(own) : Py_NewRef(args[7]);
  END_HANDLE_TH_ERRORS
}

// paged_decode(q, k_cache, v_cache, block_table, seq_lens, scale, window, max_len, k_scale, v_scale, o,
//              lse, out_dtype, workspace, stream) -> o; with workspace False: the workspace's bytes
PyObject* paged_decode(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  arguments(nargs, 15);
  const at::Tensor &q = tensor(args[0], "q"), &k_cache = tensor(args[1], "k_cache"),
                   &v_cache = tensor(args[2], "v_cache"), &table = tensor(args[3], "block_table"),
                   &lens = tensor(args[4], "seq_lens");
  Opt k_scale = optional(args[8], "k_scale"), v_scale = optional(args[9], "v_scale"),
      o = optional(args[10], "o"), lse = optional(args[11], "lse");
  const bool query = args[13] == Py_False;
  Opt given = query ? nullptr : optional(args[13], "workspace");
  const On on(q);
  if (q.dim() != 4 || k_cache.dim() != 4)
    value_error("q must be of shape [N, m, Hq, d], k_cache and v_cache of shape "
                            "[pages, page_size, Hkv, d]");
  const int64_t N = q.size(0), m = q.size(1), Hq = q.size(2), d = q.size(3), Hkv = k_cache.size(2);
  const at::ScalarType out = out_type(o, args[12]);
  kda_paged_decode_args a{};
  a.N = to_int("N", N), a.m = to_int("m", m), a.Hq = to_int("Hq", Hq), a.Hkv = to_int("Hkv", Hkv);
  a.d = to_int("d", d);
  a.act_dtype = act_type(q, "q");
  a.out_dtype = out == at::kFloat ? KDA_F32 : KDA_BF16;
  heads(on, "q", q, q.scalar_type(), N, m, d, &a.q_token_stride, &a.q_head_stride);
  page_cache(on, k_cache, v_cache, table, k_scale, v_scale, N, Hkv, d, &a.cache);
  plain(on, "seq_lens", &lens, at::kInt, {N});
  plain(on, "o", o, out, q.sizes());
  plain(on, "lse", lse, at::kFloat, q.sizes().slice(0, 3));
  a.q = q.data_ptr();
  a.seq_lens = ints(&lens);
  a.scale = args[5] == Py_None ? 1.f / std::sqrt((float)std::max<int64_t>(d, 1)) : (float)PyFloat_AsDouble(args[5]);
  if (PyErr_Occurred()) throw python_error();
  a.window = number(args[6], "window");
  a.max_len = args[7] == Py_None
                  ? (int)std::min<int64_t>((int64_t)a.cache.max_pages * a.cache.page_size, 1 << 30)
                  : number(args[7], "max_len");
  if (query) {
    const size_t bytes = lib.decode_bytes(&a);
    if (bytes == SIZE_MAX) check(KDA_ERR_BAD_SHAPE);
    return PyLong_FromSize_t(bytes);
  }
  const Stream stream(args[14], on);
  at::Tensor own, scratch;
  if (!o) own = stream.empty(q.sizes(), out, on);
  a.o = o ? o->data_ptr() : own.data_ptr();
  a.lse = lse ? static_cast<float*>(lse->data_ptr()) : nullptr;
  workspace(&a, given, lib.decode_bytes, stream, on, &scratch);
  const c10::DeviceGuard guard(on.device);
  check(lib.decode(&a, stream.raw));
  return o ? Py_NewRef(args[10]) : THPVariable_Wrap(own);
  END_HANDLE_TH_ERRORS
}

// Heads, dims, types, strides and decays of linear attention: q, k [lead0, lead1, Hk, dk], v [lead0, lead1,
// H, dv], g [lead0, lead1, H] or [H]; or all of one token, without lead1.
template <typename Args>
void linear(const On& on, const at::Tensor& q, const at::Tensor& k, const at::Tensor& v, const at::Tensor& g,
            PyObject* scale, Args* a) {
  const int dim = (int)q.dim();
  const int64_t lead0 = q.size(0), lead1 = dim == 3 ? 1 : q.size(1), dk = q.size(dim - 1);
  const int64_t Hk = q.size(dim - 2), H = v.size(dim - 2), dv = v.size(dim - 1);
  a->act_dtype = act_type(q, "q");
  heads(on, "q", q, q.scalar_type(), lead0, lead1, dk, &a->q_token_stride, &a->q_head_stride, dim);
  heads(on, "k", k, q.scalar_type(), lead0, lead1, dk, &a->k_token_stride, &a->k_head_stride, dim);
  heads(on, "v", v, q.scalar_type(), lead0, lead1, dv, &a->v_token_stride, &a->v_head_stride, dim);
  if (k.size(dim - 2) != Hk) value_error("q and k must have the same heads");
  a->gate_dtype = act_type(g, "g");
  const bool fixed = g.dim() == 1;
  const int64_t three[] = {lead0, lead1, H}, two[] = {lead0, H};
  plain(on, "g", &g, g.scalar_type(),
        fixed ? at::IntArrayRef(two + 1, two + 2) : dim == 3 ? at::IntArrayRef(two) : at::IntArrayRef(three));
  a->Hk = to_int("Hk", Hk), a->H = to_int("H", H);
  a->dk = to_int("dk", dk), a->dv = to_int("dv", dv);
  a->q = q.data_ptr(), a->k = k.data_ptr(), a->v = v.data_ptr(), a->g = g.data_ptr();
  a->scale = (float)PyFloat_AsDouble(scale);
  if (PyErr_Occurred()) throw python_error();
  a->flags = fixed ? KDA_LIN_FIXED_DECAY : 0;
}

// lin_chunk_fwd(q, k, v, g, S0, cu_seqlens, scale, o, S_T, want_state, out_dtype, workspace, stream)
//   -> (o, S_T or None); with workspace False: the workspace's bytes
PyObject* lin_chunk_fwd(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  arguments(nargs, 13);
  const at::Tensor &q = tensor(args[0], "q"), &k = tensor(args[1], "k"), &v = tensor(args[2], "v"),
                   &g = tensor(args[3], "g");
  Opt S0 = optional(args[4], "S0"), cu = optional(args[5], "cu_seqlens"), o = optional(args[7], "o"),
      S_T = optional(args[8], "S_T");
  const bool query = args[11] == Py_False, want = S_T || truth(args[9]);
  Opt given = query ? nullptr : optional(args[11], "workspace");
  const On on(q);
  if (q.dim() != 4 || v.dim() != 4)
    value_error("q and k must be of shape [B, T, Hk, dk], v of shape [B, T, H, dv]");
  const at::ScalarType out = out_type(o, args[10]);
  kda_lin_chunk_args a{};
  linear(on, q, k, v, g, args[6], &a);
  const int64_t n_seq = cu ? cu->numel() - 1 : q.size(0);
  const int64_t state[] = {n_seq, v.size(2), q.size(3), v.size(3)};
  plain(on, "cu_seqlens", cu, at::kInt, {n_seq + 1});
  plain(on, "S0", S0, at::kFloat, state);
  plain(on, "S_T", S_T, at::kFloat, state);
  plain(on, "o", o, out, v.sizes());
  a.B = to_int("B", q.size(0)), a.T = to_int("T", q.size(1));
  a.cu_seqlens = ints(cu);
  a.N = cu ? to_int("N", n_seq) : 0;
  a.out_dtype = out == at::kFloat ? KDA_F32 : KDA_BF16;
  if (query) {
    const size_t bytes = lib.lin_chunk_bytes(&a);
    if (bytes == SIZE_MAX) check(KDA_ERR_BAD_SHAPE);
    return PyLong_FromSize_t(bytes);
  }
  const Stream stream(args[12], on);
  at::Tensor own_o, own_state, scratch;
  if (!o) own_o = stream.empty(v.sizes(), out, on);
  if (!S_T && want) own_state = stream.empty(state, at::kFloat, on);
  a.S0 = S0 ? static_cast<const float*>(S0->data_ptr()) : nullptr;
  a.o = o ? o->data_ptr() : own_o.data_ptr();
  a.S_T = S_T ? static_cast<float*>(S_T->data_ptr()) : want ? static_cast<float*>(own_state.data_ptr()) : nullptr;
  workspace(&a, given, lib.lin_chunk_bytes, stream, on, &scratch);
  const c10::DeviceGuard guard(on.device);
  check(lib.lin_chunk(&a, stream.raw));
  PyObject* r = PyTuple_New(2);
  if (!r) return nullptr;
  PyTuple_SET_ITEM(r, 0, o ? Py_NewRef(args[7]) : THPVariable_Wrap(own_o));
  PyTuple_SET_ITEM(r, 1, S_T ? Py_NewRef(args[8]) : want ? THPVariable_Wrap(own_state) : Py_NewRef(Py_None));
  return r;
  END_HANDLE_TH_ERRORS
}

// lin_decode(q, k, v, g, S, accept, scale, o, want_output, out_dtype, step, stream) -> o or None
PyObject* lin_decode(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  arguments(nargs, 12);
  const at::Tensor &q = tensor(args[0], "q"), &k = tensor(args[1], "k"), &v = tensor(args[2], "v"),
                   &g = tensor(args[3], "g"), &S = tensor(args[4], "S");
  Opt accept = optional(args[5], "accept"), o = optional(args[7], "o");
  const bool want = o || truth(args[8]), step = truth(args[10]);
  const On on(q);
  const int64_t dim = step ? 3 : 4;
  if (q.dim() != dim || k.dim() != dim || v.dim() != dim || (g.dim() != 1 && g.dim() != dim - 1)) {
    if (step)
      value_error("q and k must be of shape [N, Hk, dk], v of shape [N, H, dv], g of shape [N, H] or [H]");
    value_error("q and k must be of shape [N, m, Hk, dk], v of shape [N, m, H, dv], g of shape [N, m, H] or [H]");
  }
  const at::ScalarType out = out_type(o, args[9]);
  kda_lin_decode_args a{};
  linear(on, q, k, v, g, args[6], &a);
  const int64_t N = q.size(0);
  plain(on, "S", &S, at::kFloat, {N, a.H, a.dk, a.dv});
  plain(on, "accept", accept, at::kInt, {N});
  plain(on, "o", o, out, v.sizes());
  a.N = to_int("N", N), a.m = step ? 1 : to_int("m", q.size(1));
  a.out_dtype = out == at::kFloat ? KDA_F32 : KDA_BF16;
  const Stream stream(args[11], on);
  at::Tensor own;
  if (!o && want) own = stream.empty(v.sizes(), out, on);
  a.S = static_cast<float*>(S.data_ptr());
  a.o = o ? o->data_ptr() : want ? own.data_ptr() : nullptr;
  a.accept = ints(accept);
  const c10::DeviceGuard guard(on.device);
  check((step ? lib.lin_step : lib.lin_multi)(&a, stream.raw));
  return o ? Py_NewRef(args[7]) : want ? THPVariable_Wrap(own) : Py_NewRef(Py_None);
  END_HANDLE_TH_ERRORS
}

// page_plan(block_table, held, lens, new_lens, free_pages, ring, page_size, max_tokens, held_out, ring_out,
//           seq_lens, cu_seqlens, slots, positions, stream)
//   -> (held, ring, seq_lens, cu_seqlens, slots, positions)
PyObject* page_plan(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  arguments(nargs, 15);
  const at::Tensor &table = tensor(args[0], "block_table"), &held = tensor(args[1], "held"),
                   &lens = tensor(args[2], "lens"), &fresh = tensor(args[3], "new_lens"),
                   &pages = tensor(args[4], "free_pages"), &ring = tensor(args[5], "ring");
  const On on(table);
  of_type("block_table", table, at::kInt);
  if (table.dim() != 2 || (table.size(1) > 1 && table.stride(1) != 1))
    value_error("block_table must be of shape [N, max_pages], pages side by side");
  const int64_t N = table.size(0);
  plain(on, "held", &held, at::kInt, {N});
  plain(on, "lens", &lens, at::kInt, {N});
  plain(on, "new_lens", &fresh, at::kInt, {N});
  plain(on, "free_pages", &pages, at::kInt, {pages.numel()});
  plain(on, "ring", &ring, at::kInt, {2});
  kda_page_plan_args a{};
  a.N = to_int("N", N);
  a.page_size = number(args[6], "page_size");
  a.max_tokens = number(args[7], "max_tokens");
  a.max_pages = to_int("block_table", table.size(1));
  a.free_capacity = to_int("free_pages", pages.numel());
  const Stream stream(args[14], on);
  static const char* const names[] = {"held_out", "ring_out", "seq_lens", "cu_seqlens", "slots", "positions"};
  const int64_t sizes[] = {N, 2, N, N + 1, a.max_tokens, a.max_tokens};
  // What is not given: parts of one allocation, each 256-byte aligned (six of their own take the host 2 us more).
  at::Tensor own[6], all;
  void* to[6];
  int64_t begin[6], bytes = 0;
  for (int i = 0; i < 6; ++i) {
    Opt x = optional(args[8 + i], names[i]);
    plain(on, names[i], x, i == 4 ? at::kLong : at::kInt, {sizes[i]});
    to[i] = x ? x->data_ptr() : nullptr;
    begin[i] = x ? -1 : bytes;
    if (!x) bytes += (std::max<int64_t>(sizes[i], 0) * (i == 4 ? 8 : 4) + 255) / 256 * 256;
  }
  if (bytes) all = stream.empty({bytes}, at::kByte, on);
  for (int i = 0; i < 6; ++i) {
    if (begin[i] < 0) continue;
    own[i] = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all.storage()), all.key_set(),
                                                      c10::scalarTypeToTypeMeta(i == 4 ? at::kLong : at::kInt));
    own[i].unsafeGetTensorImpl()->set_sizes_contiguous({std::max<int64_t>(sizes[i], 0)});
    own[i].unsafeGetTensorImpl()->set_storage_offset(begin[i] / (i == 4 ? 8 : 4));
    to[i] = static_cast<char*>(all.data_ptr()) + begin[i];
  }
  a.block_table = out_ints(table);
  a.table_stride = N > 1 ? table.stride(0) : std::max<int64_t>(table.size(1), 1);
  a.held = ints(&held), a.lens = ints(&lens), a.new_lens = ints(&fresh);
  a.free_pages = out_ints(pages), a.ring = ints(&ring);
  a.held_out = static_cast<int32_t*>(to[0]), a.ring_out = static_cast<int32_t*>(to[1]);
  a.seq_lens = static_cast<int32_t*>(to[2]), a.cu_seqlens = static_cast<int32_t*>(to[3]);
  a.slots = static_cast<int64_t*>(to[4]), a.positions = static_cast<int32_t*>(to[5]);
  const c10::DeviceGuard guard(on.device);
  check(lib.plan(&a, stream.raw));
  PyObject* r = PyTuple_New(6);
  if (!r) return nullptr;
  for (int i = 0; i < 6; ++i)
    PyTuple_SET_ITEM(r, i, own[i].defined() ? THPVariable_Wrap(own[i]) : Py_NewRef(args[8 + i]));
  return r;
  END_HANDLE_TH_ERRORS
}

// Strides of a [N, rows, V] view with contiguous rows.
void rows(const On& on, const char* name, const at::Tensor& t, at::ScalarType type, int64_t N, int64_t n_rows,
          int64_t V, int64_t* seq, int64_t* row) {
  on.also(name, &t);
  of_type(name, t, type);
  if (t.dim() != 3 || t.size(0) != N || t.size(1) != n_rows || t.size(2) != V || (V > 1 && t.stride(2) != 1))
    value_error("%s must be of shape [%lld, %lld, %lld] with contiguous rows", name, (long long)N,
                            (long long)n_rows, (long long)V);
  *seq = t.stride(0);
  *row = t.stride(1);
}

// verify_drafts(p, q, drafts, uniform, n_drafts, accept, tokens, workspace, stream) -> (accept, tokens)
PyObject* verify_drafts(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  arguments(nargs, 9);
  const at::Tensor &p = tensor(args[0], "p"), &drafts = tensor(args[2], "drafts"),
                   &uniform = tensor(args[3], "uniform");
  Opt q = optional(args[1], "q"), n_drafts = optional(args[4], "n_drafts"), accept = optional(args[5], "accept"),
      tokens = optional(args[6], "tokens"), given = optional(args[7], "workspace");
  const On on(p);
  if (p.dim() != 3 || drafts.dim() != 2)
    value_error("p must be of shape [N, m + 1, V] and drafts of shape [N, m]");
  const int64_t N = drafts.size(0), m = drafts.size(1), V = p.size(2);
  kda_verify_args a{};
  a.N = to_int("N", N), a.m = to_int("m", m), a.V = to_int("V", V);
  a.dtype = act_type(p, "p");
  rows(on, "p", p, p.scalar_type(), N, m + 1, V, &a.p_seq_stride, &a.p_row_stride);
  a.p = p.data_ptr();
  if (q) {
    rows(on, "q", *q, p.scalar_type(), N, m, V, &a.q_seq_stride, &a.q_row_stride);
    a.q = q->data_ptr();
  }
  plain(on, "drafts", &drafts, at::kInt, {N, m});
  plain(on, "uniform", &uniform, at::kFloat, {N, m + 1});
  plain(on, "n_drafts", n_drafts, at::kInt, {N});
  plain(on, "accept", accept, at::kInt, {N});
  plain(on, "tokens", tokens, at::kInt, {N, m + 1});
  const Stream stream(args[8], on);
  at::Tensor own_accept, own_tokens, scratch;
  if (!accept) own_accept = stream.empty({N}, at::kInt, on);
  if (!tokens) own_tokens = stream.empty({N, m + 1}, at::kInt, on);
  a.drafts = ints(&drafts);
  a.n_drafts = ints(n_drafts);
  a.uniform = static_cast<const float*>(uniform.data_ptr());
  a.accept = out_ints(accept ? *accept : own_accept);
  a.tokens = out_ints(tokens ? *tokens : own_tokens);
  workspace(&a, given, lib.verify_bytes, stream, on, &scratch);
  const c10::DeviceGuard guard(on.device);
  check(lib.verify(&a, stream.raw));
  PyObject* r = PyTuple_New(2);
  if (!r) return nullptr;
  PyTuple_SET_ITEM(r, 0, accept ? Py_NewRef(args[5]) : THPVariable_Wrap(own_accept));
  PyTuple_SET_ITEM(r, 1, tokens ? Py_NewRef(args[6]) : THPVariable_Wrap(own_tokens));
  return r;
  END_HANDLE_TH_ERRORS
}

// adjust_logits(logits, history, history_lens, prompt_lens, drafts, repetition, frequency, presence, bias_ids,
//               bias, bias_counts, mask, temperature, probs, out, out_dtype, workspace, stream) -> out
PyObject* adjust_logits(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  arguments(nargs, 18);
  const at::Tensor& logits = tensor(args[0], "logits");
  Opt history = optional(args[1], "history"), history_lens = optional(args[2], "history_lens"),
      prompt_lens = optional(args[3], "prompt_lens"), drafts = optional(args[4], "drafts"),
      repetition = optional(args[5], "repetition"), frequency = optional(args[6], "frequency"),
      presence = optional(args[7], "presence"), bias_ids = optional(args[8], "bias_ids"),
      bias = optional(args[9], "bias"), bias_counts = optional(args[10], "bias_counts"),
      mask = optional(args[11], "mask"), temperature = optional(args[12], "temperature"),
      o = optional(args[14], "out"), given = optional(args[16], "workspace");
  const On on(logits);
  if (logits.dim() != 3) value_error("logits must be of shape [N, R, V]");
  const int64_t N = logits.size(0), R = logits.size(1), V = logits.size(2);
  kda_logits_args a{};
  a.N = to_int("N", N), a.R = to_int("R", R), a.V = to_int("V", V);
  a.dtype = act_type(logits, "logits");
  rows(on, "logits", logits, logits.scalar_type(), N, R, V, &a.seq_stride, &a.row_stride);
  const at::ScalarType out = out_type(o, args[15]);
  a.out_dtype = out == at::kFloat ? KDA_F32 : KDA_BF16;
  if ((history != nullptr) != (history_lens != nullptr)) value_error("history and history_lens go together");
  if (prompt_lens && !history) value_error("prompt_lens needs history");
  if (history) {
    on.also("history", history);
    of_type("history", *history, at::kInt);
    if (history->dim() != 2 || history->size(0) != N || (history->size(1) > 1 && history->stride(1) != 1))
      value_error("history must be of shape [%lld, ids], ids side by side", (long long)N);
    a.max_history = to_int("history", history->size(1));
    a.history_stride = N > 1 ? history->stride(0) : a.max_history;
    if (a.max_history > 0) {  // a history of no columns is none
      a.history = ints(history);
      a.history_lens = ints(history_lens);
      a.prompt_lens = ints(prompt_lens);
    }
  }
  plain(on, "history_lens", history_lens, at::kInt, {N});
  plain(on, "prompt_lens", prompt_lens, at::kInt, {N});
  plain(on, "drafts", drafts, at::kInt, {N, R - 1});
  plain(on, "repetition", repetition, at::kFloat, {N});
  plain(on, "frequency", frequency, at::kFloat, {N});
  plain(on, "presence", presence, at::kFloat, {N});
  plain(on, "temperature", temperature, at::kFloat, {N});
  if ((bias != nullptr) != (bias_ids != nullptr)) value_error("bias and bias_ids go together");
  if (bias_counts && !bias) value_error("bias_counts needs bias and bias_ids");
  if (bias) {
    if (bias->dim() != 2) value_error("bias must be of shape [%lld, entries]", (long long)N);
    plain(on, "bias", bias, at::kFloat, {N, bias->size(1)});
    plain(on, "bias_ids", bias_ids, at::kInt, {N, bias->size(1)});
    plain(on, "bias_counts", bias_counts, at::kInt, {N});
    a.max_bias = to_int("bias", bias->size(1));
    if (a.max_bias > 0) {
      a.bias_ids = ints(bias_ids);
      a.bias = static_cast<const float*>(bias->data_ptr());
      a.bias_counts = ints(bias_counts);
    }
  }
  if (mask) {
    rows(on, "mask", *mask, at::kInt, N, R, (V + 31) / 32, &a.mask_seq_stride, &a.mask_row_stride);
    a.mask = reinterpret_cast<const uint32_t*>(ints(mask));
  }
  const auto floats = [](Opt x) { return x ? static_cast<const float*>(x->data_ptr()) : nullptr; };
  a.drafts = drafts && R > 1 ? ints(drafts) : nullptr;
  a.repetition = floats(repetition), a.frequency = floats(frequency), a.presence = floats(presence);
  a.temperature = floats(temperature);
  a.flags = truth(args[13]) ? KDA_LOGITS_PROBS : 0;
  const Stream stream(args[17], on);
  at::Tensor own, scratch;
  if (!o) own = stream.empty(logits.sizes(), out, on);
  const at::Tensor& to = o ? *o : own;
  rows(on, "out", to, out, N, R, V, &a.out_seq_stride, &a.out_row_stride);
  a.logits = logits.data_ptr();
  a.out = to.data_ptr();
  workspace(&a, given, lib.logits_bytes, stream, on, &scratch);
  const c10::DeviceGuard guard(on.device);
  check(lib.logits(&a, stream.raw));
  return o ? Py_NewRef(args[14]) : THPVariable_Wrap(own);
  END_HANDLE_TH_ERRORS
}

#define METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    METHOD(bind), METHOD(kv_append), METHOD(paged_decode), METHOD(verify_drafts), METHOD(lin_chunk_fwd),
    METHOD(lin_decode), METHOD(page_plan), METHOD(adjust_logits),
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
