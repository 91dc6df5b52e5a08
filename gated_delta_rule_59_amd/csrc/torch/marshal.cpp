// Tensor marshalling of kda_kv_append, kda_paged_decode and kda_verify_drafts for binding.py: checks
// the tensors, fills the argument structs of include/kda.h, allocates what the caller left out, and
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

#include "kda.h"

namespace {

struct Library {
  decltype(&kda_kv_append) append;
  decltype(&kda_paged_decode) decode;
  decltype(&kda_paged_decode_workspace_bytes) decode_bytes;
  decltype(&kda_verify_drafts) verify;
  decltype(&kda_verify_drafts_workspace_bytes) verify_bytes;
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

// Token and head strides of a [lead0, lead1, heads, d] view whose tokens lie evenly apart.
void heads(const On& on, const char* name, const at::Tensor& t, at::ScalarType type, int64_t lead0,
           int64_t lead1, int64_t d, int64_t* token, int64_t* head) {
  on.also(name, &t);
  of_type(name, t, type);
  if (t.dim() != 4 || t.size(0) != lead0 || t.size(1) != lead1 || t.size(3) != d)
    value_error("%s must be of shape [%lld, %lld, heads, %lld]", name, (long long)lead0,
                            (long long)lead1, (long long)d);
  const int64_t H = t.size(2);
  *token = H * d;
  *head = d;
  if (t.numel() == 0) return;
  const auto s = t.strides();
  if ((s[3] != 1 && d > 1) || (lead0 > 1 && lead1 > 1 && s[0] != lead1 * s[1]))
    value_error("%s must have contiguous channels and evenly spaced tokens", name);
  if (lead1 > 1) *token = s[1];
  else if (lead0 > 1) *token = s[0];
  if (H > 1) *head = s[2];
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
  arguments(n, 7);
  void* p[6];
  for (int i = 0; i < 6; ++i) {
    p[i] = PyLong_AsVoidPtr(args[i]);
    if (!p[i] && PyErr_Occurred()) throw python_error();
  }
  Py_INCREF(args[6]);
  Py_XDECREF(lib.error);
  lib = Library{reinterpret_cast<decltype(lib.append)>(p[0]), reinterpret_cast<decltype(lib.decode)>(p[1]),
                reinterpret_cast<decltype(lib.decode_bytes)>(p[2]), reinterpret_cast<decltype(lib.verify)>(p[3]),
                reinterpret_cast<decltype(lib.verify_bytes)>(p[4]),
                reinterpret_cast<decltype(lib.last_error)>(p[5]), args[6]};
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
  if (!o && !THPDtype_Check(args[12])) type_error("out_dtype must be a torch.dtype");
  const at::ScalarType out = o ? o->scalar_type() : reinterpret_cast<THPDtype*>(args[12])->scalar_type;
  if (out != at::kFloat && out != at::kBFloat16)
    type_error("the output must be float32 or bfloat16");
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

PyMethodDef methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(bind)), METH_FASTCALL, nullptr},
    {"kv_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(kv_append)), METH_FASTCALL, nullptr},
    {"paged_decode", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(paged_decode)), METH_FASTCALL, nullptr},
    {"verify_drafts", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(verify_drafts)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
