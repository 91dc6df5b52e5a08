// libkda C ABI: argument validation, path selection, workspace sizing and launches.
// Every check happens on the host before anything is enqueued; see include/kda.h.
#include "../../include/kda.h"

#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <string>

#include "kda_internal.h"

namespace {

thread_local std::string g_last_error;

kda_status fail(kda_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return s;
}

kda_status ok() {
  g_last_error.clear();
  return KDA_OK;
}

// A launch's grid holds at most 2^32 - 1 work-items. The decode kernels run one
// 256-work-item workgroup per (sequence, head).
constexpr int64_t kMaxGridItems = 0xffffffffLL;
constexpr int64_t kMaxDecodePairs = kMaxGridItems / 256;
// kda_verify_drafts: a wave per sequence, in workgroups of four in one launch and alone in the other;
// where the first has more waves than sequences, they are at most 65,536.
constexpr int64_t kMaxVerifySequences = 4 * kMaxDecodePairs;

bool head_dim_ok(int d) { return d == 32 || d == 64 || d == 128; }
bool dtype_ok(kda_dtype t) { return t == KDA_F32 || t == KDA_BF16; }
size_t dsize(kda_dtype t) { return t == KDA_F32 ? 4 : 2; }

struct Range {
  const char* name;
  uintptr_t lo, hi;  // [lo, hi)
};

Range range(const char* name, const void* p, size_t bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return Range{name, a, a + bytes};
}

bool overlap(const Range& a, const Range& b) {
  return a.lo < b.hi && b.lo < a.hi && a.hi > a.lo && b.hi > b.lo;
}

bool env_check() {
  const char* s = std::getenv("KDA_CHECK");
  return s && s[0] == '1';
}

// Counts g outside [-5, 0] and beta outside [0, 1] on the device into counts[0 .. n_counts)
// (caller-owned device memory; at most kda::check_blocks() of them are used), copies them to
// the host and synchronises the stream.
kda_status run_gate_check(const void* g, int64_t n_g, const void* beta, int64_t n_beta,
                          kda_dtype dt, int64_t* counts, int64_t n_counts, hipStream_t stream,
                          int64_t* n_bad) {
  int64_t host[1024];
  static_assert(sizeof(host) / sizeof(host[0]) >= 1024, "host copy of the counters");
  const int nb = (int)std::min<int64_t>(n_counts, kda::check_blocks());
  hipError_t e = kda::launch_check_gates(g, n_g, beta, n_beta, dt == KDA_BF16, counts, nb, stream);
  if (e == hipSuccess)
    e = hipMemcpyAsync(host, counts, sizeof(int64_t) * nb, hipMemcpyDeviceToHost, stream);
  if (e == hipSuccess) e = hipStreamSynchronize(stream);
  if (e != hipSuccess) return fail(KDA_ERR_HIP, "gate check: %s", hipGetErrorString(e));
  int64_t total = 0;
  for (int i = 0; i < nb; ++i) total += host[i];
  *n_bad = total;
  return ok();
}

// KDA_CHECK=1: the gate check before a call, its counters held in the call's output buffer o
// (which the call overwrites afterwards, and which overlaps no input), so that nothing is
// allocated. o_bytes >= 64 (one token of one head), so at least seven 8-byte aligned
// counters fit.
kda_status env_gate_check(const void* g, int64_t n_g, const void* beta, int64_t n_beta,
                          kda_dtype dt, void* o, size_t o_bytes, hipStream_t stream) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(o), end = lo + o_bytes;
  const uintptr_t c0 = (lo + 7) & ~uintptr_t(7);
  int64_t bad = 0;
  kda_status s = run_gate_check(g, n_g, beta, n_beta, dt, reinterpret_cast<int64_t*>(c0),
                                (int64_t)((end - c0) / sizeof(int64_t)), stream, &bad);
  if (s != KDA_OK) return s;
  if (bad) return fail(KDA_ERR_DECAY_RANGE, "%lld gate values outside their range", (long long)bad);
  return KDA_OK;
}

// Tokens per step of the matrix-core walk. Two chunks composed into one 128-token step halve
// the serial steps and the workspace bytes, but the composition costs the parallel part about
// 30 % more; measured on MI355X it pays where the walk dominates, i.e. few (sequence, head)
// pairs (one 65,536-token sequence: 0.708 -> 0.446 ms with 2 heads, 1.12 -> 1.00 ms with 8),
// and is even with 16 or 32 heads. One chunk per step when asked, and whenever checkpoints fall
// between 128-token steps (decided from ckpt_every alone, so that the workspace size does not
// depend on ckpt_slots).
constexpr int kComposeMaxPairs = 8;
int walk_block(const kda_chunk_args* a, int n_seq) {
  if ((a->flags & KDA_FLAG_WALK64) || (a->ckpt_every > 0 && a->ckpt_every % 128 != 0)) return 64;
  if (a->flags & KDA_FLAG_WALK128) return 128;
  return (int64_t)n_seq * a->H <= kComposeMaxPairs ? 128 : 64;
}

// Shape/dtype validation shared by kda_chunk_fwd and kda_chunk_fwd_workspace_bytes.
kda_status validate_chunk_shapes(const kda_chunk_args* a, kda::ChunkPlan* p) {
  if (!a) return fail(KDA_ERR_NULL_PTR, "args is NULL");
  if (a->B < 1 || a->T < 0 || a->H < 1)
    return fail(KDA_ERR_BAD_SHAPE, "need B >= 1, T >= 0, H >= 1 (got B=%d T=%d H=%d)", a->B, a->T,
                a->H);
  if (!head_dim_ok(a->dk) || !head_dim_ok(a->dv))
    return fail(KDA_ERR_BAD_SHAPE, "dk and dv must be 32, 64 or 128 (got %d, %d)", a->dk, a->dv);
  if (a->chunk != 16 && a->chunk != 32 && a->chunk != 64)
    return fail(KDA_ERR_BAD_SHAPE, "chunk must be 16, 32 or 64 (got %d)", a->chunk);
  if (a->cu_seqlens) {
    if (a->B != 1) return fail(KDA_ERR_BAD_SHAPE, "cu_seqlens requires B == 1 (got %d)", a->B);
    if (a->N < 1) return fail(KDA_ERR_BAD_SHAPE, "cu_seqlens requires N >= 1 (got %d)", a->N);
  }
  if (!dtype_ok(a->act_dtype) || !dtype_ok(a->gate_dtype) || !dtype_ok(a->out_dtype))
    return fail(KDA_ERR_BAD_DTYPE, "unknown dtype");
  if (a->act_dtype != a->gate_dtype)
    return fail(KDA_ERR_BAD_DTYPE, "act_dtype and gate_dtype must match (both F32 or both BF16)");
  if (a->flags & ~(KDA_FLAG_GENERIC | KDA_FLAG_PAIRWISE_DIAG | KDA_FLAG_WALK64 | KDA_FLAG_WALK128))
    return fail(KDA_ERR_UNSUPPORTED, "unknown flags 0x%x", a->flags);
  if ((a->flags & KDA_FLAG_WALK64) && (a->flags & KDA_FLAG_WALK128))
    return fail(KDA_ERR_UNSUPPORTED, "KDA_FLAG_WALK64 and KDA_FLAG_WALK128 exclude each other");
  if ((a->flags & KDA_FLAG_WALK128) && a->ckpt_every > 0 && a->ckpt_every % 128 != 0)
    return fail(KDA_ERR_UNSUPPORTED,
                "KDA_FLAG_WALK128: checkpoints every %d tokens fall between 128-token steps",
                a->ckpt_every);
  const int64_t tokens = (int64_t)a->B * a->T;
  const int n_seq = a->cu_seqlens ? a->N : a->B;
  if (tokens * a->H * (int64_t)(a->dk > a->dv ? a->dk : a->dv) > (int64_t(1) << 40))
    return fail(KDA_ERR_BAD_SHAPE, "problem too large");
  if ((int64_t)n_seq * a->H * (a->dv / 16) > 0x7fffffffLL)
    return fail(KDA_ERR_BAD_SHAPE, "too many (sequence, head) pairs");
  // the largest grid either prefill path launches (work-items): the per-(chunk, head)
  // kernel, and the walk's (sequence, head, column strip) workgroups of up to 512 work-items,
  // two per strip, for each of up to 15 segment walks
  const int64_t chunks = (a->cu_seqlens ? ((int64_t)a->T + 63) / 64 + n_seq
                                        : (int64_t)a->B * (((int64_t)a->T + 63) / 64));
  const int64_t walk_items = ((int64_t)n_seq * a->H + 7) / 8 * 8 * (a->dv / 16) * 2 * 512 *
                             (a->segments >= 3 ? 2 * a->segments - 3 : 1);
  if (chunks * a->H * 256 > kMaxGridItems || walk_items > kMaxGridItems)
    return fail(KDA_ERR_BAD_SHAPE, "the problem needs more work-items than one launch holds");
  if (a->ckpt_every < 0 || (a->ckpt_every > 0 && a->ckpt_every % a->chunk != 0))
    return fail(KDA_ERR_BAD_SHAPE, "ckpt_every must be 0 or a positive multiple of chunk (got %d)",
                a->ckpt_every);
  if (a->ckpt_every > 0 && a->ckpt_slots < 0)
    return fail(KDA_ERR_BAD_SHAPE, "ckpt_slots must be >= 0 (got %d)", a->ckpt_slots);
  if (a->segments < 0 || a->segments > 8)
    return fail(KDA_ERR_BAD_SHAPE, "segments must be in 0 .. 8 (got %d)", a->segments);
  const bool ck = a->ckpt_every > 0 && a->ckpt_slots > 0;
  *p = kda::ChunkPlan{a->B, a->T, a->H, a->dk, a->dv, a->chunk, a->cu_seqlens, n_seq,
                      a->act_dtype == KDA_BF16, a->out_dtype == KDA_BF16,
                      a->q, a->k, a->v, a->g, a->beta, a->S0, a->o, a->S_T,
                      a->workspace, a->workspace_bytes,
                      ck ? a->ckpt : nullptr, ck ? a->ckpt_every : 0, ck ? a->ckpt_slots : 0,
                      (a->flags & KDA_FLAG_PAIRWISE_DIAG) != 0, a->segments,
                      walk_block(a, n_seq)};
  return KDA_OK;
}

bool use_fast(const kda_chunk_args* a, const kda::ChunkPlan& p) {
  return !(a->flags & KDA_FLAG_GENERIC) && kda::fast_path_applies(p);
}

// kda_chunk_fwd and kda_chunk_fwd_noalloc. With noalloc the workspace fields of *a are
// ignored and the library's fixed device scratch takes the workspace's place.
kda_status chunk_fwd(const kda_chunk_args* a, void* hip_stream, bool noalloc) {
  kda::ChunkPlan p;
  kda_status s = validate_chunk_shapes(a, &p);
  if (s != KDA_OK) return s;
  const size_t es = dsize(a->act_dtype), os = dsize(a->out_dtype);
  const size_t tok = (size_t)a->B * a->T * a->H;
  // zero tokens: the per-token arrays are empty and may be NULL (as an empty tensor's is)
  if (tok > 0 && (!a->q || !a->k || !a->v || !a->g || !a->beta || !a->o))
    return fail(KDA_ERR_NULL_PTR, "q, k, v, g, beta and o must be non-NULL");
  const size_t st = (size_t)p.n_seq * a->H * a->dk * a->dv * 4;
  const Range in[] = {range("q", a->q, tok * a->dk * es), range("k", a->k, tok * a->dk * es),
                      range("v", a->v, tok * a->dv * es), range("g", a->g, tok * a->dk * es),
                      range("beta", a->beta, tok * es),
                      range("S0", a->S0, a->S0 ? st : 0),
                      range("cu_seqlens", a->cu_seqlens,
                            a->cu_seqlens ? sizeof(int32_t) * (a->N + 1) : 0)};
  const Range o = range("o", a->o, tok * a->dv * os);
  const Range sT = range("S_T", a->S_T, a->S_T ? st : 0);
  for (const Range& r : in)
    if (overlap(o, r)) return fail(KDA_ERR_ALIAS, "o overlaps %s", r.name);
  for (const Range& r : in) {
    if (!overlap(sT, r)) continue;
    if (std::strcmp(r.name, "S0") == 0 && a->S_T == a->S0) continue;  // in-place continue
    return fail(KDA_ERR_ALIAS, "S_T overlaps %s", r.name);
  }
  if (overlap(sT, o)) return fail(KDA_ERR_ALIAS, "S_T overlaps o");
  if (p.ckpt_every > 0 && !a->ckpt) return fail(KDA_ERR_NULL_PTR, "ckpt is NULL with ckpt_every > 0");
  const Range ck = range("ckpt", p.ckpt, p.ckpt ? (size_t)p.ckpt_slots * a->H * a->dk * a->dv * 4 : 0);
  for (const Range& r : in)
    if (overlap(ck, r)) return fail(KDA_ERR_ALIAS, "ckpt overlaps %s", r.name);
  if (overlap(ck, o) || overlap(ck, sT)) return fail(KDA_ERR_ALIAS, "ckpt overlaps an output");

  const bool fast = use_fast(a, p);
  if (fast && noalloc) {
    const size_t need = kda::fast_workspace_bytes(p);
    if (need > kda::noalloc_scratch_bytes())
      return fail(KDA_ERR_WORKSPACE,
                  "kda_chunk_fwd_noalloc: these sizes need %zu bytes of scratch, more than the "
                  "%zu bytes of the library's fixed scratch (use kda_chunk_fwd with a workspace)",
                  need, kda::noalloc_scratch_bytes());
    void* ws = nullptr;
    const hipError_t e = kda::noalloc_scratch(&ws);
    if (e != hipSuccess)
      return fail(KDA_ERR_HIP, "kda_chunk_fwd_noalloc: scratch address: %s", hipGetErrorString(e));
    p.workspace = ws;
    p.workspace_bytes = kda::noalloc_scratch_bytes();
  } else if (fast) {
    const size_t need = kda::fast_workspace_bytes(p);
    if (need && (!a->workspace || a->workspace_bytes < need))
      return fail(KDA_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need,
                  a->workspace ? a->workspace_bytes : (size_t)0);
    if (reinterpret_cast<uintptr_t>(a->workspace) % 256)
      return fail(KDA_ERR_WORKSPACE, "workspace must be 256-byte aligned");
    const Range ws = range("workspace", a->workspace, need);
    for (const Range& r : in)
      if (overlap(ws, r)) return fail(KDA_ERR_ALIAS, "workspace overlaps %s", r.name);
    if (overlap(ws, o) || overlap(ws, sT) || overlap(ws, ck))
      return fail(KDA_ERR_ALIAS, "workspace overlaps an output");
  }
  hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  if (env_check() && tok > 0) {
    s = env_gate_check(a->g, (int64_t)(tok * a->dk), a->beta, (int64_t)tok, a->gate_dtype, a->o,
                       tok * a->dv * os, stream);
    if (s != KDA_OK) return s;
  }
  const hipError_t e = fast ? kda::launch_chunk_fast(p, stream) : kda::launch_chunk_generic(p, stream);
  if (e != hipSuccess) return fail(KDA_ERR_HIP, "kda_chunk_fwd launch: %s", hipGetErrorString(e));
  return ok();
}

// ---- paged caches -----------------------------------------------------------------------

bool cache_dtype_ok(kda_dtype t) { return t == KDA_F32 || t == KDA_BF16 || t == KDA_F8E4M3; }
size_t cache_dsize(kda_dtype t) { return t == KDA_F32 ? 4 : t == KDA_BF16 ? 2 : 1; }
constexpr int64_t kMaxStride = int64_t(1) << 40;  // bytes; keeps every address below 2^63

// A stride (elements of `es` bytes) of an array read and written 16 bytes at a time.
bool stride_ok(int64_t s, size_t es) {
  return s >= 0 && s <= kMaxStride / (int64_t)es && s * (int64_t)es % 16 == 0;
}
bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// Shapes, dtypes and strides of a paged cache beside activations of type `act`.
kda_status validate_cache_shapes(const kda_page_cache& c, kda_dtype act) {
  if (!cache_dtype_ok(c.dtype)) return fail(KDA_ERR_BAD_DTYPE, "unknown cache dtype");
  if ((act == KDA_F32) != (c.dtype == KDA_F32))
    return fail(KDA_ERR_BAD_DTYPE, "an F32 cache goes with F32 activations, BF16 and F8E4M3 with BF16");
  if (c.num_pages < 1 || c.page_size < 1 || c.max_pages < 1)
    return fail(KDA_ERR_BAD_SHAPE, "need num_pages, page_size, max_pages >= 1 (got %d, %d, %d)",
                c.num_pages, c.page_size, c.max_pages);
  return KDA_OK;
}

kda_status validate_cache(const kda_page_cache& c, int Hkv, int d, Range* k, Range* v) {
  if (!c.k || !c.v || !c.block_table)
    return fail(KDA_ERR_NULL_PTR, "cache k, v and block_table must be non-NULL");
  if (c.dtype != KDA_F8E4M3 && (c.k_scale || c.v_scale))
    return fail(KDA_ERR_UNSUPPORTED, "k_scale and v_scale are for F8E4M3 caches");
  const size_t es = cache_dsize(c.dtype);
  const int64_t strides[] = {c.k_page_stride, c.k_token_stride, c.k_head_stride,
                             c.v_page_stride, c.v_token_stride, c.v_head_stride};
  for (int64_t s : strides)
    if (!stride_ok(s, es))
      return fail(KDA_ERR_BAD_SHAPE, "cache strides must be >= 0 and multiples of 16 bytes");
  if (!aligned16(c.k) || !aligned16(c.v))
    return fail(KDA_ERR_BAD_SHAPE, "cache k and v must be 16-byte aligned");
  if (c.table_stride < 0 || c.table_stride > kMaxStride)
    return fail(KDA_ERR_BAD_SHAPE, "table_stride must be >= 0");
  auto bytes = [&](int64_t page, int64_t token, int64_t head) {
    const double top = (double)(c.num_pages - 1) * (double)page +
                       (double)(c.page_size - 1) * (double)token + (double)(Hkv - 1) * (double)head;
    if (top * (double)es > 0x1p60) return SIZE_MAX;
    return (size_t)(((int64_t)(c.num_pages - 1) * page + (int64_t)(c.page_size - 1) * token +
                     (int64_t)(Hkv - 1) * head + d) * (int64_t)es);
  };
  const size_t kb = bytes(c.k_page_stride, c.k_token_stride, c.k_head_stride);
  const size_t vb = bytes(c.v_page_stride, c.v_token_stride, c.v_head_stride);
  if (kb == SIZE_MAX || vb == SIZE_MAX) return fail(KDA_ERR_BAD_SHAPE, "cache too large");
  *k = range("the key cache", c.k, kb);
  *v = range("the value cache", c.v, vb);
  return KDA_OK;
}

kda::PageCache page_cache(const kda_page_cache& c) {
  const int64_t es = (int64_t)cache_dsize(c.dtype);
  kda::PageCache r{};
  r.k = static_cast<char*>(c.k);
  r.v = static_cast<char*>(c.v);
  r.num_pages = c.num_pages;
  r.page_size = c.page_size;
  kda::divide_by(c.page_size, &r.ps_mul, &r.ps_shift);
  r.k_page = c.k_page_stride * es, r.k_token = c.k_token_stride * es, r.k_head = c.k_head_stride * es;
  r.v_page = c.v_page_stride * es, r.v_token = c.v_token_stride * es, r.v_head = c.v_head_stride * es;
  r.k_page16 = (unsigned)(r.k_page / 16), r.v_page16 = (unsigned)(r.v_page / 16);
  r.table = c.block_table;
  r.table_stride = c.table_stride;
  r.max_pages = c.max_pages;
  r.k_scale = c.k_scale;
  r.v_scale = c.v_scale;
  return r;
}

Range table_range(const kda_page_cache& c, int n_seq) {
  return range("block_table", c.block_table,
               sizeof(int32_t) * ((size_t)(n_seq - 1) * c.table_stride + c.max_pages));
}

// Rows of [tokens, heads, d] by strides (elements): what they span.
size_t span_bytes(int64_t tokens, int64_t token_stride, int heads, int64_t head_stride, int d, size_t es) {
  return tokens ? (size_t)((tokens - 1) * token_stride + (heads - 1) * head_stride + d) * es : 0;
}
bool span_ok(int64_t tokens, int64_t token_stride, int heads, int64_t head_stride) {
  return (double)tokens * (double)token_stride + (double)heads * (double)head_stride < 0x1p58;
}

// Shapes of kda_paged_decode, and its launch.
kda_status validate_decode_shapes(const kda_paged_decode_args* a, kda::PagedDecodePlan* p, size_t* ws) {
  if (!a) return fail(KDA_ERR_NULL_PTR, "args is NULL");
  if (a->N < 1 || a->m < 1 || a->Hq < 1 || a->Hkv < 1 || a->Hq % a->Hkv)
    return fail(KDA_ERR_BAD_SHAPE, "need N, m, Hkv >= 1 and Hq a multiple of Hkv (got N=%d m=%d Hq=%d Hkv=%d)",
                a->N, a->m, a->Hq, a->Hkv);
  if (!head_dim_ok(a->d)) return fail(KDA_ERR_BAD_SHAPE, "d must be 32, 64 or 128 (got %d)", a->d);
  if (!dtype_ok(a->act_dtype) || !dtype_ok(a->out_dtype)) return fail(KDA_ERR_BAD_DTYPE, "unknown dtype");
  if (a->flags) return fail(KDA_ERR_UNSUPPORTED, "unknown flags 0x%x", a->flags);
  kda_status s = validate_cache_shapes(a->cache, a->act_dtype);
  if (s != KDA_OK) return s;
  if (a->max_len < 1 || a->max_len > (int64_t)a->cache.max_pages * a->cache.page_size ||
      a->max_len > (1 << 30))
    return fail(KDA_ERR_BAD_SHAPE, "max_len must be in 1 .. max_pages * page_size, at most 2^30 (got %d)",
                a->max_len);
  if (a->window < 0) return fail(KDA_ERR_BAD_SHAPE, "window must be >= 0 (got %d)", a->window);
  if ((int64_t)a->m * a->Hq > (1 << 24)) return fail(KDA_ERR_BAD_SHAPE, "m * Hq too large");
  // one 256-work-item workgroup per (sequence, row block, head); a row block holds 16 rows or more
  const int64_t pairs = (int64_t)a->N * a->Hkv * (((int64_t)a->m * (a->Hq / a->Hkv) + 15) / 16);
  if (pairs > kMaxDecodePairs || (int64_t)a->N * a->m * a->Hq > (int64_t(1) << 40) ||
      pairs / a->N * (a->max_len / 32 + 1) > 0x7fffffffLL)
    return fail(KDA_ERR_BAD_SHAPE, "N * m * Hq or max_len * m * Hq too large for one launch");
  *p = kda::PagedDecodePlan{};
  p->N = a->N, p->m = a->m, p->Hq = a->Hq, p->Hkv = a->Hkv, p->d = a->d;
  p->out_bf16 = a->out_dtype == KDA_BF16;
  p->cache_type = a->cache.dtype;
  p->max_len = a->max_len;
  p->window = a->window;
  *ws = kda::plan_paged_decode(p);
  return KDA_OK;
}

kda_status validate_verify_shapes(const kda_verify_args* a) {
  if (!a) return fail(KDA_ERR_NULL_PTR, "args is NULL");
  if (a->N < 1 || a->m < 1 || a->V < 1)
    return fail(KDA_ERR_BAD_SHAPE, "need N, m, V >= 1 (got N=%d m=%d V=%d)", a->N, a->m, a->V);
  if (!dtype_ok(a->dtype)) return fail(KDA_ERR_BAD_DTYPE, "unknown dtype");
  if (a->m > (1 << 24)) return fail(KDA_ERR_BAD_SHAPE, "m too large (got %d)", a->m);
  if (a->V > (1 << 30)) return fail(KDA_ERR_BAD_SHAPE, "V too large (got %d)", a->V);
  if (a->N > kMaxVerifySequences) return fail(KDA_ERR_BAD_SHAPE, "N too large for one launch (got %d)", a->N);
  return KDA_OK;
}

}  // namespace

extern "C" {

kda_status kda_chunk_fwd(const kda_chunk_args* a, void* hip_stream) {
  return chunk_fwd(a, hip_stream, false);
}

kda_status kda_chunk_fwd_noalloc(const kda_chunk_args* a, void* hip_stream) {
  return chunk_fwd(a, hip_stream, true);
}

size_t kda_chunk_fwd_workspace_bytes(const kda_chunk_args* a) {
  kda::ChunkPlan p;
  if (validate_chunk_shapes(a, &p) != KDA_OK) return SIZE_MAX;
  ok();
  return use_fast(a, p) ? kda::fast_workspace_bytes(p) : 0;
}

kda_status kda_decode_step(const kda_decode_args* a, void* hip_stream) {
  if (!a) return fail(KDA_ERR_NULL_PTR, "args is NULL");
  if (a->N < 1 || a->H < 1)
    return fail(KDA_ERR_BAD_SHAPE, "need N >= 1 and H >= 1 (got N=%d H=%d)", a->N, a->H);
  if (!head_dim_ok(a->dk) || !head_dim_ok(a->dv))
    return fail(KDA_ERR_BAD_SHAPE, "dk and dv must be 32, 64 or 128 (got %d, %d)", a->dk, a->dv);
  if ((int64_t)a->N * a->H > kMaxDecodePairs)
    return fail(KDA_ERR_BAD_SHAPE, "N * H = %lld exceeds one launch (%lld)",
                (long long)a->N * a->H, (long long)kMaxDecodePairs);
  if (!dtype_ok(a->act_dtype) || !dtype_ok(a->gate_dtype) || !dtype_ok(a->out_dtype))
    return fail(KDA_ERR_BAD_DTYPE, "unknown dtype");
  if (a->act_dtype != a->gate_dtype)
    return fail(KDA_ERR_BAD_DTYPE, "act_dtype and gate_dtype must match (both F32 or both BF16)");
  if (!a->q || !a->k || !a->v || !a->g || !a->beta || !a->S || !a->o)
    return fail(KDA_ERR_NULL_PTR, "q, k, v, g, beta, S and o must be non-NULL");
  const size_t es = dsize(a->act_dtype), os = dsize(a->out_dtype);
  const size_t nh = (size_t)a->N * a->H;
  const Range in[] = {range("q", a->q, nh * a->dk * es), range("k", a->k, nh * a->dk * es),
                      range("v", a->v, nh * a->dv * es), range("g", a->g, nh * a->dk * es),
                      range("beta", a->beta, nh * es)};
  const Range S = range("S", a->S, nh * a->dk * a->dv * 4);
  const Range o = range("o", a->o, nh * a->dv * os);
  for (const Range& r : in) {
    if (overlap(o, r)) return fail(KDA_ERR_ALIAS, "o overlaps %s", r.name);
    if (overlap(S, r)) return fail(KDA_ERR_ALIAS, "S overlaps %s", r.name);
  }
  if (overlap(S, o)) return fail(KDA_ERR_ALIAS, "S overlaps o");
  hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  if (env_check()) {
    kda_status s = env_gate_check(a->g, (int64_t)(nh * a->dk), a->beta, (int64_t)nh,
                                  a->gate_dtype, a->o, nh * a->dv * os, stream);
    if (s != KDA_OK) return s;
  }
  const kda::DecodePlan p{a->N, a->H, a->dk, a->dv, a->act_dtype == KDA_BF16,
                          a->out_dtype == KDA_BF16, a->q, a->k, a->v, a->g, a->beta, a->S, a->o};
  const hipError_t e = kda::launch_decode(p, stream);
  if (e != hipSuccess) return fail(KDA_ERR_HIP, "kda_decode_step launch: %s", hipGetErrorString(e));
  return ok();
}

kda_status kda_decode_multi(const kda_decode_multi_args* a, void* hip_stream) {
  if (!a) return fail(KDA_ERR_NULL_PTR, "args is NULL");
  if (a->N < 1 || a->H < 1 || a->m < 1)
    return fail(KDA_ERR_BAD_SHAPE, "need N, H, m >= 1 (got N=%d H=%d m=%d)", a->N, a->H, a->m);
  if (!head_dim_ok(a->dk) || !head_dim_ok(a->dv))
    return fail(KDA_ERR_BAD_SHAPE, "dk and dv must be 32, 64 or 128 (got %d, %d)", a->dk, a->dv);
  if ((int64_t)a->N * a->H > kMaxDecodePairs || (int64_t)a->N * a->m * a->H > (int64_t(1) << 40))
    return fail(KDA_ERR_BAD_SHAPE, "N * H or N * m * H too large for one launch");
  if (!dtype_ok(a->act_dtype) || !dtype_ok(a->gate_dtype) || !dtype_ok(a->out_dtype))
    return fail(KDA_ERR_BAD_DTYPE, "unknown dtype");
  if (a->act_dtype != a->gate_dtype)
    return fail(KDA_ERR_BAD_DTYPE, "act_dtype and gate_dtype must match (both F32 or both BF16)");
  if (!a->q || !a->k || !a->v || !a->g || !a->beta || !a->S)
    return fail(KDA_ERR_NULL_PTR, "q, k, v, g, beta and S must be non-NULL");
  const size_t es = dsize(a->act_dtype), os = dsize(a->out_dtype);
  const size_t nh = (size_t)a->N * a->H, nmh = nh * a->m;
  const Range in[] = {range("q", a->q, nmh * a->dk * es), range("k", a->k, nmh * a->dk * es),
                      range("v", a->v, nmh * a->dv * es), range("g", a->g, nmh * a->dk * es),
                      range("beta", a->beta, nmh * es),
                      range("accept", a->accept, a->accept ? sizeof(int32_t) * a->N : 0)};
  const Range S = range("S", a->S, nh * a->dk * a->dv * 4);
  const Range o = range("o", a->o, a->o ? nmh * a->dv * os : 0);
  for (const Range& r : in) {
    if (overlap(o, r)) return fail(KDA_ERR_ALIAS, "o overlaps %s", r.name);
    if (overlap(S, r)) return fail(KDA_ERR_ALIAS, "S overlaps %s", r.name);
  }
  if (overlap(S, o)) return fail(KDA_ERR_ALIAS, "S overlaps o");
  if (!a->o && !a->accept) return ok();
  hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  if (env_check()) {
    if (!a->o)
      return fail(KDA_ERR_UNSUPPORTED, "KDA_CHECK=1 needs o (the check keeps its counters there)");
    kda_status s = env_gate_check(a->g, (int64_t)(nmh * a->dk), a->beta, (int64_t)nmh,
                                  a->gate_dtype, a->o, nmh * a->dv * os, stream);
    if (s != KDA_OK) return s;
  }
  const kda::DecodeMultiPlan p{a->N, a->H, a->dk, a->dv, a->m, a->act_dtype == KDA_BF16,
                               a->out_dtype == KDA_BF16, a->q, a->k, a->v, a->g, a->beta,
                               a->S, a->o, a->accept};
  const hipError_t e = kda::launch_decode_multi(p, stream);
  if (e != hipSuccess) return fail(KDA_ERR_HIP, "kda_decode_multi launch: %s", hipGetErrorString(e));
  return ok();
}

kda_status kda_check_gates(const void* g, int64_t n_g, const void* beta, int64_t n_beta,
                           kda_dtype gate_dtype, int64_t* counts, int n_counts,
                           void* hip_stream, int64_t* n_bad) {
  if (!n_bad) return fail(KDA_ERR_NULL_PTR, "n_bad is NULL");
  if (n_g < 0 || n_beta < 0) return fail(KDA_ERR_BAD_SHAPE, "negative element count");
  if ((n_g && !g) || (n_beta && !beta)) return fail(KDA_ERR_NULL_PTR, "g or beta is NULL");
  if (!counts) return fail(KDA_ERR_NULL_PTR, "counts is NULL");
  if (n_counts < 1) return fail(KDA_ERR_BAD_SHAPE, "n_counts must be >= 1 (got %d)", n_counts);
  if (!dtype_ok(gate_dtype)) return fail(KDA_ERR_BAD_DTYPE, "unknown dtype");
  const size_t es = dsize(gate_dtype);
  const size_t used = sizeof(int64_t) * (size_t)std::min(n_counts, kda::check_blocks());
  const Range c = range("counts", counts, used);
  if (overlap(c, range("g", g, (size_t)n_g * es)) || overlap(c, range("beta", beta, (size_t)n_beta * es)))
    return fail(KDA_ERR_ALIAS, "counts overlaps g or beta");
  return run_gate_check(g, n_g, beta, n_beta, gate_dtype, counts, n_counts,
                        static_cast<hipStream_t>(hip_stream), n_bad);
}

kda_status kda_kv_append(const kda_kv_append_args* a, void* hip_stream) {
  if (!a) return fail(KDA_ERR_NULL_PTR, "args is NULL");
  if (a->B < 1 || a->T < 0 || a->Hq < 0 || a->Hkv < 1)
    return fail(KDA_ERR_BAD_SHAPE, "need B >= 1, T >= 0, Hq >= 0, Hkv >= 1 (got B=%d T=%d Hq=%d Hkv=%d)",
                a->B, a->T, a->Hq, a->Hkv);
  if (!head_dim_ok(a->d)) return fail(KDA_ERR_BAD_SHAPE, "d must be 32, 64 or 128 (got %d)", a->d);
  if (a->cu_seqlens && (a->B != 1 || a->N < 1))
    return fail(KDA_ERR_BAD_SHAPE, "cu_seqlens requires B == 1 and N >= 1 (got B=%d N=%d)", a->B, a->N);
  if (!dtype_ok(a->act_dtype)) return fail(KDA_ERR_BAD_DTYPE, "unknown dtype");
  if (a->flags & ~KDA_APPEND_PAIRS) return fail(KDA_ERR_UNSUPPORTED, "unknown flags 0x%x", a->flags);
  if (a->rot < 0 || a->rot > a->d || a->rot % 16)
    return fail(KDA_ERR_BAD_SHAPE, "rot must be a multiple of 16 in 0 .. d (got %d)", a->rot);
  kda_status s = validate_cache_shapes(a->cache, a->act_dtype);
  if (s != KDA_OK) return s;
  const int64_t tok = (int64_t)a->B * a->T;
  const int n_seq = a->cu_seqlens ? a->N : a->B;
  const int Hq = a->q ? a->Hq : 0;
  if (tok > kMaxDecodePairs || tok * ((int64_t)Hq + a->Hkv) * a->d > (int64_t(1) << 42) ||
      (int64_t)Hq + 2 * (int64_t)a->Hkv > (1 << 24))
    return fail(KDA_ERR_BAD_SHAPE, "too many tokens or heads for one launch");
  if ((a->rot > 0) != (a->inv_freq != nullptr))
    return fail(KDA_ERR_NULL_PTR, "inv_freq goes with rot > 0, and NULL with rot = 0");
  if ((a->q != nullptr) != (a->q_out != nullptr) && tok > 0)
    return fail(KDA_ERR_NULL_PTR, "q and q_out go together");
  if (a->q && Hq < 1) return fail(KDA_ERR_BAD_SHAPE, "q needs Hq >= 1");
  Range kc{}, vc{};
  s = validate_cache(a->cache, a->Hkv, a->d, &kc, &vc);
  if (s != KDA_OK) return s;
  // rows that are written lie apart (an expanded view's do not)
  const kda_page_cache& c = a->cache;
  if ((c.num_pages > 1 && std::min(c.k_page_stride, c.v_page_stride) < a->d) ||
      (c.page_size > 1 && std::min(c.k_token_stride, c.v_token_stride) < a->d) ||
      (a->Hkv > 1 && std::min(c.k_head_stride, c.v_head_stride) < a->d))
    return fail(KDA_ERR_BAD_SHAPE, "cache rows overlap: strides below d = %d", a->d);
  if (!a->start || (tok > 0 && (!a->k || !a->v)))
    return fail(KDA_ERR_NULL_PTR, "k, v and start must be non-NULL");
  const size_t es = dsize(a->act_dtype);
  const int64_t strides[] = {a->k_token_stride, a->k_head_stride, a->v_token_stride, a->v_head_stride,
                             a->q ? a->q_token_stride : 0, a->q ? a->q_head_stride : 0};
  for (int64_t x : strides)
    if (!stride_ok(x, es))
      return fail(KDA_ERR_BAD_SHAPE, "q, k and v strides must be >= 0 and multiples of 16 bytes");
  if (!aligned16(a->q) || !aligned16(a->k) || !aligned16(a->v) || !aligned16(a->q_out))
    return fail(KDA_ERR_BAD_SHAPE, "q, k, v and q_out must be 16-byte aligned");
  if (!span_ok(tok, a->k_token_stride, a->Hkv, a->k_head_stride) ||
      !span_ok(tok, a->v_token_stride, a->Hkv, a->v_head_stride) ||
      (a->q && !span_ok(tok, a->q_token_stride, Hq, a->q_head_stride)))
    return fail(KDA_ERR_BAD_SHAPE, "q, k or v too large");
  const Range in[] = {
      range("q", a->q, a->q ? span_bytes(tok, a->q_token_stride, Hq, a->q_head_stride, a->d, es) : 0),
      range("k", a->k, span_bytes(tok, a->k_token_stride, a->Hkv, a->k_head_stride, a->d, es)),
      range("v", a->v, span_bytes(tok, a->v_token_stride, a->Hkv, a->v_head_stride, a->d, es)),
      range("start", a->start, sizeof(int32_t) * (size_t)n_seq),
      range("inv_freq", a->inv_freq, a->inv_freq ? sizeof(float) * (a->rot / 2) : 0),
      range("cu_seqlens", a->cu_seqlens, a->cu_seqlens ? sizeof(int32_t) * ((size_t)a->N + 1) : 0),
      range("k_scale", a->cache.k_scale, a->cache.k_scale ? sizeof(float) * a->Hkv : 0),
      range("v_scale", a->cache.v_scale, a->cache.v_scale ? sizeof(float) * a->Hkv : 0),
      table_range(a->cache, n_seq)};
  const Range qo = range("q_out", a->q_out, a->q ? (size_t)tok * Hq * a->d * es : 0);
  const bool in_place = a->q_out == a->q && a->q_head_stride == a->d &&
                        a->q_token_stride == (int64_t)Hq * a->d;
  for (const Range& r : in) {
    if (overlap(kc, r) || overlap(vc, r)) return fail(KDA_ERR_ALIAS, "the cache overlaps %s", r.name);
    if (overlap(qo, r) && !(in_place && std::strcmp(r.name, "q") == 0))
      return fail(KDA_ERR_ALIAS, "q_out overlaps %s", r.name);
  }
  if (overlap(kc, qo) || overlap(vc, qo)) return fail(KDA_ERR_ALIAS, "the cache overlaps q_out");
  kda::KvAppendPlan p{};
  p.B = a->B, p.T = a->T, p.Hq = Hq, p.Hkv = a->Hkv, p.d = a->d, p.rot = a->rot, p.n_seq = n_seq;
  p.cu_seqlens = a->cu_seqlens;
  p.act_bf16 = a->act_dtype == KDA_BF16;
  p.pairs = (a->flags & KDA_APPEND_PAIRS) != 0;
  p.cache_type = a->cache.dtype;
  p.q = static_cast<const char*>(a->q);
  p.k = static_cast<const char*>(a->k);
  p.v = static_cast<const char*>(a->v);
  const int64_t e = (int64_t)es;
  p.q_token = strides[4] * e, p.q_head = strides[5] * e;
  p.k_token = a->k_token_stride * e, p.k_head = a->k_head_stride * e;
  p.v_token = a->v_token_stride * e, p.v_head = a->v_head_stride * e;
  p.q_out = static_cast<char*>(a->q_out);
  p.start = a->start;
  p.inv_freq = a->inv_freq;
  p.c = page_cache(a->cache);
  const hipError_t err = kda::launch_kv_append(p, static_cast<hipStream_t>(hip_stream));
  if (err != hipSuccess) return fail(KDA_ERR_HIP, "kda_kv_append launch: %s", hipGetErrorString(err));
  return ok();
}

size_t kda_paged_decode_workspace_bytes(const kda_paged_decode_args* a) {
  kda::PagedDecodePlan p;
  size_t ws = 0;
  if (validate_decode_shapes(a, &p, &ws) != KDA_OK) return SIZE_MAX;
  ok();
  return ws;
}

kda_status kda_paged_decode(const kda_paged_decode_args* a, void* hip_stream) {
  kda::PagedDecodePlan p;
  size_t need = 0;
  kda_status s = validate_decode_shapes(a, &p, &need);
  if (s != KDA_OK) return s;
  if (!a->q || !a->seq_lens || !a->o)
    return fail(KDA_ERR_NULL_PTR, "q, seq_lens and o must be non-NULL");
  if (!std::isfinite(a->scale)) return fail(KDA_ERR_BAD_SHAPE, "scale must be finite");
  Range kc{}, vc{};
  s = validate_cache(a->cache, a->Hkv, a->d, &kc, &vc);
  if (s != KDA_OK) return s;
  const size_t es = dsize(a->act_dtype), os = dsize(a->out_dtype);
  const int64_t tok = (int64_t)a->N * a->m;
  if (!stride_ok(a->q_token_stride, es) || !stride_ok(a->q_head_stride, es))
    return fail(KDA_ERR_BAD_SHAPE, "q strides must be >= 0 and multiples of 16 bytes");
  if (!aligned16(a->q) || !aligned16(a->o))
    return fail(KDA_ERR_BAD_SHAPE, "q and o must be 16-byte aligned");
  if (!span_ok(tok, a->q_token_stride, a->Hq, a->q_head_stride))
    return fail(KDA_ERR_BAD_SHAPE, "q too large");
  if (need && (!a->workspace || a->workspace_bytes < need))
    return fail(KDA_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need,
                a->workspace ? a->workspace_bytes : (size_t)0);
  if (reinterpret_cast<uintptr_t>(a->workspace) % 256)
    return fail(KDA_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  const Range in[] = {
      range("q", a->q, span_bytes(tok, a->q_token_stride, a->Hq, a->q_head_stride, a->d, es)),
      kc, vc, table_range(a->cache, a->N), range("seq_lens", a->seq_lens, sizeof(int32_t) * (size_t)a->N),
      range("k_scale", a->cache.k_scale, a->cache.k_scale ? sizeof(float) * a->Hkv : 0),
      range("v_scale", a->cache.v_scale, a->cache.v_scale ? sizeof(float) * a->Hkv : 0)};
  const Range out[] = {range("o", a->o, (size_t)tok * a->Hq * a->d * os),
                       range("lse", a->lse, a->lse ? (size_t)tok * a->Hq * sizeof(float) : 0),
                       range("workspace", a->workspace, need)};
  for (const Range& w : out)
    for (const Range& r : in)
      if (overlap(w, r)) return fail(KDA_ERR_ALIAS, "%s overlaps %s", w.name, r.name);
  if (overlap(out[0], out[1]) || overlap(out[0], out[2]) || overlap(out[1], out[2]))
    return fail(KDA_ERR_ALIAS, "o, lse and workspace must not overlap");
  p.q = static_cast<const char*>(a->q);
  p.q_token = a->q_token_stride * (int64_t)es;
  p.q_head = a->q_head_stride * (int64_t)es;
  p.c = page_cache(a->cache);
  p.seq_lens = a->seq_lens;
  p.scale = a->scale;
  p.o = a->o;
  p.lse = a->lse;
  kda::paged_decode_workspace(&p, a->workspace);
  const hipError_t e = kda::launch_paged_decode(p, static_cast<hipStream_t>(hip_stream));
  if (e != hipSuccess) return fail(KDA_ERR_HIP, "kda_paged_decode launch: %s", hipGetErrorString(e));
  return ok();
}

size_t kda_verify_drafts_workspace_bytes(const kda_verify_args* a) {
  if (validate_verify_shapes(a) != KDA_OK) return SIZE_MAX;
  ok();
  return kda::verify_workspace_bytes(a->N, a->V);
}

kda_status kda_verify_drafts(const kda_verify_args* a, void* hip_stream) {
  kda_status s = validate_verify_shapes(a);
  if (s != KDA_OK) return s;
  if (!a->p || !a->drafts || !a->uniform || !a->accept || !a->tokens)
    return fail(KDA_ERR_NULL_PTR, "p, drafts, uniform, accept and tokens must be non-NULL");
  const int64_t most = int64_t(1) << 42;  // elements: keeps every offset below 2^63
  auto rows_ok = [&](int64_t seq, int64_t row, int rows) {
    return row >= 0 && seq >= 0 && row <= most && seq <= most &&
           (double)(a->N - 1) * (double)seq + (double)(rows - 1) * (double)row < 0x1p58;
  };
  if (!rows_ok(a->p_seq_stride, a->p_row_stride, a->m + 1) ||
      (a->q && !rows_ok(a->q_seq_stride, a->q_row_stride, a->m)))
    return fail(KDA_ERR_BAD_SHAPE, "p and q strides must be >= 0 and in range");
  const size_t es = dsize(a->dtype);
  auto rows_bytes = [&](int64_t seq, int64_t row, int rows) {
    return (size_t)((a->N - 1) * seq + (int64_t)(rows - 1) * row + a->V) * es;
  };
  const size_t need = kda::verify_workspace_bytes(a->N, a->V);
  if (!a->workspace || a->workspace_bytes < need)
    return fail(KDA_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need,
                a->workspace ? a->workspace_bytes : (size_t)0);
  if (reinterpret_cast<uintptr_t>(a->workspace) % 256)
    return fail(KDA_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  const size_t nm = (size_t)a->N * a->m, nm1 = nm + a->N;
  const Range in[] = {range("p", a->p, rows_bytes(a->p_seq_stride, a->p_row_stride, a->m + 1)),
                      range("q", a->q, a->q ? rows_bytes(a->q_seq_stride, a->q_row_stride, a->m) : 0),
                      range("drafts", a->drafts, nm * sizeof(int32_t)),
                      range("n_drafts", a->n_drafts, a->n_drafts ? a->N * sizeof(int32_t) : 0),
                      range("uniform", a->uniform, nm1 * sizeof(float))};
  const Range out[] = {range("accept", a->accept, a->N * sizeof(int32_t)),
                       range("tokens", a->tokens, nm1 * sizeof(int32_t)),
                       range("workspace", a->workspace, need)};
  for (const Range& w : out)
    for (const Range& r : in)
      if (overlap(w, r)) return fail(KDA_ERR_ALIAS, "%s overlaps %s", w.name, r.name);
  if (overlap(out[0], out[1]) || overlap(out[0], out[2]) || overlap(out[1], out[2]))
    return fail(KDA_ERR_ALIAS, "accept, tokens and workspace must not overlap");
  const kda::VerifyPlan p{a->N, a->m, a->V, a->dtype == KDA_BF16, a->p, a->q,
                          a->p_seq_stride, a->p_row_stride, a->q_seq_stride, a->q_row_stride,
                          a->drafts, a->n_drafts, a->uniform, a->accept, a->tokens, a->workspace};
  const hipError_t e = kda::launch_verify(p, static_cast<hipStream_t>(hip_stream));
  if (e != hipSuccess) return fail(KDA_ERR_HIP, "kda_verify_drafts launch: %s", hipGetErrorString(e));
  return ok();
}

const char* kda_status_string(kda_status s) {
  switch (s) {
    case KDA_OK: return "KDA_OK";
    case KDA_ERR_NULL_PTR: return "KDA_ERR_NULL_PTR";
    case KDA_ERR_BAD_SHAPE: return "KDA_ERR_BAD_SHAPE";
    case KDA_ERR_BAD_DTYPE: return "KDA_ERR_BAD_DTYPE";
    case KDA_ERR_UNSUPPORTED: return "KDA_ERR_UNSUPPORTED";
    case KDA_ERR_DECAY_RANGE: return "KDA_ERR_DECAY_RANGE";
    case KDA_ERR_WORKSPACE: return "KDA_ERR_WORKSPACE";
    case KDA_ERR_HIP: return "KDA_ERR_HIP";
    case KDA_ERR_ALIAS: return "KDA_ERR_ALIAS";
  }
  return "KDA_ERR_UNKNOWN";
}

const char* kda_last_error(void) { return g_last_error.c_str(); }

int kda_abi_version(void) { return KDA_ABI_VERSION; }

}  // extern "C"
