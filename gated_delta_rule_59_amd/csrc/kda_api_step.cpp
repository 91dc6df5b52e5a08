// libkda C ABI, the calls around a step's layers: linear attention with a decay for each head, page
// plans, adjusted logits. Arguments are validated on the host before anything is enqueued; see
// include/kda.h.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "kda_api.h"
#include "kda_internal.h"

namespace {

using namespace kda::api;

// What prompts and decode share: heads, types, strides.
template <typename Args>
kda_status validate_lin(const Args* a) {
  if (a->Hk < 1 || a->H < 1 || a->H % a->Hk)
    return fail(KDA_ERR_BAD_SHAPE, "need Hk >= 1 and H a multiple of Hk (got Hk=%d H=%d)", a->Hk, a->H);
  if (!head_dim_ok(a->dk) || !head_dim_ok(a->dv))
    return fail(KDA_ERR_BAD_SHAPE, "dk and dv must be 32, 64 or 128 (got %d, %d)", a->dk, a->dv);
  if (!dtype_ok(a->act_dtype) || !dtype_ok(a->gate_dtype) || !dtype_ok(a->out_dtype))
    return fail(KDA_ERR_BAD_DTYPE, "unknown dtype");
  if (a->flags & ~KDA_LIN_FIXED_DECAY) return fail(KDA_ERR_UNSUPPORTED, "unknown flags 0x%x", a->flags);
  return KDA_OK;
}

template <typename Args>
kda_status validate_lin_rows(const Args* a, int64_t tok) {
  const size_t es = dsize(a->act_dtype);
  const int64_t strides[] = {a->q_token_stride, a->q_head_stride, a->k_token_stride,
                             a->k_head_stride,  a->v_token_stride, a->v_head_stride};
  for (int64_t s : strides)
    if (!stride_ok(s, es))
      return fail(KDA_ERR_BAD_SHAPE, "q, k and v strides must be >= 0 and multiples of 16 bytes");
  if (!aligned16(a->q) || !aligned16(a->k) || !aligned16(a->v) || !aligned16(a->o))
    return fail(KDA_ERR_BAD_SHAPE, "q, k, v and o must be 16-byte aligned");
  if (!span_ok(tok, a->q_token_stride, a->Hk, a->q_head_stride) ||
      !span_ok(tok, a->k_token_stride, a->Hk, a->k_head_stride) ||
      !span_ok(tok, a->v_token_stride, a->H, a->v_head_stride))
    return fail(KDA_ERR_BAD_SHAPE, "q, k or v too large");
  if (!std::isfinite(a->scale)) return fail(KDA_ERR_BAD_SHAPE, "scale must be finite");
  return KDA_OK;
}

template <typename Args>
void lin_inputs(const Args* a, int64_t tok, Range* r) {
  const size_t es = dsize(a->act_dtype);
  r[0] = range("q", a->q, span_bytes(tok, a->q_token_stride, a->Hk, a->q_head_stride, a->dk, es));
  r[1] = range("k", a->k, span_bytes(tok, a->k_token_stride, a->Hk, a->k_head_stride, a->dk, es));
  r[2] = range("v", a->v, span_bytes(tok, a->v_token_stride, a->H, a->v_head_stride, a->dv, es));
  r[3] = range("g", a->g, (size_t)(a->flags & KDA_LIN_FIXED_DECAY ? 1 : tok) * a->H * dsize(a->gate_dtype));
}

template <typename Args>
kda::LinPlan lin_plan(const Args* a) {
  kda::LinPlan p{};
  p.Hk = a->Hk, p.H = a->H, p.dk = a->dk, p.dv = a->dv;
  p.act_bf16 = a->act_dtype == KDA_BF16;
  p.gate_bf16 = a->gate_dtype == KDA_BF16;
  p.out_bf16 = a->out_dtype == KDA_BF16;
  p.fixed = (a->flags & KDA_LIN_FIXED_DECAY) != 0;
  p.q = static_cast<const char*>(a->q);
  p.k = static_cast<const char*>(a->k);
  p.v = static_cast<const char*>(a->v);
  const int64_t es = (int64_t)dsize(a->act_dtype);
  p.q_token = a->q_token_stride * es, p.q_head = a->q_head_stride * es;
  p.k_token = a->k_token_stride * es, p.k_head = a->k_head_stride * es;
  p.v_token = a->v_token_stride * es, p.v_head = a->v_head_stride * es;
  p.g = a->g;
  p.scale = a->scale;
  p.o = a->o;
  return p;
}

kda_status validate_lin_chunk(const kda_lin_chunk_args* a, kda::LinPlan* p, size_t* ws) {
  if (!a) return fail(KDA_ERR_NULL_PTR, "args is NULL");
  if (a->B < 1 || a->T < 0) return fail(KDA_ERR_BAD_SHAPE, "need B >= 1, T >= 0 (got B=%d T=%d)", a->B, a->T);
  if (a->cu_seqlens && (a->B != 1 || a->N < 1))
    return fail(KDA_ERR_BAD_SHAPE, "cu_seqlens requires B == 1 and N >= 1 (got B=%d N=%d)", a->B, a->N);
  const kda_status s = validate_lin(a);
  if (s != KDA_OK) return s;
  const int64_t tok = (int64_t)a->B * a->T, n_seq = a->cu_seqlens ? a->N : a->B;
  // a segment holds 64 tokens or more, and each has a workgroup per head
  if (tok * a->H > (int64_t(1) << 33) || (tok / 64 + n_seq) * a->H > kMaxDecodePairs)
    return fail(KDA_ERR_BAD_SHAPE, "too many tokens, sequences or heads for one launch");
  *p = lin_plan(a);
  p->n_seq = (int)n_seq;
  p->T = a->T;
  p->cu_seqlens = a->cu_seqlens;
  *ws = kda::plan_lin_chunk(p);
  return KDA_OK;
}

kda_status lin_decode(const char* name, const kda_lin_decode_args* a, bool step, void* hip_stream) {
  if (!a) return fail(KDA_ERR_NULL_PTR, "args is NULL");
  if (a->N < 1 || a->m < 1) return fail(KDA_ERR_BAD_SHAPE, "need N, m >= 1 (got N=%d m=%d)", a->N, a->m);
  if (step && (a->m != 1 || a->accept))
    return fail(KDA_ERR_UNSUPPORTED, "kda_lin_decode_step takes one token and no accept (got m=%d)", a->m);
  kda_status s = validate_lin(a);
  if (s != KDA_OK) return s;
  const int64_t tok = (int64_t)a->N * a->m;
  if ((int64_t)a->N * a->H > kMaxDecodePairs || tok * a->H > (int64_t(1) << 33))
    return fail(KDA_ERR_BAD_SHAPE, "N * H or N * m * H too large for one launch");
  if (!a->q || !a->k || !a->v || !a->g || !a->S || (step && !a->o))
    return fail(KDA_ERR_NULL_PTR, "q, k, v, g, S%s must be non-NULL", step ? " and o" : "");
  s = validate_lin_rows(a, tok);
  if (s != KDA_OK) return s;
  if (!aligned16(a->S)) return fail(KDA_ERR_BAD_SHAPE, "S must be 16-byte aligned");
  Range in[5];
  lin_inputs(a, tok, in);
  in[4] = range("accept", a->accept, a->accept ? sizeof(int32_t) * (size_t)a->N : 0);
  const Range S = range("S", a->S, (size_t)a->N * a->H * a->dk * a->dv * 4);
  const Range o = range("o", a->o, a->o ? (size_t)tok * a->H * a->dv * dsize(a->out_dtype) : 0);
  for (const Range& r : in) {
    if (overlap(o, r)) return fail(KDA_ERR_ALIAS, "o overlaps %s", r.name);
    if (overlap(S, r)) return fail(KDA_ERR_ALIAS, "S overlaps %s", r.name);
  }
  if (overlap(S, o)) return fail(KDA_ERR_ALIAS, "S overlaps o");
  if (!a->o && !a->accept) return ok();
  kda::LinPlan p = lin_plan(a);
  p.n_seq = a->N;
  p.T = a->m;
  p.S0 = a->S;
  p.S_T = step || a->accept ? a->S : nullptr;
  p.accept = a->accept;
  const hipError_t e = kda::launch_lin_recurrent(p, static_cast<hipStream_t>(hip_stream));
  if (e != hipSuccess) return fail(KDA_ERR_HIP, "%s launch: %s", name, hipGetErrorString(e));
  return ok();
}

kda_status validate_logits(const kda_logits_args* a) {
  if (!a) return fail(KDA_ERR_NULL_PTR, "args is NULL");
  if (a->N < 1 || a->R < 1 || a->V < 1)
    return fail(KDA_ERR_BAD_SHAPE, "need N, R, V >= 1 (got N=%d R=%d V=%d)", a->N, a->R, a->V);
  if (!dtype_ok(a->dtype) || !dtype_ok(a->out_dtype)) return fail(KDA_ERR_BAD_DTYPE, "unknown dtype");
  if (a->flags & ~KDA_LOGITS_PROBS) return fail(KDA_ERR_UNSUPPORTED, "unknown flags 0x%x", a->flags);
  if (a->V > (1 << 30)) return fail(KDA_ERR_BAD_SHAPE, "V too large (got %d)", a->V);
  // one 256-work-item workgroup per (sequence, row, block of 1,024 tokens or more)
  if (a->R > (1 << 24) || (int64_t)a->N * a->R > kMaxDecodePairs ||
      (int64_t)a->N * a->R * (((int64_t)a->V + 1023) / 1024) > kMaxDecodePairs)
    return fail(KDA_ERR_BAD_SHAPE, "N * R * V too large for one launch");
  return KDA_OK;
}

}  // namespace

extern "C" {

size_t kda_lin_chunk_fwd_workspace_bytes(const kda_lin_chunk_args* a) {
  kda::LinPlan p;
  size_t ws = 0;
  if (validate_lin_chunk(a, &p, &ws) != KDA_OK) return SIZE_MAX;
  ok();
  return ws;
}

kda_status kda_lin_chunk_fwd(const kda_lin_chunk_args* a, void* hip_stream) {
  kda::LinPlan p;
  size_t need = 0;
  kda_status s = validate_lin_chunk(a, &p, &need);
  if (s != KDA_OK) return s;
  const int64_t tok = (int64_t)a->B * a->T;
  if (tok > 0 && (!a->q || !a->k || !a->v || !a->g || !a->o))
    return fail(KDA_ERR_NULL_PTR, "q, k, v, g and o must be non-NULL");
  s = validate_lin_rows(a, tok);
  if (s != KDA_OK) return s;
  // a chunk's 64 rows lie within 2^32 bytes
  if (std::max({a->q_token_stride, a->k_token_stride, a->v_token_stride}) * (int64_t)dsize(a->act_dtype) >= (1 << 26))
    return fail(KDA_ERR_BAD_SHAPE, "token strides of q, k and v must be below 2^26 bytes");
  if (!aligned16(a->S0) || !aligned16(a->S_T))
    return fail(KDA_ERR_BAD_SHAPE, "S0 and S_T must be 16-byte aligned");
  if (need && (!a->workspace || a->workspace_bytes < need))
    return fail(KDA_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need,
                a->workspace ? a->workspace_bytes : (size_t)0);
  if (reinterpret_cast<uintptr_t>(a->workspace) % 256)
    return fail(KDA_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  const size_t state = (size_t)p.n_seq * a->H * a->dk * a->dv * 4;
  Range in[6];
  lin_inputs(a, tok, in);
  if (tok == 0)
    for (int i = 0; i < 4; ++i) in[i].hi = in[i].lo;
  in[4] = range("S0", a->S0, a->S0 ? state : 0);
  in[5] = range("cu_seqlens", a->cu_seqlens, a->cu_seqlens ? sizeof(int32_t) * ((size_t)a->N + 1) : 0);
  const Range out[] = {range("o", a->o, (size_t)tok * a->H * a->dv * dsize(a->out_dtype)),
                       range("S_T", a->S_T, a->S_T ? state : 0), range("workspace", a->workspace, need)};
  for (const Range& w : out)
    for (const Range& r : in)
      if (overlap(w, r) && !(&w == &out[1] && &r == &in[4] && a->S_T == a->S0))
        return fail(KDA_ERR_ALIAS, "%s overlaps %s", w.name, r.name);
  if (overlap(out[0], out[1]) || overlap(out[0], out[2]) || overlap(out[1], out[2]))
    return fail(KDA_ERR_ALIAS, "o, S_T and workspace must not overlap");
  p.S0 = a->S0;
  p.S_T = a->S_T;
  p.workspace = a->workspace;
  const hipError_t e = kda::launch_lin_chunk(p, static_cast<hipStream_t>(hip_stream));
  if (e != hipSuccess) return fail(KDA_ERR_HIP, "kda_lin_chunk_fwd launch: %s", hipGetErrorString(e));
  return ok();
}

kda_status kda_lin_decode_step(const kda_lin_decode_args* a, void* hip_stream) {
  return lin_decode("kda_lin_decode_step", a, true, hip_stream);
}

kda_status kda_lin_decode_multi(const kda_lin_decode_args* a, void* hip_stream) {
  return lin_decode("kda_lin_decode_multi", a, false, hip_stream);
}

kda_status kda_page_plan(const kda_page_plan_args* a, void* hip_stream) {
  if (!a) return fail(KDA_ERR_NULL_PTR, "args is NULL");
  if (a->N < 1 || a->page_size < 1 || a->max_pages < 1 || a->max_tokens < 1 || a->free_capacity < 1)
    return fail(KDA_ERR_BAD_SHAPE,
                "need N, page_size, max_pages, max_tokens, free_capacity >= 1 (got %d, %d, %d, %d, %d)", a->N,
                a->page_size, a->max_pages, a->max_tokens, a->free_capacity);
  if (a->table_stride < a->max_pages || a->table_stride > kMaxStride / 4)
    return fail(KDA_ERR_BAD_SHAPE, "table_stride must be >= max_pages");
  if ((double)a->N * (double)a->table_stride > 0x1p58) return fail(KDA_ERR_BAD_SHAPE, "block_table too large");
  if (a->N > (1 << 30)) return fail(KDA_ERR_BAD_SHAPE, "N too large (got %d)", a->N);
  if (!a->block_table || !a->held || !a->lens || !a->new_lens || !a->free_pages || !a->ring || !a->held_out ||
      !a->ring_out || !a->seq_lens || !a->cu_seqlens)
    return fail(KDA_ERR_NULL_PTR, "every array but slots and positions must be non-NULL");
  const size_t n = sizeof(int32_t) * (size_t)a->N;
  const Range in[] = {range("held", a->held, n), range("lens", a->lens, n), range("new_lens", a->new_lens, n),
                      range("ring", a->ring, 2 * sizeof(int32_t))};
  const Range out[] = {
      range("block_table", a->block_table,
            sizeof(int32_t) * ((size_t)(a->N - 1) * a->table_stride + a->max_pages)),
      range("free_pages", a->free_pages, sizeof(int32_t) * (size_t)a->free_capacity),
      range("held_out", a->held_out, n), range("ring_out", a->ring_out, 2 * sizeof(int32_t)),
      range("seq_lens", a->seq_lens, n), range("cu_seqlens", a->cu_seqlens, n + sizeof(int32_t)),
      range("slots", a->slots, a->slots ? sizeof(int64_t) * (size_t)a->max_tokens : 0),
      range("positions", a->positions, a->positions ? sizeof(int32_t) * (size_t)a->max_tokens : 0)};
  for (const Range& w : out) {
    for (const Range& r : in)
      if (overlap(w, r)) return fail(KDA_ERR_ALIAS, "%s overlaps %s", w.name, r.name);
    for (const Range& r : out)
      if (&r != &w && overlap(w, r)) return fail(KDA_ERR_ALIAS, "%s overlaps %s", w.name, r.name);
  }
  const kda::PagePlan p{a->N, a->page_size, a->max_pages, a->max_tokens, a->free_capacity, a->block_table,
                        a->table_stride, a->held, a->lens, a->new_lens, a->free_pages, a->ring, a->held_out,
                        a->ring_out, a->seq_lens, a->cu_seqlens, a->slots, a->positions};
  const hipError_t e = kda::launch_page_plan(p, static_cast<hipStream_t>(hip_stream));
  if (e != hipSuccess) return fail(KDA_ERR_HIP, "kda_page_plan launch: %s", hipGetErrorString(e));
  return ok();
}

size_t kda_adjust_logits_workspace_bytes(const kda_logits_args* a) {
  if (validate_logits(a) != KDA_OK) return SIZE_MAX;
  ok();
  return a->flags & KDA_LOGITS_PROBS ? kda::logits_workspace_bytes(a->N, a->R, a->V) : 0;
}

kda_status kda_adjust_logits(const kda_logits_args* a, void* hip_stream) {
  const kda_status s = validate_logits(a);
  if (s != KDA_OK) return s;
  if (!a->logits || !a->out) return fail(KDA_ERR_NULL_PTR, "logits and out must be non-NULL");
  if (a->history ? a->max_history < 1 || !a->history_lens : a->prompt_lens || a->history_lens)
    return fail(KDA_ERR_NULL_PTR, "history goes with history_lens and max_history >= 1; prompt_lens needs it");
  if ((a->bias_ids != nullptr) != (a->bias != nullptr) || (a->bias_ids ? a->max_bias < 1 : a->bias_counts != nullptr))
    return fail(KDA_ERR_NULL_PTR, "bias_ids and bias go together, with max_bias >= 1; bias_counts needs them");
  if (a->history && (a->max_history > (1 << 30) || (a->history_stride && a->history_stride < a->max_history)))
    return fail(KDA_ERR_BAD_SHAPE, "max_history must be at most 2^30, history_stride no less than it, or 0");
  if (a->drafts && a->R < 2) return fail(KDA_ERR_BAD_SHAPE, "drafts need R >= 2 (got %d)", a->R);
  const int64_t most = int64_t(1) << 42;  // elements: keeps every offset below 2^63
  auto rows_ok = [&](int64_t seq, int64_t row) {
    return row >= 0 && seq >= 0 && row <= most && seq <= most &&
           (double)(a->N - 1) * (double)seq + (double)(a->R - 1) * (double)row < 0x1p58;
  };
  if (!rows_ok(a->seq_stride, a->row_stride) || !rows_ok(a->out_seq_stride, a->out_row_stride) ||
      (a->mask && !rows_ok(a->mask_seq_stride, a->mask_row_stride)) ||
      (a->history && (a->history_stride > most || (double)a->N * (double)a->history_stride > 0x1p58)))
    return fail(KDA_ERR_BAD_SHAPE, "strides must be >= 0 and in range");
  // rows that are written lie apart: rows of a sequence inside its stride, or sequences inside a row's
  const int64_t V = a->V, seq = a->out_seq_stride, row = a->out_row_stride;
  const bool apart = (a->R == 1 || row >= V) && (a->N == 1 || seq >= V) &&
                     (a->R == 1 || a->N == 1 || seq >= (a->R - 1) * row + V || row >= (a->N - 1) * seq + V);
  if (!apart) return fail(KDA_ERR_BAD_SHAPE, "rows of out overlap");
  auto bytes = [&](int64_t s0, int64_t s1, int64_t width, size_t es) {
    return (size_t)((a->N - 1) * s0 + (a->R - 1) * s1 + width) * es;
  };
  const size_t need = a->flags & KDA_LOGITS_PROBS ? kda::logits_workspace_bytes(a->N, a->R, a->V) : 0;
  if (need && (!a->workspace || a->workspace_bytes < need))
    return fail(KDA_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need,
                a->workspace ? a->workspace_bytes : (size_t)0);
  if (reinterpret_cast<uintptr_t>(a->workspace) % 256)
    return fail(KDA_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  const size_t n4 = 4 * (size_t)a->N;
  const Range in[] = {
      range("logits", a->logits, bytes(a->seq_stride, a->row_stride, V, dsize(a->dtype))),
      range("history", a->history, a->history ? 4 * (size_t)((a->N - 1) * a->history_stride + a->max_history) : 0),
      range("history_lens", a->history_lens, a->history_lens ? n4 : 0),
      range("prompt_lens", a->prompt_lens, a->prompt_lens ? n4 : 0),
      range("drafts", a->drafts, a->drafts ? n4 * (a->R - 1) : 0),
      range("repetition", a->repetition, a->repetition ? n4 : 0),
      range("frequency", a->frequency, a->frequency ? n4 : 0),
      range("presence", a->presence, a->presence ? n4 : 0),
      range("bias_ids", a->bias_ids, a->bias_ids ? n4 * a->max_bias : 0),
      range("bias", a->bias, a->bias ? n4 * a->max_bias : 0),
      range("bias_counts", a->bias_counts, a->bias_counts ? n4 : 0),
      range("mask", a->mask, a->mask ? bytes(a->mask_seq_stride, a->mask_row_stride, (V + 31) / 32, 4) : 0),
      range("temperature", a->temperature, a->temperature ? n4 : 0)};
  const Range out = range("out", a->out, bytes(seq, row, V, dsize(a->out_dtype)));
  const Range ws = range("workspace", a->workspace, need);
  const bool in_place = a->out == a->logits && a->out_dtype == a->dtype && (a->N == 1 || seq == a->seq_stride) &&
                        (a->R == 1 || row == a->row_stride);
  for (const Range& r : in) {
    if (overlap(out, r) && !(&r == &in[0] && in_place)) return fail(KDA_ERR_ALIAS, "out overlaps %s", r.name);
    if (overlap(ws, r)) return fail(KDA_ERR_ALIAS, "workspace overlaps %s", r.name);
  }
  if (overlap(ws, out)) return fail(KDA_ERR_ALIAS, "workspace overlaps out");
  kda::LogitsPlan p{};
  p.N = a->N, p.R = a->R, p.V = a->V;
  p.bf16 = a->dtype == KDA_BF16;
  p.out_bf16 = a->out_dtype == KDA_BF16;
  p.probs = (a->flags & KDA_LOGITS_PROBS) != 0;
  p.logits = a->logits, p.seq = a->seq_stride, p.row = a->row_stride;
  p.out = a->out, p.out_seq = seq, p.out_row = row;
  p.history = a->history, p.history_stride = a->history_stride, p.max_history = a->max_history;
  p.history_lens = a->history_lens, p.prompt_lens = a->prompt_lens, p.drafts = a->drafts;
  p.repetition = a->repetition, p.frequency = a->frequency, p.presence = a->presence;
  p.bias_ids = a->bias_ids, p.bias = a->bias, p.bias_counts = a->bias_counts, p.max_bias = a->max_bias;
  p.mask = a->mask, p.mask_seq = a->mask_seq_stride, p.mask_row = a->mask_row_stride;
  p.temperature = a->temperature;
  p.workspace = a->workspace;
  const hipError_t e = kda::launch_logits(p, static_cast<hipStream_t>(hip_stream));
  if (e != hipSuccess) return fail(KDA_ERR_HIP, "kda_adjust_logits launch: %s", hipGetErrorString(e));
  return ok();
}

}  // extern "C"
