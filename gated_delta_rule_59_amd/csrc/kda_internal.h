// Host-side launch descriptions passed from the C ABI layer (kda_api.cpp) to the kernel
// launchers. Arguments are validated before a plan is built.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace kda {

struct DecodePlan {
  int N, H, dk, dv;
  bool act_bf16, out_bf16;
  const void *q, *k, *v, *g, *beta;
  float* S;
  void* o;
};

struct ChunkPlan {
  int B, T, H, dk, dv, chunk;
  const int32_t* cu_seqlens;  // device, or nullptr for a dense batch
  int n_seq;                  // B (dense) or N (packed)
  bool act_bf16, out_bf16;
  const void *q, *k, *v, *g, *beta;
  const float* S0;
  void* o;
  float* S_T;
  void* workspace;
  size_t workspace_bytes;
  float* ckpt;      // state checkpoints [ckpt_slots, H, dk, dv], or nullptr
  int ckpt_every;   // tokens between checkpoints (a multiple of chunk), 0 = none
  int ckpt_slots;
  bool pairwise_diag;  // matrix-core path: diagonal tiles pairwise (no decay bound needed)
  int segments;        // matrix-core path: walk each sequence in this many segments (>= 3), else 1
  int walk_block;      // matrix-core path: tokens per walk step, 64 (one chunk) or 128 (two
                       // chunks composed into one step)
};

hipError_t launch_decode(const DecodePlan& p, hipStream_t stream);

struct DecodeMultiPlan {
  int N, H, dk, dv, m;
  bool act_bf16, out_bf16;
  const void *q, *k, *v, *g, *beta;
  float* S;
  void* o;                // nullptr: outputs not written
  const int32_t* accept;  // nullptr: S not modified
};

hipError_t launch_decode_multi(const DecodeMultiPlan& p, hipStream_t stream);

// Generic path: fp32 arithmetic on the vector ALUs, any supported dk/dv/chunk; used for
// fp32 activations and for shapes the matrix-core path does not take.
hipError_t launch_chunk_generic(const ChunkPlan& p, hipStream_t stream);

// Matrix-core path: bf16 activations, dk = dv = 128, chunk = 64.
bool fast_path_applies(const ChunkPlan& p);
size_t fast_workspace_bytes(const ChunkPlan& p);
hipError_t launch_chunk_fast(const ChunkPlan& p, hipStream_t stream);

// Fixed device scratch of the allocation-free prefill entry point: its size, and its device
// address on the current device (looked up on the first call per device).
size_t noalloc_scratch_bytes();
hipError_t noalloc_scratch(void** ptr);

// n / d = (n * mul) >> shift for 0 <= n < 2^31, d >= 1: shift = 31 + ceil(log2 d) and mul =
// floor(2^shift / d) + 1, which is below 2^32.
inline void divide_by(int d, unsigned* mul, int* shift) {
  int up = 0;
  while ((int64_t(1) << up) < d) ++up;
  *shift = 31 + up;
  *mul = (unsigned)((uint64_t(1) << *shift) / (uint64_t)d + 1);
}

// A paged cache as the kernels take it (validated; strides in bytes).
struct PageCache {
  char *k, *v;
  int num_pages, page_size;
  unsigned ps_mul;  // token / page_size = (token * ps_mul) >> ps_shift for 0 <= token < 2^31
  int ps_shift;
  int64_t k_page, k_token, k_head, v_page, v_token, v_head;
  unsigned k_page16, v_page16;  // page strides in 16 bytes (where they fit)
  const int32_t* table;
  int64_t table_stride;
  int max_pages;
  const float *k_scale, *v_scale;
};

struct KvAppendPlan {
  int B, T, Hq, Hkv, d, rot, n_seq;
  const int32_t* cu_seqlens;
  bool act_bf16, pairs;
  int cache_type;                // a kda_dtype
  const char *q, *k, *v;         // strides in bytes
  int64_t q_token, q_head, k_token, k_head, v_token, v_head;
  char* q_out;
  const int32_t* start;
  const float* inv_freq;
  PageCache c;
};
hipError_t launch_kv_append(const KvAppendPlan& p, hipStream_t stream);

struct PagedDecodePlan {
  int N, m, Hq, Hkv, d;
  int group, rows;               // Hq / Hkv; m * group query rows per key/value head
  int row_blocks;                // blocks of 16 * tiles rows
  int tiles;                     // 16-row tiles a workgroup carries
  bool out_bf16;
  int cache_type;
  const char* q;                 // strides in bytes
  int64_t q_token, q_head;
  PageCache c;
  const int32_t* seq_lens;
  int max_len, window;
  float scale;
  void* o;
  float* lse;
  int heads, groups;             // neighbouring key/value heads a workgroup carries (1, 2 or 4),
                                 // Hkv / heads
  int unit_log;                  // log2 of the tokens that its waves take at a time
  unsigned group_mul;            // row / group = (row * group_mul) >> group_shift
  int group_shift;
  int split;                     // workgroups that share all work evenly; 0: one per (n, row
                                 // block, head group)
  int start;                     // units that beginning a group counts for (0 without split)
  int part_rows;                 // rows of a part
  int hold;                      // heads == 4: bytes of LDS in which a wave holds results back
  float *part_o, *part_ml;       // workspace: parts of shared groups, [split][2][heads][part_rows]
                                 // of d values, and of (maximum, sum)
  int* part_of;                  // [n][row block][head group]: first and last workgroup
};
// Fills in the launch shape (tiles to part_rows) and returns the workspace bytes; and the
// workspace's arrays.
size_t plan_paged_decode(PagedDecodePlan* p);
void paged_decode_workspace(PagedDecodePlan* p, void* workspace);
hipError_t launch_paged_decode(const PagedDecodePlan& p, hipStream_t stream);

struct VerifyPlan {
  int N, m, V;
  bool bf16;
  const void *p, *q;
  int64_t p_seq, p_row, q_seq, q_row;  // elements
  const int32_t *drafts, *n_drafts;
  const float* uniform;
  int32_t *accept, *tokens;
  void* workspace;
};
size_t verify_workspace_bytes(int N, int V);
hipError_t launch_verify(const VerifyPlan& p, hipStream_t stream);

// Device check of g in [-5, 0] and beta in [0, 1] over n_blocks workgroups (1 .. check_blocks());
// writes each workgroup's count of violations into counts[0 .. n_blocks).
int check_blocks();
hipError_t launch_check_gates(const void* g, int64_t n_g, const void* beta, int64_t n_beta,
                              bool bf16, int64_t* counts, int n_blocks, hipStream_t stream);

}  // namespace kda
