/* libkda: Kimi Delta Attention (KDA) on AMD MI355X (gfx950). C ABI.
 *
 * KDA is the fixed-size-state linear-attention layer of Kimi K3 (the "Sequenz" section of
 * the orkas.ai Kimi K3 architecture page: a running state of fixed size that decays, so
 * newer tokens weigh more). Per (sequence, head) the state S is a dk x dv fp32 matrix,
 * rows indexed by key channel, and each token t does
 *
 *     S <- Diag(exp(g_t)) S;   u = v_t - S^T k_t;   S <- S + beta_t k_t u^T;   o_t = S^T q_t
 *
 * i.e. the incoming state goes through a token-dependent transition before the write,
 * which is why per-device states cannot simply be summed (same page, section
 * "Die Rechnung landet in der Bereitstellungsinfrastruktur").
 *
 * Two core calls (decode_multi and the calls for the layers beside KDA are declared below):
 *   kda_chunk_fwd    - prefill: the whole sequence(s), chunkwise parallel. Chunks are split
 *                      into 16-token tiles whose cumulative log-decay stays in [-80, 0]
 *                      because each step's log-decay is >= -5 (section "Eine Untergrenze,
 *                      die einen GPU-Codepfad beseitigte"), so the diagonal tiles use the
 *                      same dense matrix products as all the others.
 *   kda_decode_step  - one new token per sequence; the state is updated in place and the
 *                      work does not grow with the context (studioglobal.ai Kimi K3 pages,
 *                      "KDA haandterer den vedvarende sekvensbehandling" and "Architektur fuer
 *                      lange Kontexte und guenstigeres Decoding"; orkas.ai infrastructure
 *                      section: the state is updated in place).
 *
 * Conventions shared by every call
 *   - Pointers named q, k, v, g, beta, o, S0, S_T, S, workspace, cu_seqlens are DEVICE
 *     pointers (hipMalloc'ed or torch tensors); argument structs live in host memory.
 *   - The caller allocates and owns every buffer it passes. The library allocates no device
 *     memory; its only device memory is the fixed scratch array of kda_chunk_fwd_noalloc
 *     (below). Its only other global state is a per-thread error string and, per device, the
 *     looked-up address of that array; every call is thread safe except that concurrent
 *     kda_chunk_fwd_noalloc calls on one GPU share the array.
 *   - Sizes whose kernels would need more than 2^32 - 1 work-items in one launch are refused
 *     with KDA_ERR_BAD_SHAPE.
 *   - Every call validates its arguments on the host, before any launch, and returns a
 *     kda_status. On failure nothing has been enqueued and kda_last_error() describes why.
 *   - Work is enqueued on the caller's HIP stream (NULL = the default stream) and the call
 *     returns without synchronising. Launch failures are reported as KDA_ERR_HIP.
 *   - Nothing is printed and no exception crosses the ABI.
 *   - Preconditions not checked by default: g in [-5, 0], beta in [0, 1], q and k rows of
 *     unit L2 norm. With the environment variable KDA_CHECK=1, kda_chunk_fwd, kda_decode_step
 *     and kda_decode_multi first run a device check of g and beta, synchronise the stream and
 *     return KDA_ERR_DECAY_RANGE if any value is outside its range. The check keeps its
 *     counters in the call's output buffer o (overwritten by the call afterwards; o overlaps
 *     no input), so it allocates nothing; kda_decode_multi without o then returns
 *     KDA_ERR_UNSUPPORTED. Nothing is clamped.
 *   - When a call returns an error after enqueueing work (KDA_ERR_HIP, KDA_ERR_DECAY_RANGE),
 *     the contents of its outputs are unspecified.
 *   - Layout: token-major, [B, T, H, d] contiguous (d fastest). States [n_seq, H, dk, dv]
 *     fp32 row-major (key channel rows, value channel columns).
 */
#ifndef KDA_H
#define KDA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define KDA_ABI_VERSION 4

typedef enum {
    KDA_OK = 0,
    KDA_ERR_NULL_PTR = 1,     /* a required pointer is NULL */
    KDA_ERR_BAD_SHAPE = 2,    /* sizes out of range or inconsistent */
    KDA_ERR_BAD_DTYPE = 3,    /* dtype combination not offered */
    KDA_ERR_UNSUPPORTED = 4,  /* valid request the library does not implement */
    KDA_ERR_DECAY_RANGE = 5,  /* KDA_CHECK=1 found g outside [-5, 0] or beta outside [0, 1] */
    KDA_ERR_WORKSPACE = 6,    /* workspace missing or smaller than kda_chunk_fwd_workspace_bytes() */
    KDA_ERR_HIP = 7,          /* a HIP runtime call or kernel launch failed */
    KDA_ERR_ALIAS = 8         /* an output overlaps an input it must not overlap */
} kda_status;

/* KDA_F8E4M3 (OCP e4m3, largest value 448) is offered for paged caches only (kda_page_cache). */
typedef enum { KDA_F32 = 0, KDA_BF16 = 1, KDA_F8E4M3 = 2 } kda_dtype;

/* Arguments of kda_chunk_fwd (prefill).
 *
 *   B, T       dense batch: B sequences of T tokens each. With cu_seqlens: B must be 1 and
 *              T is the packed total length. T = 0 is allowed: no token is read or written
 *              (q, k, v, g, beta and o may then be NULL) and S_T receives S0 (zeros if NULL).
 *   H          heads (independent).
 *   dk, dv     key and value head dims, each in {32, 64, 128}.
 *   chunk      chunk length in {16, 32, 64}; a performance knob (results agree across
 *              chunk lengths to rounding). Each chunk is processed as 16-token tiles.
 *   cu_seqlens device int32 [N + 1], token offsets of N packed sequences (0 = cu[0] <= ...
 *              <= cu[N] = T), or NULL for the dense batch. Chunks never straddle a sequence
 *              boundary and each sequence starts from its own S0[n].
 *   N          number of packed sequences (ignored when cu_seqlens is NULL; n_seq = B then).
 *   act_dtype  dtype of q, k, v.   gate_dtype  dtype of g, beta.   out_dtype  dtype of o.
 *              Offered: act = gate = BF16 or act = gate = F32; out F32 or BF16.
 *   q, k, g    [B, T, H, dk];  v [B, T, H, dv];  beta [B, T, H].  Read only.
 *              g is the natural-log per-step decay of each key channel, beta the write
 *              strength.
 *   S0         [n_seq, H, dk, dv] fp32 initial states, or NULL for zeros.
 *   o          [B, T, H, dv] out_dtype. Written. Must not overlap any input.
 *   S_T        [n_seq, H, dk, dv] fp32 final states, or NULL. May be the same buffer as S0
 *              (continue in place); must not partially overlap it.
 *   workspace  device scratch of at least kda_chunk_fwd_workspace_bytes() bytes (may be NULL
 *              when that is 0), 256-byte aligned; contents on entry are ignored.
 *   flags      0, or any of:
 *              KDA_FLAG_GENERIC to force the fp32 vector-ALU path (needs no workspace; slower;
 *              used to cross-check the matrix-core path);
 *              KDA_FLAG_PAIRWISE_DIAG to evaluate the diagonal 16-token tiles of the
 *              matrix-core path pairwise (each e^{G_r - G_j} per pair and key channel, fp32, on
 *              the vector ALUs) as the earlier generation did, instead of by the dense product
 *              that the decay bound makes possible (orkas.ai Kimi K3 page, "Eine Untergrenze, die
 *              einen GPU-Codepfad beseitigte"). It needs no lower bound on g (any g <= 0) and is
 *              slower: the ablation of that bound. (KDA_CHECK=1 still checks g >= -5.)
 *              KDA_FLAG_WALK64 / KDA_FLAG_WALK128 to make the matrix-core path's serial walk
 *              over the chunks take one 64-token chunk per step, or two consecutive chunks
 *              composed into one 128-token step (S -> S + Z + Psi S for the pair, formed in
 *              parallel beforehand). Performance knobs (results agree to rounding): composing
 *              halves the serial steps and the workspace bytes per token, at about 30 % more
 *              parallel work. Without either flag the library composes when there are at most
 *              8 (sequence, head) pairs (where the serial walk dominates). One chunk per step is
 *              always taken when ckpt_every is not a multiple of 128, since checkpoints are
 *              taken between steps (KDA_FLAG_WALK128 is then refused); the workspace size
 *              depends on ckpt_every, so query it with the same value.
 *   ckpt, ckpt_every, ckpt_slots
 *              Sparse state checkpoints for prefix reuse: the fixed-size state is the whole
 *              memory of a prefix, so a later request that shares the prefix can resume from
 *              a stored state instead of recomputing it (orkas.ai Kimi K3 page, the
 *              serving-infrastructure section on per-request state). ckpt_every = 0 writes
 *              none (ckpt and ckpt_slots are then ignored). Otherwise ckpt_every is a positive
 *              multiple of chunk, and ckpt is fp32 [ckpt_slots, H, dk, dv]: checkpoint j >= 1
 *              of sequence n is its state after its first j * ckpt_every tokens (for every j
 *              with j * ckpt_every <= len_n), stored in slot
 *                  sum_{m < n} floor(len_m / ckpt_every) + j - 1.
 *              Slots at or past ckpt_slots are not written (a caller that allocates
 *              sum_n floor(len_n / ckpt_every) slots gets every checkpoint; that sum is at
 *              most floor(B * T / ckpt_every)). ckpt must not overlap any input, o, S_T or
 *              the workspace.
 *   segments   0, 1 or 2: every sequence is walked chunk after chunk (the default). 3 .. 8:
 *              the matrix-core path cuts each sequence into that many segments and walks them
 *              in parallel with the transition form of a segment, S_exit = Phi S_entry + Z
 *              (orkas.ai Kimi K3 page, serving-infrastructure section on splitting a sequence):
 *              one pass computes every middle segment's transition Phi and zero-start summary
 *              Z alongside the first segment, the entries follow in order from those, and a
 *              second pass walks the remaining segments from their entries. It trades about
 *              twice the recurrence work for more parallelism, which pays when few (sequence,
 *              head) pairs leave the GPU idle. The result equals the sequential walk to
 *              rounding; the workspace grows by (3 segments - 5) state-sized buffers. Other
 *              paths ignore it.
 */
typedef struct {
    int B, T, H, dk, dv, chunk;
    const int32_t* cu_seqlens;
    int N;
    kda_dtype act_dtype, gate_dtype, out_dtype;
    const void *q, *k, *v, *g, *beta;
    const float* S0;
    void* o;
    float* S_T;
    void* workspace;
    size_t workspace_bytes;
    unsigned flags;
    float* ckpt;
    int ckpt_every;
    int ckpt_slots;
    int segments;
} kda_chunk_args;

#define KDA_FLAG_GENERIC 1u
#define KDA_FLAG_PAIRWISE_DIAG 2u
#define KDA_FLAG_WALK64 4u
#define KDA_FLAG_WALK128 8u

/* Arguments of kda_decode_step: one token for each of N independent sequences.
 *   q, k, g [N, H, dk];  v [N, H, dv];  beta [N, H]   (act_dtype / gate_dtype as above)
 *   S       [N, H, dk, dv] fp32, read and updated in place.
 *   o       [N, H, dv] out_dtype, the output of the new token (read after the update).
 */
typedef struct {
    int N, H, dk, dv;
    kda_dtype act_dtype, gate_dtype, out_dtype;
    const void *q, *k, *v, *g, *beta;
    float* S;
    void* o;
} kda_decode_args;

/* Arguments of kda_decode_multi: m tokens for each of N independent sequences, evaluated
 * from one read of the state. It serves speculative decoding, which must evaluate draft
 * tokens without committing them and then commit the accepted prefix (orkas.ai Kimi K3
 * page, serving-infrastructure section on speculative decoding and in-place state).
 *   m       tokens per sequence, >= 1.
 *   q, k, g [N, m, H, dk];  v [N, m, H, dv];  beta [N, m, H]: token j of sequence n at [n, j].
 *   S       [N, H, dk, dv] fp32. Token j sees the state after tokens 0..j-1 of its sequence.
 *   o       [N, m, H, dv] out_dtype, every token's output (read after its update); or NULL.
 *   accept  device int32 [N], or NULL. NULL: S is left unchanged (verification). Otherwise
 *           S[n] becomes the state after the first clamp(accept[n], 0, m) tokens (commit;
 *           0 leaves S[n] unchanged). A verify call followed by a commit call with the same
 *           inputs replays the accepted tokens; o of the two calls agree bitwise.
 *   Inputs and accept must not overlap S or o; S and o must not overlap.
 */
typedef struct {
    int N, H, dk, dv, m;
    kda_dtype act_dtype, gate_dtype, out_dtype;
    const void *q, *k, *v, *g, *beta;
    float* S;
    void* o;
    const int32_t* accept;
} kda_decode_multi_args;

/* Bytes of device workspace kda_chunk_fwd needs for these arguments (pointers are not
 * inspected); 0 when the chosen path needs none. Validates shapes and dtypes like
 * kda_chunk_fwd and returns SIZE_MAX (with kda_last_error() set) when they are invalid.
 * The matrix-core path needs one 114,688-byte block per 64-token chunk and head when it walks
 * one chunk per step, or one 163,840-byte block per 128 tokens (two chunks) and head when it
 * composes two per step, plus small tables. */
size_t kda_chunk_fwd_workspace_bytes(const kda_chunk_args* args);

/* Prefill: o and S_T from q, k, v, g, beta and S0, enqueued on hip_stream (hipStream_t). */
kda_status kda_chunk_fwd(const kda_chunk_args* args, void* hip_stream);

/* Prefill without a workspace, for callers that cannot allocate device memory (code under
 * HIP graph capture, tight serving loops, harnesses that forbid allocation). Same arguments
 * and results as kda_chunk_fwd, except that workspace and workspace_bytes are ignored: the
 * library's own fixed device scratch of KDA_NOALLOC_SCRATCH_BYTES takes the workspace's place.
 * That scratch is a static array of the library, held by every GPU the library runs on from
 * the first use there until the process ends. Calls whose kda_chunk_fwd_workspace_bytes()
 * exceeds KDA_NOALLOC_SCRATCH_BYTES return KDA_ERR_WORKSPACE before anything is enqueued (at
 * most 1,170 (64-token chunk, head) pairs with one chunk per walk step, or 819 (128-token
 * block, head) pairs with composed steps; prefill-4k, 4,096 tokens with 16 heads, fits). No device
 * or host memory is allocated. All calls on one GPU share its scratch, whatever their stream:
 * calls that overlap in time on one GPU race (serialise them, e.g. on one stream). */
#define KDA_NOALLOC_SCRATCH_BYTES ((size_t)128 << 20)
kda_status kda_chunk_fwd_noalloc(const kda_chunk_args* args, void* hip_stream);

/* Decode: one step for every (sequence, head); S updated in place, o written. */
kda_status kda_decode_step(const kda_decode_args* args, void* hip_stream);

/* Decode, m tokens per sequence: outputs of all m, and optionally the commit of an accepted
 * prefix into S (see kda_decode_multi_args). With o and accept both NULL nothing is done. */
kda_status kda_decode_multi(const kda_decode_multi_args* args, void* hip_stream);

/* Device check of the preconditions on the gates: counts g values outside [-5, 0] and
 * beta values outside [0, 1] (NaN counts as outside); the floor of -5 is the bound on the
 * per-step log-decay (orkas.ai Kimi K3 page, "Eine Untergrenze, die einen GPU-Codepfad
 * beseitigte"). n_g, n_beta elements; dtype of both is gate_dtype.
 *   counts    caller-owned device scratch of n_counts int64 (n_counts >= 1; up to
 *             KDA_CHECK_COUNTERS of them are used, one per workgroup of the check, so
 *             KDA_CHECK_COUNTERS entries give the most parallel check). Must not overlap g or
 *             beta; its contents on return are unspecified.
 * Synchronises hip_stream; *n_bad receives the count. Allocates nothing. */
#define KDA_CHECK_COUNTERS 1024
kda_status kda_check_gates(const void* g, int64_t n_g, const void* beta, int64_t n_beta,
                           kda_dtype gate_dtype, int64_t* counts, int n_counts,
                           void* hip_stream, int64_t* n_bad);

/* ---- The other half of a serving step -------------------------------------------------
 *
 * A hybrid stack puts global attention layers between the KDA layers (three KDA layers to one;
 * orkas.ai Kimi K3 page, section "Sequenz"). Their memory grows with the context and is kept in
 * pages per token (same page, serving-infrastructure section). kda_kv_append fills such a paged
 * cache, kda_paged_decode attends to it for the new tokens, and kda_verify_drafts decides how
 * many drafted tokens stand, which is the `accept` of kda_decode_multi.
 *
 * Values that live on the device cannot be checked on the host. The three calls below read and
 * write nothing out of bounds whatever block tables, lengths, positions, counts and token ids
 * hold; what such a value means is said at its field.
 */

/* A paged key/value cache of one layer.
 *   k, v         num_pages pages of page_size tokens of Hkv heads of d channels each: element
 *                (page, slot, head, c) lies at page * page_stride + slot * token_stride +
 *                head * head_stride + c, strides in elements (>= 0). Pages with the token
 *                outermost or the head outermost, and k and v interleaved in one allocation, are
 *                all a matter of strides. k, v and every stride are multiples of 16 bytes.
 *   dtype        KDA_BF16 or KDA_F8E4M3 beside bf16 activations, KDA_F32 beside fp32 ones.
 *   page_size    tokens per page, >= 1. Multiples of 16 are read faster than others.
 *   block_table  device int32: page p of sequence n is block_table[n * table_stride + p],
 *                p < max_pages. Entries past a sequence's last page are not read. A page id
 *                outside [0, num_pages) is no page: nothing is written to it, and its tokens
 *                are seen by no query.
 *   k_scale, v_scale
 *                device fp32 [Hkv], or NULL for ones: a stored value times its head's scale is
 *                the value meant. Finite and positive. Only with KDA_F8E4M3 (NULL otherwise).
 */
typedef struct {
    void *k, *v;
    kda_dtype dtype;
    int num_pages, page_size;
    int64_t k_page_stride, k_token_stride, k_head_stride;
    int64_t v_page_stride, v_token_stride, v_head_stride;
    const int32_t* block_table;
    int64_t table_stride;
    int max_pages;
    const float *k_scale, *v_scale;
} kda_page_cache;

/* Arguments of kda_kv_append: new tokens' keys and values into a paged cache, rotated by
 * position on the way; queries rotated alongside.
 *   B, T, cu_seqlens, N
 *              dense batch of B sequences with T new tokens each, or packed sequences, as in
 *              kda_chunk_args (T = 0 is allowed; tokens at or past cu_seqlens[N] are left alone,
 *              their rows of q_out included). n_seq = B or N.
 *   Hq, Hkv, d heads of q and of k and v, channels per head: d in {32, 64, 128}.
 *   act_dtype  of q, k, v and q_out: KDA_F32 or KDA_BF16.
 *   q, k, v    [B, T, heads, d]: token t = b * T + j of head h begins at t * token_stride +
 *              h * head_stride (elements), so views of a fused projection can be passed. The
 *              pointers and strides are multiples of 16 bytes. q may be NULL.
 *   q_out      [B, T, Hq, d] contiguous, 16-byte aligned, NULL exactly if q is. May be q itself
 *              if q is contiguous; otherwise it overlaps no input.
 *   start      device int32 [n_seq]: tokens of each sequence in the cache so far. New token j
 *              has position start[n] + j, and goes to slot position % page_size of page
 *              position / page_size. Tokens whose position is negative, or at or past
 *              max_pages * page_size or 2^31, are not stored; their q_out is written all the
 *              same. Two new tokens must not go to the same slot of the same page.
 *   inv_freq   device fp32 [rot / 2], or NULL with rot = 0 (no rotation: k is stored and q
 *              copied as they are). Channel pair i < rot / 2 of a token at position p is turned
 *              by the angle p * inv_freq[i] (formed and reduced in 64 bits):
 *                  x' = x cos - y sin,   y' = y cos + x sin.
 *   rot        channels that turn, a multiple of 16, 0 <= rot <= d. Channels rot .. d - 1 stay.
 *   flags      0: pair i is channels (i, i + rot / 2). KDA_APPEND_PAIRS: (2i, 2i + 1).
 *   cache      where k and v go. With KDA_F8E4M3 a value is divided by its scale, limited to
 *              [-448, 448] and rounded to nearest even; NaN stays NaN. The k and v arrays
 *              overlap no other argument, and no two of their rows share elements.
 */
#define KDA_APPEND_PAIRS 1u
typedef struct {
    int B, T, Hq, Hkv, d;
    const int32_t* cu_seqlens;
    int N;
    kda_dtype act_dtype;
    const void *q, *k, *v;
    int64_t q_token_stride, q_head_stride, k_token_stride, k_head_stride;
    int64_t v_token_stride, v_head_stride;
    void* q_out;
    const int32_t* start;
    const float* inv_freq;
    int rot;
    unsigned flags;
    kda_page_cache cache;
} kda_kv_append_args;

/* Arguments of kda_paged_decode: attention of m new tokens of each of N sequences (m = 1: plain
 * decode; m drafts for speculative decoding) over a paged cache that already holds them.
 *   Hq, Hkv, d Hq is a multiple of Hkv: query head h reads key/value head h / (Hq / Hkv).
 *              d in {32, 64, 128}.
 *   act_dtype  of q: KDA_F32 or KDA_BF16.   out_dtype  of o, either.
 *   q          [N, m, Hq, d] by q_token_stride (from (n, j) to the next, n * m + j counted) and
 *              q_head_stride; 16-byte aligned like kda_kv_append's.
 *   seq_lens   device int32 [N]: tokens of each sequence in the cache, the new ones included.
 *              Values outside [0, max_len] are taken as the nearer bound.
 *   max_len    no length is larger; 1 <= max_len <= max_pages * page_size. The launch is shaped
 *              by it, so a tight one is faster; the result depends on it by rounding only.
 *   window     0, or the number of latest tokens that a query sees (its own included).
 *   scale      finite; o = softmax(scale * q k^T) v, scores in 32 bits (beyond 3.4e38 they are
 *              infinite). New token j of sequence n sees positions
 *              t < hi = seq_lens[n] - m + 1 + j, with a window t >= hi - window too. What it does
 *              not see does not reach it, NaN and infinities included; a value that it does
 *              see and that is not finite makes its channel of o infinite or NaN. If it sees
 *              none, its o is 0 and its lse -inf.
 *   o          [N, m, Hq, d] contiguous, out_dtype, 16-byte aligned.
 *   lse        fp32 [N, m, Hq], or NULL: natural logarithm of sum_t e^{scale q k_t} (for joining
 *              results over parts of a context).
 *   workspace  device scratch of at least kda_paged_decode_workspace_bytes() bytes, 256-byte
 *              aligned; contents on entry are ignored. (NULL when that is 0.) Calls that overlap
 *              in time need one each.
 *   flags      0.
 */
typedef struct {
    int N, m, Hq, Hkv, d;
    kda_dtype act_dtype, out_dtype;
    const void* q;
    int64_t q_token_stride, q_head_stride;
    kda_page_cache cache;
    const int32_t* seq_lens;
    int max_len, window;
    float scale;
    void* o;
    float* lse;
    void* workspace;
    size_t workspace_bytes;
    unsigned flags;
} kda_paged_decode_args;

/* Arguments of kda_verify_drafts: how many of m drafted tokens of each of N sequences stand
 * against the target model's probabilities, and the token that follows them, so that the
 * tokens are distributed as if drawn from the target alone.
 *   m, V       drafts per sequence (1 .. 2^24) and vocabulary size (1 .. 2^30).
 *   dtype      of p and q: KDA_F32 or KDA_BF16.
 *   p          target probabilities [N, m + 1, V]: row j of sequence n, for the token after j
 *              drafts, begins at n * p_seq_stride + j * p_row_stride (elements).
 *   q          probabilities the drafts were drawn from, [N, m, V] by its strides; or NULL if the
 *              drafts were picked, not drawn (looked up, or the most probable ones): q is then
 *              one at the draft and zero elsewhere.
 *   drafts     device int32 [N, m].   n_drafts  device int32 [N] or NULL: sequence n has only the
 *              first clamp(n_drafts[n], 0, m) drafts.
 *   uniform    device fp32 [N, m + 1], uniform random numbers in [0, 1) (values below 0 and NaN
 *              are taken as 0, values of 1 and above as the largest below 1). Draft j stands if
 *              those before it do and
 *                  uniform[n, j] * q_j(x_j) < p_j(x_j)
 *              (in 64 bits, where the product is exact). A draft outside [0, V), or
 *              whose p or q is not finite, does not stand.
 *              uniform[n, m] picks the token that follows.
 *   accept     int32 [N]: drafts that stand, a: the `accept` of a kda_decode_multi whose tokens
 *              are the drafts (a + 1 for one whose tokens are the last token and the drafts).
 *   tokens     int32 [N, m + 1]: the a drafts, then the following token, then -1. The following
 *              token is the smallest i with sum_{i' <= i} w_i' > uniform[n, m] * sum w (sums in
 *              64 bits, the same on every run), where w = max(p_a - q_a, 0) if a draft fell, and
 *              w = p_a if all stood or if no w is positive. Probabilities that are negative or
 *              not finite count as 0 in w. If p_a has nothing positive either, the token is -1.
 *   workspace  device scratch of at least kda_verify_drafts_workspace_bytes() bytes, 256-byte
 *              aligned; contents on entry are ignored. Calls that overlap in time need one each.
 */
typedef struct {
    int N, m, V;
    kda_dtype dtype;
    const void *p, *q;
    int64_t p_seq_stride, p_row_stride, q_seq_stride, q_row_stride;
    const int32_t *drafts, *n_drafts;
    const float* uniform;
    int32_t *accept, *tokens;
    void* workspace;
    size_t workspace_bytes;
} kda_verify_args;

/* New keys and values into a paged cache (see kda_kv_append_args). */
kda_status kda_kv_append(const kda_kv_append_args* args, void* hip_stream);

/* Attention of new tokens over a paged cache (see kda_paged_decode_args). The workspace query
 * looks at shapes, dtypes, max_len and window, not at pointers; SIZE_MAX when they are invalid. A
 * window or a smaller max_len never needs more: the size for window = 0 and the longest max_len
 * serves every call of otherwise the same shapes. */
size_t kda_paged_decode_workspace_bytes(const kda_paged_decode_args* args);
kda_status kda_paged_decode(const kda_paged_decode_args* args, void* hip_stream);

/* Verification of drafted tokens (see kda_verify_args). The workspace query looks at N, m, V and
 * dtype only; SIZE_MAX when they are invalid. */
size_t kda_verify_drafts_workspace_bytes(const kda_verify_args* args);
kda_status kda_verify_drafts(const kda_verify_args* args, void* hip_stream);

const char* kda_status_string(kda_status s);
const char* kda_last_error(void);   /* detail of the last failure on this thread */
int kda_abi_version(void);           /* KDA_ABI_VERSION of the built library */

#ifdef __cplusplus
}
#endif

#endif /* KDA_H */
