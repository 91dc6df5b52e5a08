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

/* ---- Around the layers of a step -------------------------------------------------------
 *
 * What the step of a hybrid stack needs beside the calls above: its layers whose state decays by
 * one number per head (kda_lin_*), the block tables and slots that its paged cache works by
 * (kda_page_plan), and the way from logits to the probabilities that kda_verify_drafts takes
 * (kda_adjust_logits). As above, values on the device cannot be checked on the host: nothing is
 * read or written out of bounds whatever lengths, counts, page ids and token ids hold.
 */

/* Linear attention with a decay for each head. Per (sequence, head) the state S is a dk x dv fp32
 * matrix, rows indexed by key channel, and each token t does
 *
 *     S <- exp(g_t) S + k_t v_t^T;   o_t = scale * S^T q_t
 *
 *   Hk, H      heads of q and k, and of v, g, S and o: H is a multiple of Hk, and head h reads
 *              query and key head h / (H / Hk).
 *   dk, dv     each in {32, 64, 128}.
 *   act_dtype  of q, k, v: KDA_F32 or KDA_BF16. gate_dtype of g, out_dtype of o: either. With
 *              KDA_BF16 activations products that need more than bf16 holds (states, weights, and
 *              values times decays) go in several bf16 parts. In prompts o is off by its own rounding
 *              and 2^-18 of its largest terms, S by 2^-18, beside what sums in 32
 *              bits are rounded by; a prompt of one chunk (64 tokens): 2^-20 each; terms that live
 *              through more than 384 tokens: 2^-21 more for each further 128.
 *   q, k, v    [B, T, heads, d] (decode: [N, m, heads, d]): token t = b * T + j of head h begins at
 *              t * token_stride + h * head_stride (elements), so views of a fused projection can be
 *              passed. Pointers and strides are multiples of 16 bytes (kda_lin_chunk_fwd: token
 *              strides below 2^26 bytes).
 *   g          natural logarithm of each token's decay, contiguous [B, T, H] (decode [N, m, H]); with
 *              KDA_LIN_FIXED_DECAY [H], the same for every token. -infinity is a decay of 0, which
 *              ends the memory of all earlier tokens. Values above 0 (growth) are taken as they are.
 *   scale      finite.
 *   flags      0 or KDA_LIN_FIXED_DECAY.
 *
 * States of more than 2^100 may become infinite in kda_lin_chunk_fwd before their formula does.
 * A value of q, k, v or g that is not finite reaches results of its own sequence and the heads that
 * read it only; in kda_lin_chunk_fwd, tokens up to 63 places before it too, in the decode calls
 * only its own token and later ones.
 */
#define KDA_LIN_FIXED_DECAY 1u

/* Arguments of kda_lin_chunk_fwd: whole prompts, chunkwise parallel.
 *   B, T, cu_seqlens, N
 *              dense batch or packed sequences, as in kda_chunk_args (T = 0 is allowed: S_T receives
 *              S0, zeros if NULL). Rows of o at or past cu_seqlens[N] are left as they were. Offsets
 *              outside [0, T] are taken as the nearer bound, and a sequence that ends before it begins
 *              has no tokens; where offsets give tokens to two sequences, results from the first of
 *              them on are unspecified.
 *   S0         [n_seq, H, dk, dv] fp32 initial states, or NULL for zeros.
 *   o          [B, T, H, dv] contiguous, out_dtype, 16-byte aligned. Overlaps no input.
 *   S_T        [n_seq, H, dk, dv] fp32 final states, or NULL. May be S0 itself (continue in place);
 *              does not overlap it in part. S0 and S_T are 16-byte aligned.
 *   workspace  device scratch of at least kda_lin_chunk_fwd_workspace_bytes() bytes, 256-byte
 *              aligned; contents on entry are ignored. (NULL when that is 0.) Calls that overlap in
 *              time need one each.
 */
typedef struct {
    int B, T, Hk, H, dk, dv;
    const int32_t* cu_seqlens;
    int N;
    kda_dtype act_dtype, gate_dtype, out_dtype;
    const void *q, *k, *v;
    int64_t q_token_stride, q_head_stride, k_token_stride, k_head_stride;
    int64_t v_token_stride, v_head_stride;
    const void* g;
    float scale;
    const float* S0;
    void* o;
    float* S_T;
    void* workspace;
    size_t workspace_bytes;
    unsigned flags;
} kda_lin_chunk_args;

/* Arguments of kda_lin_decode_step (m = 1, accept NULL: S is updated in place) and of
 * kda_lin_decode_multi (m >= 1 tokens of each of N sequences, S as in kda_decode_multi: unchanged
 * with accept NULL, else the state after the first clamp(accept[n], 0, m) tokens).
 *   S          [N, H, dk, dv] fp32, 16-byte aligned.
 *   o          [N, m, H, dv] contiguous, out_dtype, 16-byte aligned; kda_lin_decode_multi: or NULL.
 *              o of a call with accept and of one without agree bitwise.
 *   q, k, v, g and accept overlap neither S nor o, nor do these two each other.
 */
typedef struct {
    int N, m, Hk, H, dk, dv;
    kda_dtype act_dtype, gate_dtype, out_dtype;
    const void *q, *k, *v;
    int64_t q_token_stride, q_head_stride, k_token_stride, k_head_stride;
    int64_t v_token_stride, v_head_stride;
    const void* g;
    float scale;
    float* S;
    void* o;
    const int32_t* accept;
    unsigned flags;
} kda_lin_decode_args;

/* Arguments of kda_page_plan: pages for the new tokens of N sequences out of a ring of free ones, the
 * pages of ended sequences back into it, and everything that the layers of a step take: offsets,
 * lengths, positions and slots. Sequences are served in order. With pages_n = ceil((lens[n] +
 * new_lens[n]) / page_size):
 *   - a sequence with new_lens[n] < 0 has ended: its held[n] pages go back, and it holds none.
 *   - otherwise it asks for need_n = max(0, pages_n - held[n]) pages, unless pages_n > max_pages: then
 *     it is refused. It is refused too if it asks for pages and they and those that sequences before
 *     it asked for (refused for lack of pages or tokens or not) are more than the ring holds, or if it
 *     has new tokens and they and those before are more than max_tokens. A refused sequence keeps its
 *     pages and length, and has no new tokens in this step.
 * Pages that come back are free for the next call, not for this one.
 *
 *   N, page_size, max_pages, max_tokens    >= 1
 *   block_table  int32, page p of sequence n at n * table_stride + p; updated in place: the new pages
 *                of a served sequence are entries held[n] .. held[n] + need_n - 1. Other entries
 *                stay. table_stride >= max_pages.
 *   held         int32 [N]: entries of block_table that are the sequence's (also those that no token
 *                is in yet, or no more, as after drafts that fell). Taken as within [0, max_pages].
 *   lens         int32 [N]: tokens in the cache that stand (below 0: as 0): `start` of kda_kv_append.
 *   new_lens     int32 [N]: tokens of this step.
 *   free_pages   int32 [free_capacity], a ring: its free pages are entries (head + i) mod
 *                free_capacity, i < count. Pages are taken from its head; pages that come back are
 *                written behind its end, in place, by sequence and entry (those that find no
 *                room are lost: free_capacity >= all pages there are).
 *   ring         int32 [2]: head (taken mod free_capacity, below 0: as 0), count (taken as within
 *                [0, free_capacity]).
 *   held_out, ring_out
 *                held and ring after the call. Not held and ring themselves: every workgroup reads
 *                those.
 *   seq_lens     int32 [N]: tokens in the cache with this step's: `seq_lens` of kda_paged_decode. 0 if
 *                the sequence has ended.
 *   cu_seqlens   int32 [N + 1]: offsets of the sequences' new tokens, `cu_seqlens` of the calls above.
 *   slots        int64 [max_tokens], or NULL: where new token t goes, page * page_size + position %
 *                page_size; -1 at and past cu_seqlens[N], and where the table has a page below 0.
 *   positions    int32 [max_tokens], or NULL: its position; -1 at and past cu_seqlens[N].
 */
typedef struct {
    int N, page_size, max_pages, max_tokens, free_capacity;
    int32_t* block_table;
    int64_t table_stride;
    const int32_t *held, *lens, *new_lens;
    int32_t* free_pages;
    const int32_t* ring;
    int32_t *held_out, *ring_out, *seq_lens, *cu_seqlens;
    int64_t* slots;
    int32_t* positions;
} kda_page_plan_args;

/* Arguments of kda_adjust_logits: R rows of logits of each of N sequences, row j for the token after
 * j drafts (R = 1: plain decode; R = m + 1 beside kda_verify_drafts). For each row, in 32 bits (to 2^-22
 * of the largest of the terms) and in this order, x being the logit of token i:
 *   - if i is in the sequence's history or among its first j drafts: x = x / repetition[n] where x > 0,
 *     x * repetition[n] elsewhere.
 *   - x = x + (bias - less), where less = frequency[n] * c + presence[n] if i is c > 0 times in the
 *     history past the prompt and among the first j drafts, else 0, and the bias is the last entry's that
 *     lists i, else 0.
 *   - where the mask's bit i is 0, x = -infinity (whatever x was, NaN too).
 *   - x = x / temperature[n]. Temperatures that are not above 0 stand for the limit: x stays, and with
 *     KDA_LOGITS_PROBS the row is 1 at its largest x (the first of equal ones; NaN is never it) and
 *     0 elsewhere. +infinity is taken as the largest finite number.
 *   - with KDA_LOGITS_PROBS softmax over the row: 0 everywhere if every x is -infinity; infinite ones
 *     share the row evenly; a NaN makes the row NaN.
 *
 *   N, R, V    >= 1, V at most 2^30.
 *   dtype      of logits, out_dtype of out: KDA_F32 or KDA_BF16.
 *   logits     row (n, j) begins at n * seq_stride + j * row_stride (elements), as the row of out does
 *              by its strides. out may be logits itself where types and strides are the same; otherwise
 *              they do not overlap. Rows of out do not overlap each other.
 *   history    int32: id t of sequence n at n * history_stride + t (0 to share one), t < history_lens[n]
 *              (device int32 [N], taken as within [0, max_history]); the first prompt_lens[n] (device
 *              int32 [N] or NULL: 0) are its prompt. NULL: none. Ids outside [0, V) are no token's.
 *   drafts     int32 [N, R - 1], or NULL: none count.
 *   repetition, frequency, presence
 *              fp32 [N] each, or NULL for 1, 0, 0. repetition within 2^-126 .. 2^126.
 *   bias_ids, bias
 *              int32 and fp32 [N, max_bias], of which the first bias_counts[n] (device int32 [N] or
 *              NULL: all; taken as within [0, max_bias]) count. NULL: none.
 *   mask       32-bit words: bit i % 32 of word i / 32 is token i's, the words of row (n, j) begin at
 *              n * mask_seq_stride + j * mask_row_stride (words; 0 to share them). NULL: all allowed.
 *   temperature  fp32 [N], or NULL for 1.
 *   workspace  device scratch of at least kda_adjust_logits_workspace_bytes() bytes (0 without
 *              KDA_LOGITS_PROBS), 256-byte aligned; contents on entry are ignored. Calls that overlap
 *              in time need one each.
 *   flags      0 or KDA_LOGITS_PROBS.
 */
#define KDA_LOGITS_PROBS 1u
typedef struct {
    int N, R, V;
    kda_dtype dtype, out_dtype;
    const void* logits;
    int64_t seq_stride, row_stride;
    void* out;
    int64_t out_seq_stride, out_row_stride;
    const int32_t* history;
    int64_t history_stride;
    int max_history;
    const int32_t *history_lens, *prompt_lens;
    const int32_t* drafts;
    const float *repetition, *frequency, *presence;
    const int32_t* bias_ids;
    const float* bias;
    const int32_t* bias_counts;
    int max_bias;
    const uint32_t* mask;
    int64_t mask_seq_stride, mask_row_stride;
    const float* temperature;
    void* workspace;
    size_t workspace_bytes;
    unsigned flags;
} kda_logits_args;

/* Linear attention with a decay for each head: prompts (the workspace query looks at shapes and
 * dtypes, not at pointers, but for whether cu_seqlens is NULL; SIZE_MAX when they are invalid), one
 * token, and m tokens with the commit of an accepted prefix. */
size_t kda_lin_chunk_fwd_workspace_bytes(const kda_lin_chunk_args* args);
kda_status kda_lin_chunk_fwd(const kda_lin_chunk_args* args, void* hip_stream);
kda_status kda_lin_decode_step(const kda_lin_decode_args* args, void* hip_stream);
kda_status kda_lin_decode_multi(const kda_lin_decode_args* args, void* hip_stream);

/* Block tables, lengths, positions and slots of a step (see kda_page_plan_args). */
kda_status kda_page_plan(const kda_page_plan_args* args, void* hip_stream);

/* Penalties, biases, grammar masks and temperatures on logits, and their softmax (see
 * kda_logits_args). The workspace query looks at N, R, V, dtypes and flags only; SIZE_MAX when they
 * are invalid. */
size_t kda_adjust_logits_workspace_bytes(const kda_logits_args* args);
kda_status kda_adjust_logits(const kda_logits_args* args, void* hip_stream);

const char* kda_status_string(kda_status s);
const char* kda_last_error(void);   /* detail of the last failure on this thread */
int kda_abi_version(void);           /* KDA_ABI_VERSION of the built library */

#ifdef __cplusplus
}
#endif

#endif /* KDA_H */
