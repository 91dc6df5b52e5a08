// Attention of a few new tokens per sequence over a paged cache: the kernels, by cache type.
//
// For each key/value head, the rows (new token j, query head of the group) of a sequence share
// every key and value, so S^T = K Q^T and O^T = V^T P^T are matrix products with up to 16 rows
// as the columns of one 16 x 16 tile. One pass over the cache keeps the running maximum and sum
// of each row's softmax:
//     M' = max(M, max s),  l' = l 2^{M - M'} + sum 2^{s - M'},  O' = O 2^{M - M'} + sum 2^{s - M'} v
// (s in units of log2). Up to 32 rows the cache is read once (every 32 rows, a row block, read it again)
// and nothing else is large: HBM bounds it.
//
// Layout (no LDS and no cross-lane move between load and product). A wave takes 32 tokens at a
// time. v_mfma 16x16x32: lane l = (r = l & 15, g = l >> 4).
//   K is the A operand: lane (r, g) loads its channels of tokens r and 16 + r.
//   S^T comes out with tokens 4g + i (and 16 + 4g + i) of row r in lane (r, g), which is exactly a
//   B operand of the next product with those eight tokens as the K slots of group g.
//   V is its A operand: lane (r, g) loads channels VEC r .. VEC r + VEC - 1 (VEC = D / 16) of its
//   eight tokens, and the operand of channel tile j is element j of each: a byte permutation
//   within the lane. Tile j then holds channels {VEC r + j}, so lane (r, g) ends with the D / 4
//   consecutive channels from g D / 4 on of row r.
//
// Rounding: products, sums and the softmax weights P are held in 32 bits. Over a bf16 cache P goes into
// the V product as three bf16 parts, which hold all 24 bits. (With two, 2^-17 of each weight, fp32
// results were off by 2e-6 where they are off by 4e-7, and 0.25 % of the bf16 results a step, for
// 0.15 us of 8.85 on one short context, 2 % at 32 rows per head: 64 contexts of up to 4000 tokens 129 us,
// 131 with three; nothing that shows elsewhere, since the products hide under the loads.) An e4m3 value
// is exact in bf16 (K) and in fp16 (V), so over an e4m3 cache P is two fp16 parts (2^-23). One part
// (2^-12) put 8 % of the bf16 results a step off and saved nothing at up to 16 rows (512 contexts with 4
// drafts 347 us either way), 5 % at 32 rows (64 contexts of up to 4000 tokens with 8 drafts 85 us, 89
// with two). fp32 caches take the fp32 matrix instruction throughout.
//
// Who sees what. Rows of a block differ in what they see only near the newest token and the
// window's far edge ("private" tokens, at most m - 1 at each end). A row that does not see a token
// has weight 0 for it in the matrix product, which is exact as long as the value is finite. Where
// a private value is not, the tile's private values enter the product as zero and are added
// row by row with predicated multiply-adds instead, so that a NaN or an infinity that a row does
// not see never meets it. Values that no row sees are replaced by zero.
#pragma once

#include <math.h>

#include <algorithm>
#include <type_traits>

#include "kda_device.h"
#include "kda_internal.h"
#include "kda_paged.h"

namespace kda {
namespace paged {

// row / p.group, for 0 <= row < 2^24
__device__ __forceinline__ int div_group(const PagedDecodePlan& p, int row) {
  return (int)(((uint64_t)(unsigned)row * p.group_mul) >> p.group_shift);
}
// Work is counted in units: a workgroup's four waves carry p.heads (1, 2 or 4) neighbouring
// key/value heads, 4 / p.heads waves each, and take 32 tokens per wave at a time, so a unit is
// 2^p.unit_log = 128 / p.heads tokens of p.heads heads. The heads of a token lie side by side in a
// cache with the token outermost, and reading 1 KiB of each token at a time runs nearer to what HBM
// delivers than 256 B (4 contexts of 65k tokens, 8 heads, 512 workgroups: 213 us with one head per
// workgroup, 188 with four).
//
// Workgroups share the units of all (sequence, row block, head group)s evenly and in order, each group
// counted p.start units longer than it is: what its first loads and its results cost comes before
// its first unit. A workgroup that begins or ends inside a group's units leaves a part in the
// workspace, which paged_join_kernel joins.

// The new tokens of sequence n see positions [0, len); with a window, the first of them begins
// at len - m + 1 - window.
__device__ __forceinline__ int seq_len(const PagedDecodePlan& p, int n) {
  return min(max(p.seq_lens[n], 0), p.max_len);
}
__device__ __forceinline__ int first_unit(const PagedDecodePlan& p, int len) {
  if (!p.window) return 0;
  const int64_t lo = (int64_t)len - p.m + 1 - p.window;
  return lo > 0 ? (int)lo >> p.unit_log : 0;
}
// Units that a sequence's workgroups walk per group; one at least, which writes zeros.
__device__ __forceinline__ int seq_units(const PagedDecodePlan& p, int len) {
  return max(1, ((len + (1 << p.unit_log) - 1) >> p.unit_log) - first_unit(p, len));
}

// A result that a wave holds back in LDS: rows [row0, row0 + rows) of head h of sequence n, finished
// (part < 0) or for row `part` of part_o on. The rows follow, kHeldPad bytes apart (over the banks).
struct alignas(16) Held {
  int64_t part;
  int n, h, row0, rows;
};
constexpr int kHeldPad = 16;

template <int CT, int D>
struct Types {
  static constexpr int ES = CT == kF32 ? 4 : CT == kBF16 ? 2 : 1;
  static constexpr int VEC = D / 16;               // channels of V per lane and token
  static constexpr int KW = D * ES / 16;           // 32-bit words of a key row per lane
  static constexpr int KC = KW < 4 ? KW : 4;       // words per load
  static constexpr int NKL = KW / KC;              // loads per key row
  static constexpr int VB = VEC * ES;              // bytes of a value row per lane
  static constexpr int VW = VB < 4 ? 1 : VB / 4;   // words that hold them
  static constexpr int QW = CT == kF32 ? D / 4 : D / 8;  // words of a query row per lane
};

// Streamed: each cached value is read once per row block (4 contexts of 65k tokens: 222 -> 213 us; a plain read
// of 4 GiB runs at 7.1 TB/s with such loads, at 6.2 without).
template <int W>
__device__ __forceinline__ void load_words(const char* p, uint32_t* w) {
  if constexpr (W == 1) {
    w[0] = __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(p));
  } else if constexpr (W == 2) {
    const u32x2 x = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(p));
    w[0] = x[0]; w[1] = x[1];
  } else {
#pragma unroll
    for (int c = 0; c < W; c += 4) {
      const u32x4 x = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p + 4 * c));
      w[c] = x[0]; w[c + 1] = x[1]; w[c + 2] = x[2]; w[c + 3] = x[3];
    }
  }
}

__device__ __forceinline__ uint32_t halves_lo(uint32_t a, uint32_t b) {
  return __builtin_amdgcn_perm(b, a, 0x05040100u);
}
__device__ __forceinline__ uint32_t halves_hi(uint32_t a, uint32_t b) {
  return __builtin_amdgcn_perm(b, a, 0x07060302u);
}
typedef float floatx2 __attribute__((ext_vector_type(2)));
// op over the lanes r, 16 + r, 32 + r, 48 + r, in all of them. Row exchanges, not shuffles: those go
// through LDS, whose counter the page ids' scalar loads share, so the maximum of each tile would wait
// for the page ids of the tile two ahead (one short context 8.84 -> 8.76 us).
template <typename Op>
__device__ __forceinline__ float over_groups(float x, Op op) {
  const unsigned a = __float_as_uint(x);
  const auto y = __builtin_amdgcn_permlane16_swap(a, a, false, false);
  const unsigned b = __float_as_uint(op(__uint_as_float(y[0]), __uint_as_float(y[1])));
  const auto z = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  return op(__uint_as_float(z[0]), __uint_as_float(z[1]));
}
// Elements 2h and 2h + 1 of four e4m3 values.
template <bool H>
__device__ __forceinline__ floatx2 e4m3_pair(uint32_t w) {
  return __builtin_amdgcn_cvt_pk_f32_fp8((int)w, H);
}
// Two e4m3 values as bf16 or fp16 (both exact), elements 2h and 2h + 1.
template <bool H>
__device__ __forceinline__ uint32_t e4m3_bf16(uint32_t w) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.f, H));
}
template <bool H>
__device__ __forceinline__ uint32_t e4m3_f16(uint32_t w) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.f, H));
}
// Eight e4m3 values as a bf16 operand.
__device__ __forceinline__ bf16x8 e4m3_operand(uint32_t w0, uint32_t w1) {
  return __builtin_bit_cast(bf16x8, u32x4{e4m3_bf16<false>(w0), e4m3_bf16<true>(w0),
                                          e4m3_bf16<false>(w1), e4m3_bf16<true>(w1)});
}

// A word of cached values holds an infinity or a NaN if ((w & kMagnitude) + kStep) & kOver: adding
// a step to a magnitude whose exponent (e4m3, which has no infinities: all bits) is all ones
// carries into the sign's place and no further.
template <int CT>
struct NotFinite {
  static constexpr uint32_t kMagnitude = CT == kF32 ? 0x7fffffffu : CT == kBF16 ? 0x7fff7fffu : 0x7f7f7f7fu;
  static constexpr uint32_t kStep = CT == kF32 ? 0x00800000u : CT == kBF16 ? 0x00800080u : 0x01010101u;
  static constexpr uint32_t kOver = ~kMagnitude;
};

// The VEC channels of a lane's words of a value row, as floats.
template <int CT, int VEC>
__device__ __forceinline__ float word_value(const uint32_t* w, int x) {
  if constexpr (CT == kF32) return __uint_as_float(w[x]);
  if constexpr (CT == kBF16) return __uint_as_float(x & 1 ? w[x / 2] & 0xffff0000u : w[x / 2] << 16);
  if constexpr (CT == kF8) {
    const floatx2 v = x & 2 ? e4m3_pair<true>(w[x / 4]) : e4m3_pair<false>(w[x / 4]);
    return x & 1 ? v.y : v.x;
  }
}
template <int VB>
__device__ __forceinline__ void load_bytes(const char* p, uint32_t* w) {
  if constexpr (VB == 2)
    w[0] = *reinterpret_cast<const uint16_t*>(p);
  else
    load_words<VB / 4>(p, w);
}

// N consecutive channels, as fp32 or rounded to bf16.
template <int N, typename T>
__device__ __forceinline__ void store_channels(T* p, const float* x) {
  if constexpr (sizeof(T) == 4) {
    if constexpr (N == 2) {
      *reinterpret_cast<floatx2*>(p) = floatx2{x[0], x[1]};
    } else {
#pragma unroll
      for (int i = 0; i < N; i += 4) *reinterpret_cast<floatx4*>(p + i) = floatx4{x[i], x[i + 1], x[i + 2], x[i + 3]};
    }
  } else {
    uint32_t w[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) w[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
    if constexpr (N == 2) *reinterpret_cast<uint32_t*>(p) = w[0];
    if constexpr (N == 4) *reinterpret_cast<u32x2*>(p) = u32x2{w[0], w[1]};
    if constexpr (N == 8) *reinterpret_cast<u32x4*>(p) = u32x4{w[0], w[1], w[2], w[3]};
  }
}

// A row of o: of query row `row` of key/value head h of sequence n.
__device__ __forceinline__ int64_t out_row(const PagedDecodePlan& p, int n, int h, int row) {
  const int j = div_group(p, row);
  return ((int64_t)n * p.m + j) * p.Hq + h * p.group + row - j * p.group;
}
// Four channels (d ..) of a finished row: o and l are sums weighted by 2^{s - now}.
template <int D>
__device__ __forceinline__ void write_row(const PagedDecodePlan& p, int64_t dst, int d, float scale,
                                          float now, float l, floatx4 o) {
  const float inv = scale / l;
  if (l == 0.f) o = floatx4{0.f, 0.f, 0.f, 0.f};  // nothing was seen
  else o = floatx4{o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv};
  if (p.out_bf16)
    *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(p.o) + dst * D + d) =
        u32x2{pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3])};
  else
    *reinterpret_cast<floatx4*>(static_cast<float*>(p.o) + dst * D + d) = o;
  if (p.lse && d == 0)
    p.lse[dst] = l == 0.f ? -INFINITY : (now + log2f(l)) * 0.6931471805599453f;
}

// P16: page_size is a multiple of 16, so 16 aligned tokens have one page.
template <int CT, int D, int NT, bool P16>
__global__ __launch_bounds__(256, 2) void paged_decode_kernel(
    const PagedDecodePlan p, const int32_t* __restrict__ block_table) {
  using TY = Types<CT, D>;
  constexpr int VEC = TY::VEC;
  // Weights that become fp16 are held 2^14 times as large (at most 16384): the smallest fp16 step
  // is then 2^-38 of the largest weight, and a long tail of small weights is not lost.
  constexpr float kLift = CT == kF8 ? 14.f : 0.f, kUnlift = CT == kF8 ? 0x1p-14f : 1.f;
  constexpr int COLS = 16 * NT;
  constexpr int OS = D + 4;  // floats per row of s_o (staggered over the LDS banks)
  // Several waves per head: where they meet. One wave per head: each wave's scratch and the results
  // it holds back.
  extern __shared__ __align__(16) char lds[];
  float(*s_o)[COLS * OS] = reinterpret_cast<float(*)[COLS * OS]>(lds);
  float(*s_m)[COLS] = reinterpret_cast<float(*)[COLS]>(lds + sizeof(float) * 4 * COLS * OS);
  float(*s_l)[COLS] = s_m + 4;
  __shared__ int64_t s_scan[4];
  __shared__ int s_at[4];

  const int t = threadIdx.x, lane = t & 63, r = lane & 15, g = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(t >> 6);
  const int per_seq = p.row_blocks * p.groups;
  const int wph = 4 / p.heads;                      // waves per head
  const int head_at = wv / wph, part_at = wv % wph;  // this wave's head of the group, share of a unit
  const int unit = 1 << p.unit_log;

  // ---- this workgroup's share: `left` units, from unit `from` of (row block, head group) `pair` of
  //      sequence n on (the first p.start of a group's are not read)
  int n, pair, from = 0, len;
  int64_t left;
  if (p.split == 0) {
    n = blockIdx.x / per_seq;
    pair = blockIdx.x - n * per_seq;
    len = seq_len(p, n);
    left = seq_units(p, len);
  } else {
    // each thread the units of c sequences, of which it keeps the first's
    const int c = (p.N + 255) / 256, i0 = t * c;
    const int len0 = i0 < p.N ? seq_len(p, i0) : 0, un0 = p.start + seq_units(p, len0);
    int64_t mine = i0 < p.N ? un0 : 0;
    for (int i = i0 + 1; i < min(i0 + c, p.N); ++i) mine += p.start + seq_units(p, seq_len(p, i));
    mine *= per_seq;
    int64_t incl = mine;
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) {
      const int64_t y = __shfl_up(incl, s, 64);
      if (lane >= s) incl += y;
    }
    if (lane == 63) s_scan[wv] = incl;
    __syncthreads();
    int64_t total = 0, before = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i < wv) before += s_scan[i];
      total += s_scan[i];
    }
    const unsigned w = blockIdx.x;
    const uint64_t each = (uint64_t)total / (unsigned)p.split;
    const unsigned more = (unsigned)(total - (int64_t)(each * (unsigned)p.split));
    left = (int64_t)each + (w < more ? 1 : 0);
    if (left == 0) return;
    const int64_t u0 = (int64_t)(each * w) + min(w, more);
    int64_t excl = before + incl - mine;
    if (excl <= u0 && u0 < excl + mine) {
      int i = i0, un = un0, at_len = len0;
      while (u0 - excl >= (int64_t)un * per_seq && i + 1 < p.N) {
        excl += (int64_t)un * per_seq;
        at_len = seq_len(p, ++i);
        un = p.start + seq_units(p, at_len);
      }
      const int64_t at = u0 - excl;
      const int in = at >> 32 ? (int)(at / un) : (int)((unsigned)at / (unsigned)un);
      s_at[0] = i;
      s_at[1] = in;
      s_at[2] = (int)(at - (int64_t)in * un);
      s_at[3] = at_len;
    }
    __syncthreads();
    n = s_at[0];
    pair = s_at[1];
    from = s_at[2];
    len = s_at[3];
  }

  const float log2_scale = p.scale * kLog2e;

  // One wave per head: finished rows and parts wait in LDS until there is no room for more or the
  // wave's work is done. A few lines written now and then among the reads of everyone else cost HBM
  // a change of direction each: 512 contexts of up to 4096 e4m3 tokens with 16 rows per head, whose
  // results are 33 MB next to 2.1 GB read, 399 us with every result written at once, 357 with results
  // held back.
  char* const scratch = lds + wv * (32 * COLS * (int)sizeof(float) + p.hold);
  char* const hold = scratch + 32 * COLS * (int)sizeof(float);
  int held = 0;  // bytes
  auto put_out = [&]() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    for (int at = 0; at < held;) {
      const Held x = *reinterpret_cast<const Held*>(hold + at);
      const char* from = hold + at + sizeof(Held);
      const int es = x.part < 0 && p.out_bf16 ? 2 : 4, row = D * es, pieces = row / 16;  // a power of two
      for (int i = lane; i < x.rows * pieces; i += 64) {
        const int c = i >> __builtin_ctz(pieces), b = (i & (pieces - 1)) * 16;
        char* to = x.part < 0 ? static_cast<char*>(p.o) + out_row(p, x.n, x.h, x.row0 + c) * row
                              : reinterpret_cast<char*>(p.part_o) + (x.part + c) * row;
        *reinterpret_cast<u32x4*>(to + b) = *reinterpret_cast<const u32x4*>(from + c * (row + kHeldPad) + b);
      }
      at += sizeof(Held) + x.rows * (row + kHeldPad);
    }
    held = 0;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  };

  // ---- one (row block, head group) of one sequence after the other
  while (left > 0) {
    n = __builtin_amdgcn_readfirstlane(n);
    pair = __builtin_amdgcn_readfirstlane(pair);
    from = __builtin_amdgcn_readfirstlane(from);
    const int rb = p.row_blocks == 1 ? 0 : pair / p.groups;
    const int h0 = (pair - rb * p.groups) * p.heads, h = h0 + head_at;
    const int row0 = rb * COLS;
    const int rows = min(COLS, p.rows - row0);
    const int32_t* pages = block_table + n * p.c.table_stride;

    // ---- what does not wait for the length: the query rows (columns r of NT tiles, as B operands),
    //      and the scales
    uint32_t q[NT][TY::QW];
    int j_of[NT];  // new token of this lane's row; -1: no such row
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int row = row0 + nt * 16 + r;
      const bool there = row < p.rows;
      const int j = there ? div_group(p, row) : 0, head = h * p.group + (there ? row - j * p.group : 0);
      j_of[nt] = there ? j : -1;
      const char* qp = p.q + ((int64_t)n * p.m + j) * p.q_token + head * p.q_head;
      if constexpr (CT == kF32) {
#pragma unroll
        for (int s = 0; s < TY::QW; s += 4) load_words<4>(qp + 4 * (4 * s + 4 * g), &q[nt][s]);
      } else {
#pragma unroll
        for (int s = 0; s < D / 32; ++s) {
          const int d = CT == kF8 && D > 32 ? 64 * (s / 2) + 16 * g + 8 * (s & 1) : 32 * s + 8 * g;
          load_words<4>(qp + 2 * d, &q[nt][4 * s]);
        }
      }
    }
    const float to_log2 = log2_scale * (p.c.k_scale ? p.c.k_scale[h] : 1.f);
    const float v_scale = p.c.v_scale ? p.c.v_scale[h] : 1.f;
    const int next_len = seq_len(p, min(n + 1, p.N - 1));

    len = __builtin_amdgcn_readfirstlane(len);
    const int un = seq_units(p, len);
    const int take = __builtin_amdgcn_readfirstlane((int)min((int64_t)(p.start + un - from), left));
    const int u_first = max(from - p.start, 0), cnt = from + take - p.start - u_first;
    if (cnt <= 0) break;  // the share ends before the group's first unit

    // what the rows see: row of new token j sees [lo(j), hi(j))
    auto hi_of = [&](int j) { return len - p.m + 1 + j; };
    auto lo_of = [&](int j) {
      return p.window ? (int)max((int64_t)0, (int64_t)hi_of(j) - p.window) : 0;
    };
    const int j_first = div_group(p, row0), j_last = div_group(p, row0 + rows - 1);
    const int all_lo = lo_of(j_last), all_hi = hi_of(j_first);  // seen by every row
    const int any_lo = lo_of(j_first), any_hi = hi_of(j_last);  // seen by one at least
    int lo[NT], hi[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      lo[nt] = j_of[nt] >= 0 ? lo_of(j_of[nt]) : 0;
      hi[nt] = j_of[nt] >= 0 ? hi_of(j_of[nt]) : 0;
      // fp32 rows are scaled here (a score then overflows only if it is itself out of range), bf16
      // ones keep their values and the scores are scaled
#pragma unroll
      for (int s = 0; s < TY::QW; ++s) {
        if (CT == kF32) q[nt][s] = __float_as_uint(__uint_as_float(q[nt][s]) * to_log2);
        q[nt][s] = j_of[nt] >= 0 ? q[nt][s] : 0u;
      }
    }

    floatx4 acc[NT][VEC];
    float top[NT], sum[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      top[nt] = -INFINITY;
      sum[nt] = 0.f;
#pragma unroll
      for (int j = 0; j < VEC; ++j) acc[nt][j] = floatx4{0.f, 0.f, 0.f, 0.f};
    }

    // ---- this wave's tiles: tokens [base + unit i, + 32), those that some row sees
    const int base = (first_unit(p, len) + u_first) * unit + 32 * part_at;
    const int i0 = any_lo > base + 31 ? (any_lo - base - 32) / unit + 1 : 0;
    const int i1 = any_hi > base ? min(cnt, (any_hi - base - 1) / unit + 1) : 0;

    const char* kh = p.c.k + h * p.c.k_head;
    const char* vh = p.c.v + h * p.c.v_head;
    const int last = any_hi - 1;  // the newest token that some row sees (>= 0 if i0 < i1)

    // Where a tile's rows lie. Tokens past `last` give their place to it or to a slot of its page,
    // and ids of no page to page 0; what they read is masked below.
    auto page_at = [&](int tok) { return pages[div_page(p.c, (unsigned)tok)]; };
    auto is_page = [&](int id) { return (unsigned)id < (unsigned)p.c.num_pages; };
    // P16: 16 tokens have one page, so the rows' base is uniform and a lane adds 32 bits to it.
    // Half s of a tile: the page id and the slot of its first token; (page index, slot) of the
    // tile two ahead, whose ids are being fetched, is carried along without dividing.
    struct Halves {
      int id[2], slot[2];
    };
    const unsigned k_lane = (unsigned)(r * (int)p.c.k_token) + g * 4 * TY::KC;
    const unsigned v_lane = (unsigned)(4 * g * (int)p.c.v_token) + r * TY::VB;
    const int end = last & ~15;  // the newest half
    const int end_page = div_page(p.c, (unsigned)max(end, 0)), end_slot = end - end_page * p.c.page_size;
    const int step_pages = div_page(p.c, (unsigned)unit), step_slots = unit - step_pages * p.c.page_size;
    int ahead[2], ahead_page[2], ahead_slot[2];  // token, page index, slot of the halves looked up next
    auto look_up = [&]() {
      Halves x;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const bool past = ahead[s] > end;
        x.slot[s] = past ? end_slot : ahead_slot[s];
        x.id[s] = __builtin_amdgcn_readfirstlane(pages[past ? end_page : ahead_page[s]]);
        ahead[s] += unit;
        ahead_page[s] += step_pages;
        ahead_slot[s] += step_slots;
        if (ahead_slot[s] >= p.c.page_size) {
          ahead_slot[s] -= p.c.page_size;
          ++ahead_page[s];
        }
      }
      return x;
    };
    auto half_at = [&](const Halves& x, int s, unsigned page16, int64_t token) {
      const unsigned id = is_page(x.id[s]) ? x.id[s] : 0;
      return (int64_t)(((uint64_t)id * page16) << 4) + (int64_t)x.slot[s] * (int)token;
    };
    // else: every row by itself
    struct Rows {
      int id[10];  // page ids of the lane's 2 key rows and 8 value rows
    };
    auto k_token = [&](int tb, int s) { return min(tb + 16 * s + r, last); };
    auto v_token = [&](int tb, int i) { return min(tb + 16 * (i >> 2) + 4 * g + (i & 3), last); };
    auto look_up_rows = [&](int tb) {
      Rows x;
#pragma unroll
      for (int s = 0; s < 2; ++s) x.id[s] = page_at(k_token(tb, s));
#pragma unroll
      for (int i = 0; i < 8; ++i) x.id[2 + i] = page_at(v_token(tb, i));
      return x;
    };
    auto row_at = [&](int id, int tok, int64_t page, int64_t token) {
      const int slot = tok - div_page(p.c, (unsigned)tok) * p.c.page_size;
      return (is_page(id) ? id : 0) * page + slot * token;
    };
    typedef std::conditional_t<P16, Halves, Rows> Ids;

    uint32_t kw[2][TY::KW], vw[8][TY::VW];
    auto load_k = [&](int tb, const Ids& x) {
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const char* row;
        unsigned off;
        if constexpr (P16) {
          row = kh + half_at(x, s, p.c.k_page16, p.c.k_token);
          off = k_lane;
          asm volatile("" : "+v"(off));  // keeps base and offset apart: scalar base + 32 bits
        } else {
          row = kh + row_at(x.id[s], k_token(tb, s), p.c.k_page, p.c.k_token);
          off = g * 4 * TY::KC;
        }
#pragma unroll
        for (int c = 0; c < TY::NKL; ++c)
          load_words<TY::KC>(row + off + c * 16 * TY::KC, &kw[s][c * TY::KC]);
      }
    };
    auto load_v = [&](int tb, const Ids& x) {
      if constexpr (P16) {
        unsigned off = v_lane;
        asm volatile("" : "+v"(off));
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const char* row = vh + half_at(x, s, p.c.v_page16, p.c.v_token);
#pragma unroll
          for (int i = 0; i < 4; ++i) load_bytes<TY::VB>(row + i * p.c.v_token + off, vw[4 * s + i]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          load_bytes<TY::VB>(vh + row_at(x.id[2 + i], v_token(tb, i), p.c.v_page, p.c.v_token) + r * TY::VB,
                             vw[i]);
      }
    };

    Ids now, next, after;  // of this tile, the next, the one after (P16)
    if (i0 < i1) {
      const int tb = base + unit * i0;
      if constexpr (P16) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          ahead[s] = tb + 16 * s;
          ahead_page[s] = div_page(p.c, (unsigned)ahead[s]);
          ahead_slot[s] = ahead[s] - ahead_page[s] * p.c.page_size;
        }
        next = look_up();
        load_k(tb, next);
        after = look_up();
      } else {
        next = look_up_rows(tb);
        load_k(tb, next);
      }
    }
    for (int i = i0; i < i1; ++i) {
      const int tb = base + unit * i;
      now = next;
      if constexpr (P16) next = after;
      load_v(tb, now);
      if constexpr (!P16) next = look_up_rows(tb + unit);

      // S^T = K Q^T
      floatx4 s[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = floatx4{0.f, 0.f, 0.f, 0.f};
      if constexpr (CT == kF32) {
#pragma unroll
        for (int c = 0; c < TY::QW; ++c)
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              s[nt][u] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                  __uint_as_float(kw[u][c]), __uint_as_float(q[nt][c]), s[nt][u], 0, 0, 0);
      } else {
#pragma unroll
        for (int c = 0; c < D / 32; ++c)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            bf16x8 a;
            if constexpr (CT == kBF16)
              a = __builtin_bit_cast(bf16x8, u32x4{kw[u][4 * c], kw[u][4 * c + 1], kw[u][4 * c + 2],
                                                   kw[u][4 * c + 3]});
            else
              a = e4m3_operand(kw[u][2 * c], kw[u][2 * c + 1]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const bf16x8 b = __builtin_bit_cast(
                  bf16x8, u32x4{q[nt][4 * c], q[nt][4 * c + 1], q[nt][4 * c + 2], q[nt][4 * c + 3]});
              s[nt][u] = mfma_bf16(a, b, s[nt][u]);
            }
          }
      }

      // the next tile's keys, and the page ids of the one after. Past the last tile too (the
      // newest row once more): behind a branch, the wait for V would wait for these as well.
      load_k(tb + unit, next);
      if constexpr (P16) after = look_up();

      // tokens that not every row sees, or that are on no page
      bool on_pages = true;
#pragma unroll
      for (int x = P16 ? 0 : 2; x < (P16 ? 2 : 10); ++x) on_pages = on_pages && is_page(now.id[x]);
      const bool plain = tb >= all_lo && tb + 32 <= all_hi && (P16 ? on_pages : __all(on_pages));
#pragma unroll
      for (int i8 = 0; i8 < 8; ++i8)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) s[nt][i8 >> 2][i8 & 3] *= CT == kF32 ? 1.f : to_log2;
      bool careful = false;  // a private value is not finite
      if (!plain) {
        auto token = [&](int i8) { return tb + 4 * g + (i8 & 3) + 16 * (i8 >> 2); };
        auto on_page = [&](int i8) { return is_page(now.id[P16 ? i8 >> 2 : 2 + i8]); };
#pragma unroll
        for (int i8 = 0; i8 < 8; ++i8) {
          const int tok = token(i8);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const bool sees = on_page(i8) && tok >= lo[nt] && tok < hi[nt];
            s[nt][i8 >> 2][i8 & 3] = sees ? s[nt][i8 >> 2][i8 & 3] : -INFINITY;
          }
        }
        if (max(tb, any_lo) < all_lo || min(tb + 32, any_hi) > all_hi) {  // the tile has private tokens
          uint32_t over = 0;
#pragma unroll
          for (int i8 = 0; i8 < 8; ++i8) {
            const int tok = token(i8);
            const bool some = tok >= any_lo && tok < any_hi, all = tok >= all_lo && tok < all_hi;
            const uint32_t pick = on_page(i8) && some && !all ? NotFinite<CT>::kMagnitude : 0u;
#pragma unroll
            for (int e = 0; e < TY::VW; ++e) over |= (vw[i8][e] & pick) + NotFinite<CT>::kStep;
          }
          careful = __any((over & NotFinite<CT>::kOver) != 0);
        }
        const int from = careful ? all_lo : any_lo, to = careful ? all_hi : any_hi;
#pragma unroll
        for (int i8 = 0; i8 < 8; ++i8) {
          const int tok = token(i8);
          const uint32_t keep = on_page(i8) && tok >= from && tok < to ? ~0u : 0u;
          // In place: the compiler would copy the values on the other way round, and wait there.
#pragma unroll
          for (int e = 0; e < TY::VW; ++e) asm volatile("v_and_b32 %0, %1, %0" : "+v"(vw[i8][e]) : "v"(keep));
        }
      }

      // running maximum and sum of each row
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float mx = fmaxf(fmaxf(fmaxf(s[nt][0][0], s[nt][0][1]), fmaxf(s[nt][0][2], s[nt][0][3])),
                         fmaxf(fmaxf(s[nt][1][0], s[nt][1][1]), fmaxf(s[nt][1][2], s[nt][1][3])));
        mx = over_groups(mx, [](float a, float b) { return fmaxf(a, b); });
        const float most = fmaxf(top[nt], mx);
        const float peak = most == -INFINITY ? 0.f : most, ref = peak - kLift;
        const float fade = __builtin_amdgcn_exp2f(top[nt] - peak);
        top[nt] = most;
        float part = 0.f;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            s[nt][u][e] = __builtin_amdgcn_exp2f(s[nt][u][e] - ref);
            part += s[nt][u][e];
          }
        sum[nt] = sum[nt] * fade + part;
        if (__any(fade != 1.f)) {
#pragma unroll
          for (int j = 0; j < VEC; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[nt][j][e] *= fade;
        }
      }

      // O^T += V^T P^T
      if constexpr (CT == kF32) {
#pragma unroll
        for (int i8 = 0; i8 < 8; ++i8)
#pragma unroll
          for (int j = 0; j < VEC; ++j)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              acc[nt][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                  __uint_as_float(vw[i8][j]), s[nt][i8 >> 2][i8 & 3], acc[nt][j], 0, 0, 0);
      } else {
        typedef std::conditional_t<CT == kF8, half8, bf16x8> operand;
        typedef std::conditional_t<CT == kF8, _Float16, __bf16> element;
        constexpr int PARTS = CT == kF8 ? 2 : 3;
        operand parts[NT][PARTS];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i8 = 0; i8 < 8; ++i8) {
            float rest = s[nt][i8 >> 2][i8 & 3];
#pragma unroll
            for (int x = 0; x < PARTS; ++x) {
              const element y = static_cast<element>(rest);
              parts[nt][x][i8] = y;
              rest -= static_cast<float>(y);
            }
          }
        auto product = [&](int j, const u32x4& frag) {
          const operand a = __builtin_bit_cast(operand, frag);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int x = 0; x < PARTS; ++x) {
              if constexpr (CT == kBF16)
                acc[nt][j] = mfma_bf16(a, parts[nt][x], acc[nt][j]);
              else
                acc[nt][j] = mfma_f16(a, parts[nt][x], acc[nt][j]);
            }
        };
#pragma unroll
        for (int j = 0; j < VEC; j += 2) {
          u32x4 f0, f1;
#pragma unroll
          for (int a = 0; a < 4; ++a) {
            uint32_t x, y;  // channels j, j + 1 of two tokens
            if constexpr (CT == kBF16) {
              x = vw[2 * a][j / 2];
              y = vw[2 * a + 1][j / 2];
            } else {
              x = j & 2 ? e4m3_f16<true>(vw[2 * a][j / 4]) : e4m3_f16<false>(vw[2 * a][j / 4]);
              y = j & 2 ? e4m3_f16<true>(vw[2 * a + 1][j / 4]) : e4m3_f16<false>(vw[2 * a + 1][j / 4]);
            }
            f0[a] = halves_lo(x, y);
            f1[a] = halves_hi(x, y);
          }
          product(j, f0);
          product(j + 1, f1);
        }
      }

      // private tokens, row by row
      if (careful) {
        const int pv0 = max(tb, any_lo), pv1 = min(tb + 32, any_hi);
        float* ps = wph == 1 ? reinterpret_cast<float*>(scratch) : s_o[wv];  // [token][column]
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i8 = 0; i8 < 8; ++i8)
            ps[(4 * g + (i8 & 3) + 16 * (i8 >> 2)) * COLS + nt * 16 + r] = s[nt][i8 >> 2][i8 & 3];
        __builtin_amdgcn_wave_barrier();
        for (int tok = pv0; tok < pv1; ++tok) {
          if (tok >= all_lo && tok < all_hi) continue;
          const int pi = div_page(p.c, (unsigned)tok);
          const int pg = pages[pi];
          if ((unsigned)pg >= (unsigned)p.c.num_pages) continue;
          const char* row = vh + pg * p.c.v_page + (tok - pi * p.c.page_size) * p.c.v_token;
          uint32_t x[4][TY::VW];
#pragma unroll
          for (int e = 0; e < 4; ++e) load_bytes<TY::VB>(row + (4 * g + e) * TY::VB, x[e]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const float w = ps[(tok - tb) * COLS + nt * 16 + r];
            const bool mine = tok >= lo[nt] && tok < hi[nt];
#pragma unroll
            for (int j = 0; j < VEC; ++j)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float y = fmaf(w, word_value<CT, VEC>(x[e], j), acc[nt][j][e]);
                acc[nt][j][e] = mine ? y : acc[nt][j][e];
              }
          }
        }
        __builtin_amdgcn_wave_barrier();
      }
    }

    // ---- each head's rows, finished or as a part
    const bool whole = cnt == un;
    const int64_t slot = (2 * (int64_t)blockIdx.x + (u_first == 0 ? 1 : 0)) * p.heads * p.part_rows;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      sum[nt] = over_groups(sum[nt], [](float a, float b) { return a + b; });
      sum[nt] *= kUnlift;
    }
    if (wph == 1) {
      // a wave has all of its head
      const int row = D * (whole && p.out_bf16 ? 2 : 4) + kHeldPad;  // bytes
      const int need = (int)sizeof(Held) + rows * row;
      if (held + need > p.hold) put_out();
      char* to = hold + held;
      held += need;
      const int64_t part = slot + head_at * p.part_rows;
      if (lane == 0) *reinterpret_cast<Held*>(to) = Held{whole ? -1 : part, n, h, row0, rows};
      to += sizeof(Held);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int c = nt * 16 + r;
        if (c >= rows) continue;
        const float l = sum[nt];
        if (g == 0) {
          if (!whole)
            *reinterpret_cast<floatx2*>(p.part_ml + (part + c) * 2) = floatx2{top[nt], l};
          else if (p.lse)
            p.lse[out_row(p, n, h, row0 + c)] = l == 0.f ? -INFINITY : (top[nt] + log2f(l)) * 0.6931471805599453f;
        }
        const float inv = kUnlift * (whole ? l == 0.f ? 0.f : v_scale / l : 1.f);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x[VEC];
#pragma unroll
          for (int j = 0; j < VEC; ++j) x[j] = whole && l == 0.f ? 0.f : acc[nt][j][e] * inv;
          const int d = g * (D / 4) + VEC * e;
          if (whole && p.out_bf16)
            store_channels<VEC, uint16_t>(reinterpret_cast<uint16_t*>(to + c * row) + d, x);
          else
            store_channels<VEC, float>(reinterpret_cast<float*>(to + c * row) + d, x);
        }
      }
    } else {
      // the waves' parts of a head meet in LDS
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int c = nt * 16 + r;
        if (g == 0) {
          s_m[wv][c] = top[nt];
          s_l[wv][c] = sum[nt];
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x[VEC];
#pragma unroll
          for (int j = 0; j < VEC; ++j) x[j] = acc[nt][j][e];
          store_channels<VEC, float>(&s_o[wv][c * OS + g * (D / 4) + VEC * e], x);
        }
      }
      __syncthreads();
      for (int x = t; x < p.heads * rows * (D / 4); x += 256) {
        const int y = x / (D / 4), d = x % (D / 4) * 4, hh = y >= rows ? 1 : 0, c = y - hh * rows;  // at most two heads
        const float scale = hh == head_at ? v_scale : p.c.v_scale ? p.c.v_scale[h0 + hh] : 1.f;
        // all four waves at once, those of the other head with weight zero
        float m[4], l = 0.f, now = -INFINITY;
        floatx4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          m[w] = w / wph == hh ? s_m[w][c] : -INFINITY;
          now = fmaxf(now, m[w]);
        }
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float f = __builtin_amdgcn_exp2f(m[w] - (now == -INFINITY ? 0.f : now));
          const floatx4 ow = *reinterpret_cast<const floatx4*>(&s_o[w][c * OS + d]);
          if (w / wph != hh) continue;
          l = fmaf(s_l[w][c], f, l);
#pragma unroll
          for (int e = 0; e < 4; ++e) o[e] = fmaf(ow[e], kUnlift * f, o[e]);
        }
        if (whole) {
          write_row<D>(p, out_row(p, n, h0 + hh, row0 + c), d, scale, now, l, o);
        } else {
          const int64_t part = slot + hh * p.part_rows + c;
          *reinterpret_cast<floatx4*>(p.part_o + part * D + d) = o;
          if (d == 0) *reinterpret_cast<floatx2*>(p.part_ml + part * 2) = floatx2{now, l};
        }
      }
      if (left > take) __syncthreads();  // s_o, s_m and s_l are free again
    }
    // which workgroups have the group's first and last units
    if (p.split && t == 0) {
      int* of = p.part_of + 2 * ((int64_t)n * per_seq + pair);
      if (u_first == 0) of[0] = blockIdx.x;
      if (u_first + cnt == un) of[1] = blockIdx.x;
    }

    left -= take;
    from = 0;
    if (++pair == per_seq) {
      pair = 0;
      ++n;
      len = next_len;
    }
  }
  if (wph == 1) put_out();
}

// Joins the parts of the heads that several workgroups shared; a head that one workgroup did
// alone is finished already. A workgroup takes `rows` rows of one (sequence, row block, head):
// D / 4 threads read a part's row, and the 1024 / D such sets are given to the parts of a row
// first, so that they are read at the same time, and to further rows.
template <int D>
__global__ __launch_bounds__(256, 6) void paged_join_kernel(const PagedDecodePlan p, int rows) {
  constexpr int Q = D / 4, SETS = 256 / Q;
  __shared__ floatx4 s_o[256];
  __shared__ floatx2 s_ml[256];
  const int t = threadIdx.x, d = t % Q * 4, set = t / Q;
  const int cols = 16 * p.tiles;
  const int h = blockIdx.x % p.Hkv, nrb = blockIdx.x / p.Hkv;
  const int rb = nrb % p.row_blocks, n = nrb / p.row_blocks;
  const int* of = p.part_of + 2 * (((int64_t)n * p.row_blocks + rb) * p.groups + h / p.heads);
  const float v_scale = p.c.v_scale ? p.c.v_scale[h] : 1.f;
  const int w0 = of[0], count = of[1] - w0 + 1;
  if (count == 1) return;

  int lanes = SETS;  // sets per row, a power of two: two parts or more each
  while (lanes > 1 && lanes * 2 >= count) lanes /= 2;
  const int lane = set % lanes, at_once = SETS / lanes;
  const int row0 = rb * cols, c1 = min(min(cols, p.rows - row0), ((int)blockIdx.y + 1) * rows);
  for (int c0 = blockIdx.y * rows; c0 < c1; c0 += at_once) {
    const int c = c0 + set / lanes;
    const bool there = c < c1;
    float top = -INFINITY, l = 0.f;
    floatx4 o = {0.f, 0.f, 0.f, 0.f};
    for (int x0 = lane; there && x0 < count; x0 += 4 * lanes) {  // four parts at a time
      floatx2 ml[4];
      floatx4 y[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int x = min(x0 + k * lanes, count - 1);
        // the first workgroup's part begins the head (slot 1), the others continue it (slot 0)
        const int64_t part =
            ((2 * (int64_t)(w0 + x) + (x == 0 ? 1 : 0)) * p.heads + h % p.heads) * p.part_rows + c;
        ml[k] = *reinterpret_cast<const floatx2*>(p.part_ml + 2 * part);
        y[k] = *reinterpret_cast<const floatx4*>(p.part_o + part * D + d);
      }
      float most = top;
#pragma unroll
      for (int k = 0; k < 4; ++k) most = fmaxf(most, ml[k].x);
      const float ref = most == -INFINITY ? 0.f : most;
      const float fade = __builtin_amdgcn_exp2f(top - ref);
      top = most;
      l *= fade;
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] *= fade;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (x0 + k * lanes >= count) continue;
        const float f = __builtin_amdgcn_exp2f(ml[k].x - ref);
        l = fmaf(ml[k].y, f, l);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = fmaf(y[k][e], f, o[e]);
      }
    }
    if (lanes > 1) {
      __syncthreads();
      s_o[t] = o;
      s_ml[t] = floatx2{top, l};
      __syncthreads();
      if (lane == 0) {
        for (int x = 1; x < lanes; ++x) top = fmaxf(top, s_ml[t + x * Q].x);
        const float ref = top == -INFINITY ? 0.f : top;
        const float own = __builtin_amdgcn_exp2f(s_ml[t].x - ref);
        l *= own;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] *= own;
        for (int x = 1; x < lanes; ++x) {
          const float f = __builtin_amdgcn_exp2f(s_ml[t + x * Q].x - ref);
          const floatx4 y = s_o[t + x * Q];
          l = fmaf(s_ml[t + x * Q].y, f, l);
#pragma unroll
          for (int e = 0; e < 4; ++e) o[e] = fmaf(y[e], f, o[e]);
        }
      }
    }
    if (there && lane == 0) write_row<D>(p, out_row(p, n, h, row0 + c), d, v_scale, top, l, o);
  }
}

template <int CT, int D>
hipError_t launch_d(const PagedDecodePlan& p, hipStream_t stream) {
  const int64_t all = (int64_t)p.N * p.row_blocks * p.Hkv;
  const dim3 grid((unsigned)(p.split ? p.split : all / p.heads));
  // one page per 16 aligned tokens, whose rows lie within 32 bits of each other
  const bool p16 = p.c.page_size % 16 == 0 && p.c.k_token < (1 << 26) && p.c.v_token < (1 << 26) &&
                   p.c.k_page < (int64_t(1) << 36) && p.c.v_page < (int64_t(1) << 36);
  const auto kern = p.tiles == 1 ? (p16 ? paged_decode_kernel<CT, D, 1, true> : paged_decode_kernel<CT, D, 1, false>)
                                 : (p16 ? paged_decode_kernel<CT, D, 2, true> : paged_decode_kernel<CT, D, 2, false>);
  const int cols = 16 * p.tiles;
  const int lds = 4 * (int)sizeof(float) * (p.heads == 4 ? 32 * cols : cols * (D + 4) + 2 * cols) +
                  (p.heads == 4 ? 4 * p.hold : 0);
  hipError_t e = hipSuccess;
  if (lds > 60 * 1024)  // with the static part, past the 64 KiB that need no asking
    e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, grid, dim3(256), lds, stream, p, p.c.table);
  e = hipGetLastError();
  if (e == hipSuccess && p.split) {
    // fewer rows per workgroup where there are few heads
    const int64_t chunks = std::min<int64_t>(p.part_rows, (512 + all - 1) / all);
    const int rows = (int)((p.part_rows + chunks - 1) / chunks);
    hipLaunchKernelGGL(paged_join_kernel<D>, dim3((unsigned)all, (unsigned)((p.part_rows + rows - 1) / rows)),
                       dim3(256), 0, stream, p, rows);
    e = hipGetLastError();
  }
  return e;
}

template <int CT>
hipError_t launch_cache(const PagedDecodePlan& p, hipStream_t stream) {
  return p.d == 128 ? launch_d<CT, 128>(p, stream)
         : p.d == 64 ? launch_d<CT, 64>(p, stream)
                     : launch_d<CT, 32>(p, stream);
}

}  // namespace paged

hipError_t launch_paged_decode_f32(const PagedDecodePlan& p, hipStream_t stream);
hipError_t launch_paged_decode_bf16(const PagedDecodePlan& p, hipStream_t stream);
hipError_t launch_paged_decode_e4m3(const PagedDecodePlan& p, hipStream_t stream);

}  // namespace kda
