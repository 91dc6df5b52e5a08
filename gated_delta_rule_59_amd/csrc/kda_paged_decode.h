// Attention of a few new tokens per sequence over a paged cache: the kernels, by cache type.
//
// For each key/value head, the rows (new token j, query head of the group) of a sequence share
// every key and value, so S^T = K Q^T and O^T = V^T P^T are matrix products with up to 16 rows
// as the columns of one 16 x 16 tile. One pass over the cache keeps the running maximum and sum
// of each row's softmax:
//     M' = max(M, max s),  l' = l 2^{M - M'} + sum 2^{s - M'},  O' = O 2^{M - M'} + sum 2^{s - M'} v
// (s in units of log2). The cache is read once and nothing else is large: HBM bounds it.
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
// Rounding: products and sums are held in 32 bits. P is split into two bf16 parts (16
// significant bits, an error of 2^-17 of each weight), which costs a second V product that
// hides under the loads; one part alone (2^-9) would double the error of a bf16 result. An e4m3
// value is a bf16 value exactly. fp32 caches take the fp32 matrix instruction throughout.
//
// Who sees what. Rows of a block differ in what they see only near the newest token and the
// window's far edge. The tokens that all of them see go through the matrix product; for the
// others ("private" ones, at most m - 1 at each end) V enters it as zero and they are added by
// predicated multiply-adds, so a NaN or an infinity in a value that a row does not see never
// meets that row, not even multiplied by zero. Values no row sees are replaced by zero as well.
#pragma once

#include <math.h>

#include "kda_device.h"
#include "kda_internal.h"
#include "kda_paged.h"

namespace kda {
namespace paged {

constexpr int kUnit = 128;  // tokens a workgroup takes at a time: 32 by each of four waves

// The new tokens of sequence n see positions [0, len); with a window, the first of them begins
// at len - m + 1 - window.
__device__ __forceinline__ int seq_len(const PagedDecodePlan& p, int n) {
  return min(max(p.seq_lens[n], 0), p.max_len);
}
__device__ __forceinline__ int first_unit(const PagedDecodePlan& p, int len) {
  if (!p.window) return 0;
  const int64_t lo = (int64_t)len - p.m + 1 - p.window;
  return lo > 0 ? (int)(lo / kUnit) : 0;
}
// Units of kUnit tokens that a sequence's workgroups walk; one at least, which writes zeros.
__device__ __forceinline__ int seq_units(const PagedDecodePlan& p, int len) {
  return max(1, (len + kUnit - 1) / kUnit - first_unit(p, len));
}

// Sum over the workgroup's 256 threads (every thread gets it).
__device__ __forceinline__ int64_t block_sum(int64_t x, int64_t* s4) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) x += __shfl_xor(x, m, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s4[threadIdx.x >> 6] = x;
  __syncthreads();
  return s4[0] + s4[1] + s4[2] + s4[3];
}

// How the units of all (sequence, row block, head)s are shared: workgroup w of `gd` takes units
// [start(w), start(w + 1)) of the total.
struct Share {
  int64_t total;
  int gd;
  __device__ __forceinline__ int64_t start(int64_t w) const { return total * w / gd; }
  // the workgroup that has unit u
  __device__ __forceinline__ int owner(int64_t u) const {
    return (int)(((u + 1) * gd + total - 1) / total) - 1;
  }
};
__device__ __forceinline__ Share make_share(const PagedDecodePlan& p, int64_t total) {
  return Share{total, (int)(total < p.split ? total : (int64_t)p.split)};
}

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

template <int W>
__device__ __forceinline__ void load_words(const char* p, uint32_t* w) {
  if constexpr (W == 1) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (W == 2) {
    const u32x2 x = *reinterpret_cast<const u32x2*>(p);
    w[0] = x[0]; w[1] = x[1];
  } else {
#pragma unroll
    for (int c = 0; c < W; c += 4) {
      const u32x4 x = *reinterpret_cast<const u32x4*>(p + 4 * c);
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
// Elements 2h and 2h + 1 of four e4m3 values.
template <bool H>
__device__ __forceinline__ floatx2 e4m3_pair(uint32_t w) {
  return __builtin_amdgcn_cvt_pk_f32_fp8((int)w, H);
}
// Eight e4m3 values as a bf16 operand (exact: the dropped halves are zero).
__device__ __forceinline__ bf16x8 e4m3_operand(uint32_t w0, uint32_t w1) {
  const floatx2 a = e4m3_pair<false>(w0), b = e4m3_pair<true>(w0);
  const floatx2 c = e4m3_pair<false>(w1), d = e4m3_pair<true>(w1);
  const u32x4 v = {halves_hi(__float_as_uint(a.x), __float_as_uint(a.y)),
                   halves_hi(__float_as_uint(b.x), __float_as_uint(b.y)),
                   halves_hi(__float_as_uint(c.x), __float_as_uint(c.y)),
                   halves_hi(__float_as_uint(d.x), __float_as_uint(d.y))};
  return __builtin_bit_cast(bf16x8, v);
}

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

// P16: page_size is a multiple of 16, so 16 aligned tokens have one page.
template <int CT, int D, int NT, bool P16>
__global__ __launch_bounds__(256, 2) void paged_decode_kernel(
    const PagedDecodePlan p, const int32_t* __restrict__ block_table) {
  using TY = Types<CT, D>;
  constexpr int VEC = TY::VEC;
  constexpr int COLS = 16 * NT;
  constexpr int OS = D + 4;  // floats per row of s_o (staggered over the LDS banks)
  __shared__ __align__(16) float s_o[4][COLS * OS];
  __shared__ float s_m[4][COLS], s_l[4][COLS];
  __shared__ int64_t s_scan[4];
  __shared__ int s_n;
  __shared__ int64_t s_at;

  const int t = threadIdx.x, lane = t & 63, r = lane & 15, g = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(t >> 6);
  const int per_seq = p.row_blocks * p.Hkv;

  // ---- this workgroup's units
  int n;
  int64_t at;    // unit within sequence n (units of its first (row block, head) first)
  int64_t left;  // units to do
  if (p.split == 0) {
    n = blockIdx.x / per_seq;
    const int un = seq_units(p, seq_len(p, n));
    at = (int64_t)(blockIdx.x % per_seq) * un;
    left = un;
  } else {
    const int c = (p.N + 255) / 256;
    int64_t mine = 0;
    for (int i = 0; i < c; ++i)
      if (t * c + i < p.N) mine += seq_units(p, seq_len(p, t * c + i));
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
    const Share share = make_share(p, total);
    if ((int)blockIdx.x >= share.gd) return;
    const int64_t u0 = share.start(blockIdx.x);
    left = share.start(blockIdx.x + 1) - u0;
    int64_t excl = before + incl - mine;
    if (excl <= u0 && u0 < excl + mine) {
      int i = t * c;
      for (;; ++i) {
        const int64_t ui = (int64_t)seq_units(p, seq_len(p, i)) * per_seq;
        if (u0 < excl + ui || i + 1 == p.N) break;
        excl += ui;
      }
      s_n = i;
      s_at = u0 - excl;
    }
    __syncthreads();
    n = s_n;
    at = s_at;
  }

  const float log2_scale = p.scale * kLog2e;

  // ---- one (row block, head) of one sequence after the other
  while (left > 0) {
    n = __builtin_amdgcn_readfirstlane(n);
    const int len = __builtin_amdgcn_readfirstlane(seq_len(p, n));
    const int un = seq_units(p, len);
    const int pair = __builtin_amdgcn_readfirstlane((int)(at / un));
    const int u_first = __builtin_amdgcn_readfirstlane((int)(at % un));
    const int cnt = __builtin_amdgcn_readfirstlane((int)min((int64_t)(un - u_first), left));
    const int rb = pair / p.Hkv, h = pair % p.Hkv;
    const int row0 = rb * COLS;
    const int rows = min(COLS, p.rows - row0);

    // what the rows see: row of new token j sees [lo(j), hi(j))
    auto hi_of = [&](int j) { return len - p.m + 1 + j; };
    auto lo_of = [&](int j) {
      return p.window ? (int)max((int64_t)0, (int64_t)hi_of(j) - p.window) : 0;
    };
    const int j_first = row0 / p.group, j_last = (row0 + rows - 1) / p.group;
    const int all_lo = lo_of(j_last), all_hi = hi_of(j_first);  // seen by every row
    const int any_lo = lo_of(j_first), any_hi = hi_of(j_last);  // seen by one at least

    // ---- the query rows: columns r of NT tiles, as B operands. fp32 rows are scaled here (a
    // score then overflows only if it is itself out of range), bf16 ones keep their values and
    // the scores are scaled.
    const float to_log2 = log2_scale * (p.c.k_scale ? p.c.k_scale[h] : 1.f);
    uint32_t q[NT][TY::QW];
    int lo[NT], hi[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int row = row0 + nt * 16 + r;
      const bool there = row < p.rows;
      const int j = there ? row / p.group : 0, head = h * p.group + (there ? row % p.group : 0);
      lo[nt] = there ? lo_of(j) : 0;
      hi[nt] = there ? hi_of(j) : 0;
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
#pragma unroll
      for (int s = 0; s < TY::QW; ++s) {
        if (CT == kF32) q[nt][s] = __float_as_uint(__uint_as_float(q[nt][s]) * to_log2);
        q[nt][s] = there ? q[nt][s] : 0u;
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

    // ---- this wave's tiles: tokens [base + 128 i, + 32), those that some row sees
    const int base = (first_unit(p, len) + u_first) * kUnit + 32 * wv;
    int i0 = any_lo > base + 31 ? (any_lo - base - 32) / kUnit + 1 : 0;
    int i1 = any_hi > base ? min(cnt, (any_hi - base - 1) / kUnit + 1) : 0;

    const int32_t* pages = block_table + n * p.c.table_stride;
    const char* kh = p.c.k + h * p.c.k_head;
    const char* vh = p.c.v + h * p.c.v_head;
    const int last = any_hi - 1;  // the newest token that some row sees (>= 0 if i0 < i1)

    // Where a tile's rows lie. Tokens past `last` give their place to it or to a slot of its page,
    // and ids of no page to page 0; what they read is masked below.
    // P16: 16 tokens have one page, so the rows' base is uniform and a lane adds 32 bits to it.
    constexpr int IDS = P16 ? 2 : 10;  // page ids: of the two halves, or of the lane's 2 + 8 rows
    const unsigned k_lane = (unsigned)(r * (int)p.c.k_token) + g * 4 * TY::KC;
    const unsigned v_lane = (unsigned)(4 * g * (int)p.c.v_token) + r * TY::VB;
    // token of key row s (s = 0, 1), and of value row i (i = 0 .. 7)
    auto k_token = [&](int tb, int s) { return min(tb + 16 * s + (P16 ? 0 : r), P16 ? last & ~15 : last); };
    auto v_token = [&](int tb, int i) { return min(tb + 16 * (i >> 2) + 4 * g + (i & 3), last); };
    auto page_at = [&](int tok) { return pages[div_page(p.c, (unsigned)tok)]; };
    auto is_page = [&](int id) { return (unsigned)id < (unsigned)p.c.num_pages; };
    auto look_up = [&](int tb, int* id) {
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        id[s] = page_at(k_token(tb, s));
        if (P16) id[s] = __builtin_amdgcn_readfirstlane(id[s]);
      }
      if constexpr (!P16) {
#pragma unroll
        for (int i = 0; i < 8; ++i) id[2 + i] = page_at(v_token(tb, i));
      }
    };
    auto row_at = [&](int id, int tok, int64_t page, int64_t token) {
      const int slot = tok - div_page(p.c, (unsigned)tok) * p.c.page_size;
      return (is_page(id) ? id : 0) * page + slot * token;
    };

    uint32_t kw[2][TY::KW], vw[8][TY::VW];
    auto load_k = [&](int tb, const int* id) {
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const char* row = kh + row_at(id[s], k_token(tb, s), p.c.k_page, p.c.k_token);
        const unsigned off = P16 ? k_lane : g * 4 * TY::KC;
#pragma unroll
        for (int c = 0; c < TY::NKL; ++c)
          load_words<TY::KC>(row + off + c * 16 * TY::KC, &kw[s][c * TY::KC]);
      }
    };
    auto load_v = [&](int tb, const int* id) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const char* row;
        if constexpr (P16)
          row = vh + row_at(id[i >> 2], k_token(tb, i >> 2), p.c.v_page, p.c.v_token) +
                (i & 3) * p.c.v_token + v_lane;
        else
          row = vh + row_at(id[2 + i], v_token(tb, i), p.c.v_page, p.c.v_token) + r * TY::VB;
        load_bytes<TY::VB>(row, vw[i]);
      }
    };

    int ids[IDS], ids1[IDS], ids2[P16 ? IDS : 1];  // of this tile, the next, the one after
    if (i0 < i1) {
      look_up(base + kUnit * i0, ids1);
      load_k(base + kUnit * i0, ids1);
      if constexpr (P16) look_up(base + kUnit * (i0 + 1), ids2);
    }
    for (int i = i0; i < i1; ++i) {
      const int tb = base + kUnit * i;
#pragma unroll
      for (int x = 0; x < IDS; ++x) {
        ids[x] = ids1[x];
        if constexpr (P16) ids1[x] = ids2[x];
      }
      load_v(tb, ids);
      if constexpr (!P16) look_up(tb + kUnit, ids1);

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
      load_k(tb + kUnit, ids1);
      if constexpr (P16) look_up(tb + 2 * kUnit, ids2);

      // tokens that not every row sees, or that are on no page
      bool on_pages = true;
#pragma unroll
      for (int x = P16 ? 0 : 2; x < IDS; ++x) on_pages = on_pages && is_page(ids[x]);
      const bool plain = tb >= all_lo && tb + 32 <= all_hi && (P16 ? on_pages : __all(on_pages));
      // Bit i of `sees` / `shared`: this lane's row / every row sees token slot i. Applied in
      // every tile: a branch around them would make copies of the values, which waits for them.
      unsigned sees[NT], shared = 0xffu;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) sees[nt] = 0xffu;
      if (!plain) {
        shared = 0;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) sees[nt] = 0;
#pragma unroll
        for (int i8 = 0; i8 < 8; ++i8) {
          const int tok = tb + 4 * g + (i8 & 3) + 16 * (i8 >> 2);
          const bool in = is_page(ids[P16 ? i8 >> 2 : 2 + i8]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            sees[nt] |= in && tok >= lo[nt] && tok < hi[nt] ? 1u << i8 : 0u;
          shared |= in && tok >= all_lo && tok < all_hi ? 1u << i8 : 0u;
        }
      }
#pragma unroll
      for (int i8 = 0; i8 < 8; ++i8) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          s[nt][i8 >> 2][i8 & 3] = sees[nt] >> i8 & 1 ? s[nt][i8 >> 2][i8 & 3] * (CT == kF32 ? 1.f : to_log2)
                                                      : -INFINITY;
        const uint32_t keep = 0u - (shared >> i8 & 1);
#pragma unroll
        for (int e = 0; e < TY::VW; ++e) vw[i8][e] &= keep;
      }

      // running maximum and sum of each row
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float mx = fmaxf(fmaxf(fmaxf(s[nt][0][0], s[nt][0][1]), fmaxf(s[nt][0][2], s[nt][0][3])),
                         fmaxf(fmaxf(s[nt][1][0], s[nt][1][1]), fmaxf(s[nt][1][2], s[nt][1][3])));
        mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
        mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
        const float now = fmaxf(top[nt], mx);
        const float ref = now == -INFINITY ? 0.f : now;
        const float fade = __builtin_amdgcn_exp2f(top[nt] - ref);
        top[nt] = now;
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
        bf16x8 p_hi[NT], p_lo[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i8 = 0; i8 < 8; ++i8) {
            __bf16 a, b;
            split_bf16(s[nt][i8 >> 2][i8 & 3], a, b);
            p_hi[nt][i8] = a;
            p_lo[nt][i8] = b;
          }
        auto product = [&](int j, const u32x4& frag) {
          const bf16x8 a = __builtin_bit_cast(bf16x8, frag);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            acc[nt][j] = mfma_bf16(a, p_hi[nt], acc[nt][j]);
            acc[nt][j] = mfma_bf16(a, p_lo[nt], acc[nt][j]);
          }
        };
#pragma unroll
        for (int j = 0; j < VEC; j += 2) {
          u32x4 f0, f1;
#pragma unroll
          for (int a = 0; a < 4; ++a) {
            if constexpr (CT == kBF16) {
              f0[a] = halves_lo(vw[2 * a][j / 2], vw[2 * a + 1][j / 2]);
              f1[a] = halves_hi(vw[2 * a][j / 2], vw[2 * a + 1][j / 2]);
            } else {
              const floatx2 x = j & 2 ? e4m3_pair<true>(vw[2 * a][j / 4]) : e4m3_pair<false>(vw[2 * a][j / 4]);
              const floatx2 y = j & 2 ? e4m3_pair<true>(vw[2 * a + 1][j / 4]) : e4m3_pair<false>(vw[2 * a + 1][j / 4]);
              f0[a] = halves_hi(__float_as_uint(x.x), __float_as_uint(y.x));
              f1[a] = halves_hi(__float_as_uint(x.y), __float_as_uint(y.y));
            }
          }
          product(j, f0);
          product(j + 1, f1);
        }
      }

      // private tokens, row by row
      const int pv0 = max(tb, any_lo), pv1 = min(tb + 32, any_hi);
      if (!plain && (pv0 < all_lo || pv1 > all_hi)) {
        float* ps = s_o[wv];  // [token][column]
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

    // ---- the four waves' parts of each row become one
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      sum[nt] += __shfl_xor(sum[nt], 16, 64);
      sum[nt] += __shfl_xor(sum[nt], 32, 64);
      if (g == 0) {
        s_m[wv][nt * 16 + r] = top[nt];
        s_l[wv][nt * 16 + r] = sum[nt];
      }
    }
    __syncthreads();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int c = nt * 16 + r;
      const float now = fmaxf(fmaxf(s_m[0][c], s_m[1][c]), fmaxf(s_m[2][c], s_m[3][c]));
      const float fade = __builtin_amdgcn_exp2f(top[nt] - (now == -INFINITY ? 0.f : now));
      float* dst = &s_o[wv][c * OS + g * (D / 4)];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (VEC >= 4) {
#pragma unroll
          for (int j = 0; j < VEC; j += 4)
            *reinterpret_cast<floatx4*>(dst + VEC * e + j) =
                floatx4{acc[nt][j][e] * fade, acc[nt][j + 1][e] * fade, acc[nt][j + 2][e] * fade,
                        acc[nt][j + 3][e] * fade};
        } else {
#pragma unroll
          for (int j = 0; j < VEC; ++j) dst[VEC * e + j] = acc[nt][j][e] * fade;
        }
      }
    }
    __syncthreads();
    const bool whole = cnt == un;
    const int64_t slot = 2 * (int64_t)blockIdx.x + (u_first == 0 ? 1 : 0);
    for (int x = t; x < rows * (D / 4); x += 256) {
      const int c = x / (D / 4), d = x % (D / 4) * 4;
      float now = -INFINITY, l = 0.f;
      floatx4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < 4; ++w) now = fmaxf(now, s_m[w][c]);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        l += s_l[w][c] * __builtin_amdgcn_exp2f(s_m[w][c] - (now == -INFINITY ? 0.f : now));
        o += *reinterpret_cast<const floatx4*>(&s_o[w][c * OS + d]);
      }
      if (whole) {
        const float inv = l == 0.f ? 0.f : (p.c.v_scale ? p.c.v_scale[h] : 1.f) / l;
        const int row = row0 + c, j = row / p.group, head = h * p.group + row % p.group;
        const int64_t dst = (((int64_t)n * p.m + j) * p.Hq + head) * D + d;
        if (l == 0.f) o = floatx4{0.f, 0.f, 0.f, 0.f};
        else o = floatx4{o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv};
        if (p.out_bf16)
          *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(p.o) + dst) =
              u32x2{pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3])};
        else
          *reinterpret_cast<floatx4*>(static_cast<float*>(p.o) + dst) = o;
        if (p.lse && d == 0)
          p.lse[((int64_t)n * p.m + j) * p.Hq + head] =
              l == 0.f ? -INFINITY : (now + log2f(l)) * 0.6931471805599453f;
      } else {
        *reinterpret_cast<floatx4*>(p.part_o + (slot * COLS + c) * D + d) = o;
        if (d == 0) {
          p.part_ml[(slot * COLS + c) * 2] = now;
          p.part_ml[(slot * COLS + c) * 2 + 1] = l;
        }
      }
    }
    __syncthreads();  // s_o, s_m and s_l are free again

    left -= cnt;
    at += cnt;
    if (at == (int64_t)un * per_seq) {
      ++n;
      at = 0;
    }
  }
}

// Joins the parts of the (sequence, row block, head)s that several workgroups shared. One
// workgroup each; those that one workgroup did alone are finished already.
template <int D>
__global__ __launch_bounds__(256) void paged_join_kernel(const PagedDecodePlan p) {
  __shared__ int64_t s_scan[4];
  const int t = threadIdx.x;
  const int per_seq = p.row_blocks * p.Hkv, cols = 16 * p.tiles;
  const int n = blockIdx.x / per_seq, pair = blockIdx.x % per_seq;
  const int rb = pair / p.Hkv, h = pair % p.Hkv;
  int64_t before = 0, total = 0;
  for (int i = t; i < p.N; i += 256) {
    const int u = seq_units(p, seq_len(p, i));
    total += u;
    if (i < n) before += u;
  }
  total = block_sum(total, s_scan) * per_seq;
  before = block_sum(before, s_scan) * per_seq;
  const int un = seq_units(p, seq_len(p, n));
  const Share share = make_share(p, total);
  const int64_t u0 = before + (int64_t)pair * un;
  const int w0 = share.owner(u0), w1 = share.owner(u0 + un - 1);
  if (w0 == w1) return;

  const int row0 = rb * cols, rows = min(cols, p.rows - row0);
  for (int x = t; x < rows * (D / 4); x += 256) {
    const int c = x / (D / 4), d = x % (D / 4) * 4;
    // part of workgroup w: the first one begins the head (slot 1), the others continue it (slot 0)
    auto slot = [&](int w) { return (2 * (int64_t)w + (w == w0 ? 1 : 0)) * cols + c; };
    float now = -INFINITY;
    for (int w = w0; w <= w1; ++w) now = fmaxf(now, p.part_ml[slot(w) * 2]);
    const float ref = now == -INFINITY ? 0.f : now;
    float l = 0.f;
    floatx4 o = {0.f, 0.f, 0.f, 0.f};
    for (int w = w0; w <= w1; ++w) {
      const int64_t s = slot(w);
      const float fade = __builtin_amdgcn_exp2f(p.part_ml[s * 2] - ref);
      l += p.part_ml[s * 2 + 1] * fade;
      const floatx4 y = *reinterpret_cast<const floatx4*>(p.part_o + s * D + d);
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = fmaf(y[e], fade, o[e]);
    }
    const int row = row0 + c, j = row / p.group, head = h * p.group + row % p.group;
    const int64_t dst = (((int64_t)n * p.m + j) * p.Hq + head) * D + d;
    const float inv = (p.c.v_scale ? p.c.v_scale[h] : 1.f) / l;
    if (l == 0.f) o = floatx4{0.f, 0.f, 0.f, 0.f};
    else o = floatx4{o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv};
    if (p.out_bf16)
      *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(p.o) + dst) =
          u32x2{pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3])};
    else
      *reinterpret_cast<floatx4*>(static_cast<float*>(p.o) + dst) = o;
    if (p.lse && d == 0)
      p.lse[((int64_t)n * p.m + j) * p.Hq + head] =
          l == 0.f ? -INFINITY : (now + log2f(l)) * 0.6931471805599453f;
  }
}

template <int CT, int D>
hipError_t launch_d(const PagedDecodePlan& p, hipStream_t stream) {
  const int64_t all = (int64_t)p.N * p.row_blocks * p.Hkv;
  const dim3 grid((unsigned)(p.split ? p.split : all));
  // one page per 16 aligned tokens, whose rows lie within 32 bits of each other
  const bool p16 = p.c.page_size % 16 == 0 && p.c.k_token < (1 << 26) && p.c.v_token < (1 << 26);
  auto kern = p.tiles == 1 ? (p16 ? paged_decode_kernel<CT, D, 1, true> : paged_decode_kernel<CT, D, 1, false>)
                           : (p16 ? paged_decode_kernel<CT, D, 2, true> : paged_decode_kernel<CT, D, 2, false>);
  hipLaunchKernelGGL(kern, grid, dim3(256), 0, stream, p, p.c.table);
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && p.split) {
    hipLaunchKernelGGL(paged_join_kernel<D>, dim3((unsigned)all), dim3(256), 0, stream, p);
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
