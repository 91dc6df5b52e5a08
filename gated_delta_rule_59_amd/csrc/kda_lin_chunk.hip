// Linear attention with a decay for each head, over whole prompts: bf16 activations.
//
// With G_i the sum of the logarithms of the decays from a chunk's first token to token i, S the state
// that enters the chunk and C its last token:
//
//     o_i = scale (e^{G_i} S^T q_i + sum_{j <= i} (q_i . k_j) e^{G_i - G_j} v_j)
//     S  <- e^{G_C} S + sum_j k_j (e^{G_C - G_j} v_j)^T
//
// which are matrix products but for the factors. A workgroup walks chunk after chunk through one
// segment of one (sequence, head), the state in its accumulators. Segments of a sequence run in
// parallel: lin_walk_kernel<..., true, ...> sums up each segment but the last from a state of zeros, and
// lin_entries_kernel turns that into the states that enter the segments (S <- e^{G} S + Z from one to
// the next); then the others do the walk proper. Without segments only the last is
// launched.
//
// Layout. Every product is a v_mfma_f32_16x16x32_bf16. Each wave owns 16 or 32 value channels, for
// which it holds the state: rows key channels, columns value channels. Rows of a 32-channel block
// are spread over its two 16-row tiles so that the two results of a lane stacked are eight
// neighbouring key channels of a value channel, which is an operand as it stands; its partner, eight
// neighbouring channels of a query row, is one 16-byte read. Value channels are spread over a wave's
// two tiles in the same way, so that a lane's results are neighbouring channels of one token and go
// out 16 bytes at a time (o is computed transposed). Products over tokens take k and v transposed by
// the LDS on the way out (ds_read_b64_tr_b16: of a 4 x 16 block that 16 lanes address by quarter rows,
// each gets a column). (q_i . k_j) comes out transposed, which again is an operand as it stands, and is
// exchanged between the waves through LDS.
//
// Precision. bf16 inputs go into products as they are. What is no bf16 number goes in parts, each the
// rounded rest of the one before: decayed values, the state and the weights (q_i . k_j) e^{G_i - G_j} in three, which
// hold their 24 bits, whatever o's type. (With two parts of state and weights long prompts with bf16 results took
// 1.30 ms instead of 1.49, but results whose terms cancel were off by 2^-18 of the terms.) G is summed in 64 bits
// and kept in two 32-bit parts, so that a strong decay costs the differences after it nothing; exponents too have a
// second part, so that a decay of 2^-30 is as exact as one of 2^-1.
#include <algorithm>

#include "kda_lin_chunk.h"

namespace kda {

namespace {

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kC = 64;          // tokens of a chunk
constexpr unsigned kTileI = 0xffa94, kTileJ = 0xe4910;  // tiles (0, 0), (1, 0), (1, 1), (2, 0), ..., two bits each
constexpr double kHeld = 24.0;  // most that a state may be off by in the accumulators, in powers of 2

// Where channel c of row r lies in an LDS tile of rows of D. 16-byte pieces of a row change places with
// the row, so that 16 lanes that read one piece of 16 rows, and 16 lanes that read a quarter of a
// 32-channel block of each of four rows, meet all 64 banks. (Padded rows do the first only: 46 % of the
// LDS's cycles went to conflicts, of which 35 % are left, all accesses together.)
template <int D>
__device__ __forceinline__ int tile_at(int r, int c) {
  constexpr int kLog = D == 128 ? 0 : D == 64 ? 1 : 2;  // rows of 64 banks
  return r * D + ((((c >> 3) ^ ((r >> 2 & 3) | ((r & 3) >> kLog) << 2)) << 3) | (c & 7));
}

// Four 4 x 16 blocks of 16-bit values, one per 16 lanes, transposed on the way out of the LDS.
__device__ __forceinline__ s16x4 read_tr(const uint16_t* p) {
  typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
}
__device__ __forceinline__ bf16x8 pair(s16x4 a, s16x4 b) {
  typedef short s16x8 __attribute__((ext_vector_type(8)));
  return __builtin_bit_cast(bf16x8, s16x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]});
}

// The bf16 parts of N values.
template <int PARTS, int N, typename V>
__device__ __forceinline__ void parts_of(const float* x, V* y) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    f32x2 r{x[i], x[i + 1]};
#pragma unroll
    for (int k = 0; k < PARTS; ++k) {
      const bf16x2 b = __builtin_convertvector(r, bf16x2);
      y[k][i] = b[0];
      y[k][i + 1] = b[1];
      const uint32_t u = __builtin_bit_cast(uint32_t, b);
      if (k + 1 < PARTS) {
        r[0] -= __uint_as_float(u << 16);
        r[1] -= __uint_as_float(u & 0xffff0000u);
      }
    }
  }
}

template <int DK, int DV>
struct Shape {
  static constexpr int kWaves = DV == 32 ? 2 : 4, kThreads = 64 * kWaves, kTiles = DV / 16 / kWaves;
  static constexpr int kDK = DK, kDV = DV, kState = DK * DV;
  // Value channel of row r of a wave's tile c, and key channel of row r of a 32-channel block's tile e.
  static __device__ __forceinline__ int value(int wave, int c, int r) {
    return kTiles == 2 ? wave * 32 + 8 * (r >> 2) + 4 * c + (r & 3) : wave * 16 + r;
  }
  static __device__ __forceinline__ int key(int p, int e, int r) { return 32 * p + 8 * (r >> 2) + 4 * e + (r & 3); }
};

constexpr int kParts = 3;  // bf16 parts of what is a 32-bit number: its 24 bits

// SUM: sums of segments only.
template <int DK, int DV, bool SUM, typename O>
__global__ __launch_bounds__((Shape<DK, DV>::kThreads), (DK == 128 && DV == 32 ? 1 : 2)) void lin_walk_kernel(
    const LinPlan p) {
  using Sh = Shape<DK, DV>;
  constexpr int NP = SUM ? 1 : kParts;
  constexpr int NT = Sh::kThreads, NW = Sh::kWaves, CT = Sh::kTiles, KT = DK / 16;
  constexpr int QL = kC * DK / 8 / NT, VL = kC * DV / 8 / NT;  // 16-byte pieces per thread
  __shared__ __align__(16) uint16_t s_q[SUM ? 8 : kC * DK], s_k[kC * DK], s_v[kC * DV];
  __shared__ bf16x4 s_p[NP][SUM ? 1 : 4][2][64][2];  // [part][i tile][j pair][lane][j tile of the pair]
  __shared__ __align__(16) float s_hi[2][kC], s_lo[2][kC], s_w[2][kC], s_e[2][kC];
  __shared__ float s_settle[2], s_held;

  Job j;
  if (!lin_job(p, blockIdx.x, &j)) return;
  const int h = j.h, hk = h / (p.H / p.Hk);
  if (SUM && j.s == j.segments - 1) return;
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6, l15 = lane & 15, g = lane >> 4;
  const int wave_s = __builtin_amdgcn_readfirstlane(wave);
  const int begin = j.s * p.seg, len = min(p.seg, j.len - begin);
  const int64_t row0 = j.first + begin;
  const bool last = j.s == j.segments - 1;

  // the state that enters
  floatx4 S[KT][CT];
  const int64_t slot = slot_of<Sh>(p, j.slot, h);
  floatx4* const slots = static_cast<floatx4*>(p.workspace) + slot;
#pragma unroll
  for (int kt = 0; kt < KT; ++kt)
#pragma unroll
    for (int c = 0; c < CT; ++c) S[kt][c] = floatx4{0.f, 0.f, 0.f, 0.f};
  if (!SUM && j.segments > 1) {
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int c = 0; c < CT; ++c) S[kt][c] = slots[((wave * KT + kt) * CT + c) * 64 + lane];
  } else if (!SUM && p.S0) {
    const float* in = p.S0 + ((int64_t)j.n * p.H + h) * Sh::kState;
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int c = 0; c < CT; ++c)
#pragma unroll
        for (int x = 0; x < 4; ++x)
          S[kt][c][x] = in[Sh::key(kt >> 1, kt & 1, 4 * g + x) * DV + Sh::value(wave, c, l15)];
  }

  const char* const qp = p.q + row0 * p.q_token + hk * p.q_head;
  const char* const kp = p.k + row0 * p.k_token + hk * p.k_head;
  const char* const vp = p.v + row0 * p.v_token + h * p.v_head;
  const unsigned q_row = (unsigned)p.q_token, k_row = (unsigned)p.k_token, v_row = (unsigned)p.v_token;
  u32x4 rq[SUM ? 1 : QL], rk[QL], rv[VL];
  constexpr int kGates = NW - 1;  // a wave with fewer weights to form than others
  uint32_t gate = 0;   // that wave: a token's
  double total = 0.0;  // that wave: of the chunks so far, to base 2
  // The chunk's rows; those past the end are the last one again: o has no room for theirs, and to the
  // state they do not count (s_w).
  auto fetch = [&](int c0) {
    const unsigned most = len - 1 - c0;
#pragma unroll
    for (int i = 0; i < QL; ++i) {
      const unsigned x = t + i * NT, r = min(x / (DK / 8), most), e = x % (DK / 8) * 16;
      rk[i] = *reinterpret_cast<const u32x4*>(kp + c0 * p.k_token + (r * k_row + e));
      if (!SUM) rq[i] = *reinterpret_cast<const u32x4*>(qp + c0 * p.q_token + (r * q_row + e));
    }
#pragma unroll
    for (int i = 0; i < VL; ++i) {
      const unsigned x = t + i * NT, r = min(x / (DV / 8), most), e = x % (DV / 8) * 16;
      rv[i] = *reinterpret_cast<const u32x4*>(vp + c0 * p.v_token + (r * v_row + e));
    }
  };
  auto fetch_gate = [&](int c0) {  // as it is in memory: converting it would wait for it here
    const int64_t i = p.fixed ? h : (row0 + min(c0 + lane, len - 1)) * p.H + h;
    gate = p.gate_bf16 ? static_cast<const uint16_t*>(p.g)[i] : static_cast<const uint32_t*>(p.g)[i];
  };
  // The chunk's sums of logarithms (to base 2), and its factors. The state in the accumulators times
  // 2^held is the one meant: while 2^held is near 1, only new values are scaled (by its inverse) and the
  // accumulators stay as they are.
  double held = 0.0;
  auto sum_gates = [&](uint32_t gate, int c0, int to) {
    // a decay below e^-1000 is 0 in any case, and -infinity would leave differences undefined
    const bool real = c0 + lane < len;
    const float ln = __uint_as_float(p.gate_bf16 ? gate << 16 : gate);
    const double G = wave_sums(real ? (double)(ln < -1000.f ? -1000.f : ln) * 1.4426950408889634 : 0.0);
    const double all = lane_of(G, 63);
    const Log to_here(G), meant(G + held);
    s_hi[to][lane] = to_here.hi;
    s_lo[to][lane] = to_here.lo;
    s_e[to][lane] = p.scale * exp2_of(meant.hi, meant.lo);
    const double next = held + all;
    const bool settle = !(fabs(next) <= kHeld);
    const float w = settle ? exp2_between(lane_of(to_here.hi, 63), lane_of(to_here.lo, 63), to_here.hi, to_here.lo)
                           : exp2_of(-meant.hi, -meant.lo);
    s_w[to][lane] = real ? w : 0.f;
    if (lane == 0) s_settle[to] = settle ? exp2_of(next) : 1.f;
    held = lane_of(settle ? 0.0 : next, 0);
    if (SUM) total = lane_of(total + all, 0);
  };
  if (!SUM && t < 64) {  // weights above the diagonal that products read: tiles (0, 1) and (2, 3)
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      s_p[k][0][0][t][1] = bf16x4{0.f, 0.f, 0.f, 0.f};
      s_p[k][2][1][t][1] = bf16x4{0.f, 0.f, 0.f, 0.f};
    }
  }
  if (len > 0) {
    if (wave == kGates) {
      fetch_gate(0);
      const uint32_t had = gate;
      fetch_gate(kC);
      sum_gates(had, 0, 0);
    }
    fetch(0);
  }

  for (int c0 = 0; c0 < len; c0 += kC) {
    const int now = c0 / kC & 1;
    if (c0) lds_barrier();
#pragma unroll
    for (int i = 0; i < QL; ++i) {
      const int x = t + i * NT, at = tile_at<DK>(x / (DK / 8), x % (DK / 8) * 8);
      *reinterpret_cast<u32x4*>(&s_k[at]) = rk[i];
      if (!SUM) *reinterpret_cast<u32x4*>(&s_q[at]) = rq[i];
    }
#pragma unroll
    for (int i = 0; i < VL; ++i) {
      const int x = t + i * NT;
      *reinterpret_cast<u32x4*>(&s_v[tile_at<DV>(x / (DV / 8), x % (DV / 8) * 8)]) = rv[i];
    }
    lds_barrier();
    if (c0 + kC < len) {
      const uint32_t had = gate;
      if (wave == kGates) fetch_gate(c0 + 2 * kC);
      fetch(c0 + kC);
      if (wave == kGates) sum_gates(had, c0 + kC, now ^ 1);
    }

    // values, a column each
    bf16x8 v[2][CT];
    auto read_values = [&] {
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int c = 0; c < CT; ++c) {
          const uint16_t* at = &s_v[tile_at<DV>(4 * g + (l15 >> 2), Sh::value(wave, c, 4 * (l15 & 3))) + 32 * s * DV];
          v[s][c] = pair(read_tr(at), read_tr(at + 16 * DV));
        }
    };
    if (SUM) read_values();
    if (!SUM) {
      // Weights (q_i . k_j) e^{G_i - G_j}, 16 x 16 at a time, transposed (rows j, columns i). The ten
      // tiles with j <= i go round the waves.
#pragma unroll
      for (int x = 0; x < (10 + NW - 1) / NW; ++x) {
        int n = wave_s + x * NW;
        if (n >= 10) break;
        asm volatile("" : "+s"(n));  // keeps the tiles' LDS addresses out of registers between chunks
        const int it = kTileI >> (2 * n) & 3, jt = kTileJ >> (2 * n) & 3;
        floatx4 d{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int ks = 0; ks < DK / 32; ++ks)
          d = mfma_bf16(*reinterpret_cast<const bf16x8*>(&s_k[tile_at<DK>(l15, ks * 32 + 8 * g) + jt * 16 * DK]),
                        *reinterpret_cast<const bf16x8*>(&s_q[tile_at<DK>(l15, ks * 32 + 8 * g) + it * 16 * DK]), d);
        const int i = it * 16 + l15, j0 = jt * 16 + 4 * g;
        const float hi = s_hi[now][i], lo = s_lo[now][i];
        const floatx4 jhi = *reinterpret_cast<const floatx4*>(&s_hi[now][j0]);
        const floatx4 jlo = *reinterpret_cast<const floatx4*>(&s_lo[now][j0]);
        float w[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const float z = d[y] * (p.scale * exp2_between(hi, lo, jhi[y], jlo[y]));
          w[y] = j0 + y <= i ? z : 0.f;
        }
        bf16x4 parts[NP];
        parts_of<NP, 4>(w, parts);
#pragma unroll
        for (int k = 0; k < NP; ++k) s_p[k][it][jt >> 1][lane][jt & 1] = parts[k];
      }
      // S^T q, while the other workgroup's waves are in front of their products as far as may be
      __builtin_amdgcn_s_setprio(1);
      floatx4 o[4][CT];
#pragma unroll
      for (int it = 0; it < 4; ++it)
#pragma unroll
        for (int c = 0; c < CT; ++c) o[it][c] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int ks = 0; ks < DK / 32; ++ks) {
        bf16x8 sp[CT][NP];
#pragma unroll
        for (int c = 0; c < CT; ++c) {
          const float x[8] = {S[2 * ks][c][0],     S[2 * ks][c][1],     S[2 * ks][c][2],     S[2 * ks][c][3],
                              S[2 * ks + 1][c][0], S[2 * ks + 1][c][1], S[2 * ks + 1][c][2], S[2 * ks + 1][c][3]};
          parts_of<NP, 8>(x, sp[c]);
        }
        bf16x8 q[4];
#pragma unroll
        for (int it = 0; it < 4; ++it)
          q[it] = *reinterpret_cast<const bf16x8*>(&s_q[tile_at<DK>(it * 16 + l15, ks * 32 + 8 * g)]);
#pragma unroll
        for (int k = 0; k < NP; ++k)
#pragma unroll
          for (int it = 0; it < 4; ++it)
#pragma unroll
            for (int c = 0; c < CT; ++c) o[it][c] = mfma_bf16(sp[c][k], q[it], o[it][c]);
      }
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        const float a = s_e[now][it * 16 + l15];
#pragma unroll
        for (int c = 0; c < CT; ++c) o[it][c] *= a;
      }
      lds_barrier();
      read_values();
#pragma unroll
      for (int s = 0; s < 2; ++s) {
#pragma unroll
        for (int k = 0; k < NP; ++k)
#pragma unroll
          for (int it = 2 * s; it < 4; ++it) {
            const bf16x8 w = *reinterpret_cast<const bf16x8*>(&s_p[k][it][s][lane]);
#pragma unroll
            for (int c = 0; c < CT; ++c) o[it][c] = mfma_bf16(v[s][c], w, o[it][c]);
          }
      }
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        const int i = c0 + it * 16 + l15;
        if (i < len) {
          O* out = static_cast<O*>(p.o) + ((row0 + i) * p.H + h) * DV + Sh::value(wave, 0, 4 * g);
#pragma unroll
          for (int c = 0; c < CT; ++c) store4(out + 4 * c, o[it][c]);
        }
      }
    }

    // the state that leaves the chunk
    if (!SUM) __builtin_amdgcn_s_setprio(0);
    const float settle = s_settle[now];
    if (settle != 1.f) {
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int c = 0; c < CT; ++c) S[kt][c] *= settle;
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      bf16x8 vw[CT][kParts];
      const floatx4 w0 = *reinterpret_cast<const floatx4*>(&s_w[now][32 * s + 4 * g]);
      const floatx4 w1 = *reinterpret_cast<const floatx4*>(&s_w[now][32 * s + 16 + 4 * g]);
#pragma unroll
      for (int c = 0; c < CT; ++c) {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = static_cast<float>(v[s][c][i]) * (i < 4 ? w0[i] : w1[i - 4]);
        parts_of<kParts, 8>(x, vw[c]);
      }
      constexpr int kAtOnce = KT < 4 ? KT : 4;
#pragma unroll
      for (int k0 = 0; k0 < KT; k0 += kAtOnce) {
        bf16x8 k[kAtOnce];
#pragma unroll
        for (int x = 0; x < kAtOnce; ++x) {
          const int kt = k0 + x;
          const uint16_t* at =
              &s_k[tile_at<DK>(4 * g + (l15 >> 2), Sh::key(kt >> 1, kt & 1, 4 * (l15 & 3))) + 32 * s * DK];
          k[x] = pair(read_tr(at), read_tr(at + 16 * DK));
        }
#pragma unroll
        for (int y = 0; y < kParts; ++y)
#pragma unroll
          for (int x = 0; x < kAtOnce; ++x)
#pragma unroll
            for (int c = 0; c < CT; ++c) S[k0 + x][c] = mfma_bf16(k[x], vw[c][y], S[k0 + x][c]);
      }
    }
  }

  if (SUM || (last && p.S_T)) {
    if (t == kGates * 64) s_held = exp2_of(held);
    lds_barrier();
    const float f = s_held;
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int c = 0; c < CT; ++c) S[kt][c] *= f;
  }
  if (SUM) {
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int c = 0; c < CT; ++c) slots[((wave * KT + kt) * CT + c) * 64 + lane] = S[kt][c];
    if (t == kGates * 64) decays_of(p)[(int64_t)j.slot * p.H + h] = exp2_of(total);
  } else if (last && p.S_T) {
    float* out = p.S_T + ((int64_t)j.n * p.H + h) * Sh::kState;
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int c = 0; c < CT; ++c)
#pragma unroll
        for (int x = 0; x < 4; ++x)
          out[Sh::key(kt >> 1, kt & 1, 4 * g + x) * DV + Sh::value(wave, c, l15)] = S[kt][c][x];
  }
}

template <int DK, int DV>
hipError_t launch(const LinPlan& p, hipStream_t stream) {
  const dim3 grid((unsigned)((int64_t)p.jobs * p.H));
  constexpr int threads = Shape<DK, DV>::kThreads;
  launch_before<Shape<DK, DV>>(
      p, stream, [&] { lin_walk_kernel<DK, DV, true, float><<<sums_grid(p), threads, 0, stream>>>(p); });
  if (p.out_bf16)
    lin_walk_kernel<DK, DV, false, uint16_t><<<grid, threads, 0, stream>>>(p);
  else
    lin_walk_kernel<DK, DV, false, float><<<grid, threads, 0, stream>>>(p);
  return hipGetLastError();
}

template <int DK>
hipError_t launch_dk(const LinPlan& p, hipStream_t stream) {
  return p.dv == 32 ? launch<DK, 32>(p, stream) : p.dv == 64 ? launch<DK, 64>(p, stream) : launch<DK, 128>(p, stream);
}

}  // namespace

size_t plan_lin_chunk(LinPlan* p) {
  // Workgroups: two fit a CU and there are 256 CUs. With 256 pairs of sequence and head there are no
  // segments (8 x 32 pairs of 8,448 tokens: 727 us, in two segments each 804: a segment's sum is work
  // that the walk proper does again). Below, segments of 512 tokens or more for 512 workgroups (16 pairs of
  // 16,384 tokens: 132 us, with 256 workgroups 142), shorter ones, of 128 at least, for 256, which are
  // done sooner each (16 pairs of 4,096: 51 us, with 512 workgroups 56; 8 pairs of 1,024: 28.6 us in segments of 128,
  // 40 of 256). Packed sequences, whose lengths the host does not know, are cut as if
  // all tokens were one sequence.
  //
  // Those are bf16 of 128 x 128. Other shapes, whose workgroups are smaller, take the same cut; halved and doubled:
  // 5 x 6 pairs of 1,003 fp32 tokens of 64 x 32 25.7 us, 23.6 and 40.3; 16 of 4,096 fp32 of 128 x 128 100, 99 and 168;
  // 16 of 4,096 bf16 of 64 x 32 29.8, 25.3 and 46.2; 256 of 8,448 fp32 of 128 x 128 1,750 and halved 2,190.
  const int64_t pairs = (int64_t)p->n_seq * p->H, tokens = p->cu_seqlens ? p->T : (int64_t)p->n_seq * p->T;
  const auto cut = [&](int64_t groups) {
    const int64_t len = p->cu_seqlens ? (tokens * p->H + groups - 1) / groups
                                      : ((int64_t)p->T + std::max<int64_t>(1, groups / pairs) - 1) /
                                            std::max<int64_t>(1, groups / pairs);
    return std::min<int64_t>(std::max<int64_t>(128, (len + kC - 1) / kC * kC), 1 << 30);
  };
  int64_t seg = cut(256);
  if (pairs < 256 && seg > 512) seg = std::max<int64_t>(512, cut(512));
  // Up to four chunks of bf16 are walked sooner than they are summed up first: 16 pairs of 256 tokens of 128 x 128 24.2
  // us in one segment and 26.2 in two, 8 of 200 of 64 x 64 14.1 and 17.3. Not so eight of fp32: 53.7 and 47.8.
  if (p->T <= 256 && p->act_bf16) seg = 256;
  p->seg = (int)seg;
  const int64_t per = std::max<int64_t>(1, ((int64_t)p->T + p->seg - 1) / p->seg);
  p->jobs = (int)(p->cu_seqlens && p->T > p->seg ? p->T / p->seg + p->n_seq : per * p->n_seq);
  p->slots = p->T <= p->seg ? 0 : p->cu_seqlens ? std::min(p->jobs, 2 * (p->T / p->seg)) : p->jobs;
  const size_t states = sizeof(float) * (size_t)p->slots * p->H * ((size_t)p->dk * p->dv + 1);
  if (!p->cu_seqlens || p->n_seq <= 64) return states;
  p->tables = (states + 15) / 16 * 16;
  return p->tables + sizeof(int) * (((size_t)p->n_seq + 1) / 2 * 2 + 2 * (size_t)p->jobs);
}

hipError_t launch_lin_chunk(const LinPlan& p, hipStream_t stream) {
  if (!p.act_bf16) return launch_lin_chunk_f32(p, stream);
  return p.dk == 32 ? launch_dk<32>(p, stream) : p.dk == 64 ? launch_dk<64>(p, stream) : launch_dk<128>(p, stream);
}

}  // namespace kda
