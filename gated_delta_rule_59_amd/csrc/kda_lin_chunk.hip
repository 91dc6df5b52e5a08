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
// parallel: lin_walk_kernel<..., true> sums up each segment but the last from a state of zeros, and
// lin_entries_kernel turns that into the states that enter the segments (S <- e^{G} S + Z from one to
// the next); then lin_walk_kernel<..., false> does the walk proper. Without segments only the last is
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
// rounded rest of the one before: the state and the weights (q_i . k_j) e^{G_i - G_j} in two (2^-17
// each, what o has beside its own rounding), decayed values in three (exact to 2^-25: the state adds
// up thousands of them, and is a 32-bit result). Two of them for the state would leave it off by
// 1.6e-6. G is summed in 64 bits and kept in two 32-bit parts, so that a strong decay costs the
// differences after it nothing.
#include <algorithm>

#include "kda_lin.h"

namespace kda {

namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kC = 64;      // tokens of a chunk
constexpr int kPad = 8;     // of an LDS row: 16 neighbouring rows begin in different banks

// Which segment of which sequence job `job` is: false if there is none.
struct Job {
  int n, s, segments;
  int64_t first;   // the sequence's first row
  int len;         // its tokens
};
__device__ __forceinline__ int segments_of(const LinPlan& p, int len) { return len ? (len - 1) / p.seg + 1 : 1; }

__device__ __forceinline__ bool lin_job(const LinPlan& p, int job, Job* j) {
  if (!p.cu_seqlens) {
    j->segments = segments_of(p, p.T);
    j->n = job / j->segments;
    j->s = job % j->segments;
    lin_tokens(p, j->n, &j->first, &j->len);
    return true;
  }
  const int lane = threadIdx.x & 63;
  int before = 0;
  for (int n0 = 0; n0 < p.n_seq; n0 += 64) {
    int64_t first;
    int len = 0, x = 0;
    if (n0 + lane < p.n_seq) {
      lin_tokens(p, n0 + lane, &first, &len);
      x = segments_of(p, len);
    }
    int to = x;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int y = __shfl_up(to, d, 64);
      if (lane >= d) to += y;
    }
    const uint64_t past = __ballot(before + to > job);
    if (past) {
      const int l = __builtin_ctzll(past);
      j->n = n0 + l;
      j->s = job - before - __shfl(to - x, l, 64);
      j->segments = __shfl(x, l, 64);
      lin_tokens(p, j->n, &j->first, &j->len);
      return true;
    }
    before += __shfl(to, 63, 64);
  }
  return false;
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

// The two or three bf16 parts of eight values.
template <int PARTS>
__device__ __forceinline__ void parts_of(const float* x, bf16x8* y) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float r = x[i];
#pragma unroll
    for (int k = 0; k < PARTS; ++k) {
      const __bf16 b = static_cast<__bf16>(r);
      y[k][i] = b;
      if (k + 1 < PARTS) r -= static_cast<float>(b);
    }
  }
}

__device__ __forceinline__ float exp2_of(float x) { return __builtin_amdgcn_exp2f(x); }

template <int DK, int DV>
struct Shape {
  static constexpr int kWaves = DV == 32 ? 2 : 4, kThreads = 64 * kWaves, kTiles = DV / 16 / kWaves;
  static constexpr int kState = DK * DV;
  // Value channel of row r of a wave's tile c, and key channel of row r of a 32-channel block's tile e.
  static __device__ __forceinline__ int value(int wave, int c, int r) {
    return kTiles == 2 ? wave * 32 + 8 * (r >> 2) + 4 * c + (r & 3) : wave * 16 + r;
  }
  static __device__ __forceinline__ int key(int p, int e, int r) { return 32 * p + 8 * (r >> 2) + 4 * e + (r & 3); }
};

// A state in the workspace: [wave][key tile][value tile][lane] of four key rows each.
template <int DK, int DV>
__device__ __forceinline__ int64_t slot_of(const LinPlan& p, int64_t job, int h) {
  return (job * p.H + h) * (DK * DV / 4);
}
__device__ __forceinline__ float* decays_of(const LinPlan& p) {
  return static_cast<float*>(p.workspace) + (int64_t)p.jobs * p.H * p.dk * p.dv;
}

template <int DK, int DV, bool SUM>
__global__ __launch_bounds__((Shape<DK, DV>::kThreads), 2) void lin_walk_kernel(const LinPlan p) {
  using Sh = Shape<DK, DV>;
  constexpr int NT = Sh::kThreads, NW = Sh::kWaves, CT = Sh::kTiles, KT = DK / 16;
  constexpr int SK = DK + kPad, SV = DV + kPad;
  constexpr int QL = kC * DK / 8 / NT, VL = kC * DV / 8 / NT;  // 16-byte pieces per thread
  __shared__ __align__(16) uint16_t s_q[SUM ? 8 : kC * SK], s_k[kC * SK], s_v[kC * SV];
  __shared__ bf16x8 s_p[SUM ? 1 : 2][SUM ? 1 : 4][2][64];
  __shared__ __align__(16) float s_hi[kC], s_lo[kC], s_w[kC];
  __shared__ float s_all;

  const int job = blockIdx.x / p.H, h = blockIdx.x % p.H, hk = h / (p.H / p.Hk);
  Job j;
  if (!lin_job(p, job, &j)) return;
  if (SUM && j.s == j.segments - 1) return;
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6, l15 = lane & 15, g = lane >> 4;
  const int begin = j.s * p.seg, len = min(p.seg, j.len - begin);
  const int64_t row0 = j.first + begin;
  const bool last = j.s == j.segments - 1;

  // the state that enters
  floatx4 S[KT][CT];
  const int64_t slot = slot_of<DK, DV>(p, job, h);
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

  const char* const qp = p.q + hk * p.q_head;
  const char* const kp = p.k + hk * p.k_head;
  const char* const vp = p.v + h * p.v_head;
  u32x4 rq[SUM ? 1 : QL], rk[QL], rv[VL];
  float gate = 0.f;
  auto fetch = [&](int c0) {  // rows past the end are zeros
#pragma unroll
    for (int i = 0; i < QL; ++i) {
      const int x = t + i * NT, r = x / (DK / 8), e = x % (DK / 8) * 16;
      const bool real = c0 + r < len;
      const int64_t row = row0 + c0 + r;
      rk[i] = real ? *reinterpret_cast<const u32x4*>(kp + row * p.k_token + e) : u32x4{0, 0, 0, 0};
      if (!SUM) rq[i] = real ? *reinterpret_cast<const u32x4*>(qp + row * p.q_token + e) : u32x4{0, 0, 0, 0};
    }
#pragma unroll
    for (int i = 0; i < VL; ++i) {
      const int x = t + i * NT, r = x / (DV / 8), e = x % (DV / 8) * 16;
      rv[i] = c0 + r < len ? *reinterpret_cast<const u32x4*>(vp + (row0 + c0 + r) * p.v_token + e) : u32x4{0, 0, 0, 0};
    }
    if (wave == 0) gate = c0 + lane < len ? lin_gate(p, row0 + c0 + lane, h) : 0.f;
  };
  double total = 0.0;  // SUM, wave 0: of the chunks so far, log2
  if (len > 0) fetch(0);

  for (int c0 = 0; c0 < len; c0 += kC) {
    if (c0) __syncthreads();
#pragma unroll
    for (int i = 0; i < QL; ++i) {
      const int x = t + i * NT, at = x / (DK / 8) * SK + x % (DK / 8) * 8;
      *reinterpret_cast<u32x4*>(&s_k[at]) = rk[i];
      if (!SUM) *reinterpret_cast<u32x4*>(&s_q[at]) = rq[i];
    }
#pragma unroll
    for (int i = 0; i < VL; ++i) {
      const int x = t + i * NT;
      *reinterpret_cast<u32x4*>(&s_v[x / (DV / 8) * SV + x % (DV / 8) * 8]) = rv[i];
    }
    if (wave == 0) {
      // a decay below e^-1000 is 0 in any case, and -infinity would leave differences undefined
      double G = (double)(gate < -1000.f ? -1000.f : gate) * 1.4426950408889634;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const double y = __shfl_up(G, d, 64);
        if (lane >= d) G += y;
      }
      const double all = __shfl(G, 63, 64);
      const float hi = (float)G;
      s_hi[lane] = hi;
      s_lo[lane] = (float)(G - (double)hi);
      s_w[lane] = exp2_of((float)(all - G));
      if (lane == 0) s_all = exp2_of((float)all);
      total += all;
    }
    __syncthreads();
    if (c0 + kC < len) fetch(c0 + kC);

    if (!SUM) {
      // weights (q_i . k_j) e^{G_i - G_j} of i tile `it`, transposed: rows j, columns i
#pragma unroll
      for (int x = 0; x < 4 / NW; ++x) {
        const int it = x ? 3 - wave : wave;
        const int i = it * 16 + l15;
        const float hi = s_hi[i], lo = s_lo[i];
        bf16x8 q[DK / 32];
#pragma unroll
        for (int ks = 0; ks < DK / 32; ++ks) q[ks] = *reinterpret_cast<const bf16x8*>(&s_q[i * SK + ks * 32 + 8 * g]);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if (2 * s > it) continue;
          float w[8];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int jt = 2 * s + e;
            floatx4 d{0.f, 0.f, 0.f, 0.f};
            if (jt <= it) {
#pragma unroll
              for (int ks = 0; ks < DK / 32; ++ks)
                d = mfma_bf16(*reinterpret_cast<const bf16x8*>(&s_k[(jt * 16 + l15) * SK + ks * 32 + 8 * g]), q[ks], d);
            }
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const int jj = jt * 16 + 4 * g + y;
              w[4 * e + y] = jj <= i ? d[y] * exp2_of((hi - s_hi[jj]) + (lo - s_lo[jj])) : 0.f;
            }
          }
          bf16x8 parts[2];
          parts_of<2>(w, parts);
          s_p[0][it][s][lane] = parts[0];
          s_p[1][it][s][lane] = parts[1];
        }
      }
      // S^T q
      floatx4 o[4][CT];
#pragma unroll
      for (int it = 0; it < 4; ++it)
#pragma unroll
        for (int c = 0; c < CT; ++c) o[it][c] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int ks = 0; ks < DK / 32; ++ks) {
        bf16x8 sp[CT][2];
#pragma unroll
        for (int c = 0; c < CT; ++c) {
          const float x[8] = {S[2 * ks][c][0],     S[2 * ks][c][1],     S[2 * ks][c][2],     S[2 * ks][c][3],
                              S[2 * ks + 1][c][0], S[2 * ks + 1][c][1], S[2 * ks + 1][c][2], S[2 * ks + 1][c][3]};
          parts_of<2>(x, sp[c]);
        }
        bf16x8 q[4];
#pragma unroll
        for (int it = 0; it < 4; ++it)
          q[it] = *reinterpret_cast<const bf16x8*>(&s_q[(it * 16 + l15) * SK + ks * 32 + 8 * g]);
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int it = 0; it < 4; ++it)
#pragma unroll
            for (int c = 0; c < CT; ++c) o[it][c] = mfma_bf16(sp[c][k], q[it], o[it][c]);
      }
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        const float a = exp2_of(s_hi[it * 16 + l15]);
#pragma unroll
        for (int c = 0; c < CT; ++c) o[it][c] *= a;
      }
      __syncthreads();
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        bf16x8 v[CT];
#pragma unroll
        for (int c = 0; c < CT; ++c) {
          const uint16_t* at = &s_v[(32 * s + 4 * g + (l15 >> 2)) * SV + Sh::value(wave, c, 4 * (l15 & 3))];
          v[c] = pair(read_tr(at), read_tr(at + 16 * SV));
        }
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int it = 2 * s; it < 4; ++it) {
            const bf16x8 w = s_p[k][it][s][lane];
#pragma unroll
            for (int c = 0; c < CT; ++c) o[it][c] = mfma_bf16(v[c], w, o[it][c]);
          }
      }
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        const int i = c0 + it * 16 + l15;
        if (i < len) {
          const int64_t e = ((row0 + i) * p.H + h) * DV + Sh::value(wave, 0, 4 * g);
          if (p.out_bf16) {
            uint16_t* out = static_cast<uint16_t*>(p.o) + e;
#pragma unroll
            for (int c = 0; c < CT; ++c) {
              s16x4 y;
#pragma unroll
              for (int x = 0; x < 4; ++x) y[x] = (short)lin_bf16(p.scale * o[it][c][x]);
              *reinterpret_cast<s16x4*>(out + 4 * c) = y;
            }
          } else {
            float* out = static_cast<float*>(p.o) + e;
#pragma unroll
            for (int c = 0; c < CT; ++c) *reinterpret_cast<floatx4*>(out + 4 * c) = p.scale * o[it][c];
          }
        }
      }
    }

    // the state that leaves the chunk
    const float all = s_all;
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int c = 0; c < CT; ++c) S[kt][c] *= all;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      bf16x8 vw[CT][3];
      const floatx4 w0 = *reinterpret_cast<const floatx4*>(&s_w[32 * s + 4 * g]);
      const floatx4 w1 = *reinterpret_cast<const floatx4*>(&s_w[32 * s + 16 + 4 * g]);
#pragma unroll
      for (int c = 0; c < CT; ++c) {
        const uint16_t* at = &s_v[(32 * s + 4 * g + (l15 >> 2)) * SV + Sh::value(wave, c, 4 * (l15 & 3))];
        const s16x4 a = read_tr(at), b = read_tr(at + 16 * SV);
        float x[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[i] = bf16_bits_to_f32((uint16_t)a[i]) * w0[i];
          x[4 + i] = bf16_bits_to_f32((uint16_t)b[i]) * w1[i];
        }
        parts_of<3>(x, vw[c]);
      }
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) {
        const uint16_t* at = &s_k[(32 * s + 4 * g + (l15 >> 2)) * SK + Sh::key(kt >> 1, kt & 1, 4 * (l15 & 3))];
        const bf16x8 k = pair(read_tr(at), read_tr(at + 16 * SK));
#pragma unroll
        for (int y = 0; y < 3; ++y)
#pragma unroll
          for (int c = 0; c < CT; ++c) S[kt][c] = mfma_bf16(k, vw[c][y], S[kt][c]);
      }
    }
  }

  if (SUM) {
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int c = 0; c < CT; ++c) slots[((wave * KT + kt) * CT + c) * 64 + lane] = S[kt][c];
    if (t == 0) decays_of(p)[(int64_t)job * p.H + h] = exp2_of((float)total);
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

// From the sums of a sequence's segments to the states that enter them, in the sums' place. A thread
// takes four key rows of a value channel through all segments.
template <int DK, int DV>
__global__ __launch_bounds__(256) void lin_entries_kernel(const LinPlan p) {
  using Sh = Shape<DK, DV>;
  constexpr int CT = Sh::kTiles, KT = DK / 16;
  constexpr int kGroups = (Sh::kState / 4 + 255) / 256;
  const int part = blockIdx.x % kGroups, nh = blockIdx.x / kGroups, n = nh / p.H, h = nh % p.H;
  const int i = part * 256 + threadIdx.x;
  int64_t first;
  int len, job = 0;
  lin_tokens(p, n, &first, &len);
  const int segments = segments_of(p, len);
  if (segments == 1) return;
  if (p.cu_seqlens) {
    for (int m = threadIdx.x & 63; m < n; m += 64) {
      int64_t f;
      int l;
      lin_tokens(p, m, &f, &l);
      job += segments_of(p, l);
    }
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) job += __shfl_xor(job, d, 64);
  } else {
    job = n * segments;
  }
  const int there = min(segments, p.jobs - job);  // offsets that overlap give more segments than jobs
  if (i >= Sh::kState / 4) return;
  floatx4 e{0.f, 0.f, 0.f, 0.f};
  if (p.S0) {
    const int lane = i % 64, tile = i / 64, c = tile % CT, kt = tile / CT % KT, wave = tile / CT / KT;
    const float* in = p.S0 + (int64_t)nh * Sh::kState;
#pragma unroll
    for (int x = 0; x < 4; ++x)
      e[x] = in[Sh::key(kt >> 1, kt & 1, 4 * (lane >> 4) + x) * DV + Sh::value(wave, c, lane & 15)];
  }
  floatx4* at = static_cast<floatx4*>(p.workspace) + i;
  const float* decays = decays_of(p);
  constexpr int kAhead = 8;
  for (int s0 = 0; s0 < there; s0 += kAhead) {
    floatx4 z[kAhead];
    float a[kAhead];
#pragma unroll
    for (int s = 0; s < kAhead; ++s) {
      z[s] = floatx4{0.f, 0.f, 0.f, 0.f};
      a[s] = 1.f;
      if (s0 + s < there && s0 + s + 1 < segments) {
        z[s] = at[slot_of<DK, DV>(p, job + s0 + s, h)];
        a[s] = decays[(int64_t)(job + s0 + s) * p.H + h];
      }
    }
#pragma unroll
    for (int s = 0; s < kAhead; ++s) {
      if (s0 + s < there) {
        at[slot_of<DK, DV>(p, job + s0 + s, h)] = e;
        e = e * a[s] + z[s];
      }
    }
  }
}

template <int DK, int DV>
hipError_t launch(const LinPlan& p, hipStream_t stream) {
  const dim3 grid((unsigned)((int64_t)p.jobs * p.H));
  constexpr int threads = Shape<DK, DV>::kThreads;
  if (p.T > p.seg) {
    lin_walk_kernel<DK, DV, true><<<grid, threads, 0, stream>>>(p);
    constexpr int groups = (DK * DV / 4 + 255) / 256;
    lin_entries_kernel<DK, DV><<<dim3((unsigned)((int64_t)p.n_seq * p.H * groups)), 256, 0, stream>>>(p);
  }
  lin_walk_kernel<DK, DV, false><<<grid, threads, 0, stream>>>(p);
  return hipGetLastError();
}

template <int DK>
hipError_t launch_dk(const LinPlan& p, hipStream_t stream) {
  return p.dv == 32 ? launch<DK, 32>(p, stream) : p.dv == 64 ? launch<DK, 64>(p, stream) : launch<DK, 128>(p, stream);
}

// Two workgroups fit a CU: enough segments for 512 workgroups, of 256 tokens at least.
constexpr int kWalks = 512, kShortest = 256;

}  // namespace

size_t plan_lin_chunk(LinPlan* p) {
  if (!p->act_bf16) {
    p->seg = std::max(p->T, 1);
    p->jobs = p->n_seq;
    return 0;
  }
  const int64_t tokens = p->cu_seqlens ? p->T : (int64_t)p->n_seq * p->T;
  const int64_t want = (tokens * p->H + kWalks - 1) / kWalks;
  p->seg = (int)std::min<int64_t>(std::max<int64_t>(kShortest, (want + kC - 1) / kC * kC), 1 << 30);
  const int64_t per = std::max<int64_t>(1, ((int64_t)p->T + p->seg - 1) / p->seg);
  p->jobs = (int)(p->cu_seqlens ? p->T / p->seg + p->n_seq : per * p->n_seq);
  if (p->T <= p->seg) return 0;
  return sizeof(float) * (size_t)p->jobs * p->H * ((size_t)p->dk * p->dv + 1);
}

hipError_t launch_lin_chunk(const LinPlan& p, hipStream_t stream) {
  if (!p.act_bf16) return launch_lin_recurrent(p, stream);
  return p.dk == 32 ? launch_dk<32>(p, stream) : p.dk == 64 ? launch_dk<64>(p, stream) : launch_dk<128>(p, stream);
}

}  // namespace kda
