// Linear attention with a decay for each head, over whole prompts: fp32 activations.
//
// The walk of kda_lin_chunk.hip (its formulas, segments and state layout by waves) with chunks of 32
// tokens and v_mfma_f32_16x16x4_f32, a sixteenth of the bf16 rate, which bounds it: 32-bit operands go
// in as they are, and the result is a 32-bit one throughout.
//
// Lane l gives an operand's row l & 15 at place l >> 4 of four along the contraction. Four products
// in turn take what a lane has in four registers, so that place g of product x is element 4 g + x of
// 16: one 16-byte read of a row, or the four rows of a result that a lane holds. Results thus are
// operands as they stand here too (o and the weights are computed transposed), and channels need not
// change places. Rows of the LDS are padded by four: reads of 16 rows, and of four rows by 16 lanes
// each, meet all banks.
#include "kda_lin_chunk.h"

namespace kda {

namespace {

constexpr int kF32Chunk = 32, kPad = 4;

template <int DK, int DV>
struct ShapeF32 {
  static constexpr int kWaves = DV == 32 ? 2 : 4, kThreads = 64 * kWaves, kTiles = DV / 16 / kWaves;
  static constexpr int kDK = DK, kDV = DV, kState = DK * DV;
  static __device__ __forceinline__ int value(int wave, int c, int r) { return (wave * kTiles + c) * 16 + r; }
  static __device__ __forceinline__ int key(int p, int e, int r) { return 32 * p + 16 * e + r; }
};

__device__ __forceinline__ floatx4 mfma_f32(float a, float b, const floatx4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

template <int DK, int DV, bool SUM, typename O>
__global__ __launch_bounds__((ShapeF32<DK, DV>::kThreads), 2) void lin_walk_f32_kernel(const LinPlan p) {
  using Sh = ShapeF32<DK, DV>;
  constexpr int C = kF32Chunk, NT = Sh::kThreads, NW = Sh::kWaves, CT = Sh::kTiles, KT = DK / 16;
  constexpr int SK = DK + kPad, SV = DV + kPad;
  constexpr int QL = C * DK / 4 / NT, VL = C * DV / 4 / NT;  // 16-byte pieces per thread
  __shared__ __align__(16) float s_q[SUM ? 4 : C * SK], s_k[C * SK], s_v[C * SV];
  __shared__ floatx4 s_p[3][64];  // weights of (i tile, j tile) (0, 0), (1, 0), (1, 1)
  __shared__ __align__(16) float s_hi[C], s_lo[C], s_w[C], s_e[C];
  __shared__ float s_all;

  Job j;
  if (!lin_job(p, blockIdx.x, &j)) return;
  const int h = j.h, hk = h / (p.H / p.Hk);
  if (SUM && j.s == j.segments - 1) return;
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6, l15 = lane & 15, g = lane >> 4;
  const int begin = j.s * p.seg, len = min(p.seg, j.len - begin);
  const int64_t row0 = j.first + begin;
  const bool last = j.s == j.segments - 1;

  floatx4 S[KT][CT];
  floatx4* const slots = static_cast<floatx4*>(p.workspace) + slot_of<Sh>(p, j.slot, h);
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
  floatx4 rq[SUM ? 1 : QL], rk[QL], rv[VL];
  float gate = 0.f;
  // Rows past the end are the last one again: o has no room for theirs, and to the state they do not
  // count (s_w).
  auto fetch = [&](int c0) {
    const unsigned most = len - 1 - c0;
    if (wave == 0) gate = lin_gate(p, row0 + min(c0 + lane, len - 1), h);
#pragma unroll
    for (int i = 0; i < QL; ++i) {
      const unsigned x = t + i * NT, r = min(x / (DK / 4), most), e = x % (DK / 4) * 16;
      rk[i] = *reinterpret_cast<const floatx4*>(kp + c0 * p.k_token + (r * k_row + e));
      if (!SUM) rq[i] = *reinterpret_cast<const floatx4*>(qp + c0 * p.q_token + (r * q_row + e));
    }
#pragma unroll
    for (int i = 0; i < VL; ++i) {
      const unsigned x = t + i * NT, r = min(x / (DV / 4), most), e = x % (DV / 4) * 16;
      rv[i] = *reinterpret_cast<const floatx4*>(vp + c0 * p.v_token + (r * v_row + e));
    }
  };
  double total = 0.0;  // wave 0: of the chunks so far, to base 2
  if (len > 0) fetch(0);

  for (int c0 = 0; c0 < len; c0 += C) {
    if (c0) lds_barrier();
#pragma unroll
    for (int i = 0; i < QL; ++i) {
      const int x = t + i * NT, at = x / (DK / 4) * SK + x % (DK / 4) * 4;
      *reinterpret_cast<floatx4*>(&s_k[at]) = rk[i];
      if (!SUM) *reinterpret_cast<floatx4*>(&s_q[at]) = rq[i];
    }
#pragma unroll
    for (int i = 0; i < VL; ++i) {
      const int x = t + i * NT;
      *reinterpret_cast<floatx4*>(&s_v[x / (DV / 4) * SV + x % (DV / 4) * 4]) = rv[i];
    }
    if (wave == 0) {
      // a decay below e^-1000 is 0 in any case, and -infinity would leave differences undefined
      const bool real = lane < C && c0 + lane < len;
      const double G = wave_sums(real ? (double)(gate < -1000.f ? -1000.f : gate) * 1.4426950408889634 : 0.0);
      const double all = lane_of(G, 63);
      const Log to_here(G);
      const float all_hi = lane_of(to_here.hi, 63), all_lo = lane_of(to_here.lo, 63);
      if (lane < C) {
        s_hi[lane] = to_here.hi;
        s_lo[lane] = to_here.lo;
        s_e[lane] = p.scale * exp2_of(to_here.hi, to_here.lo);
        s_w[lane] = real ? exp2_between(all_hi, all_lo, to_here.hi, to_here.lo) : 0.f;
      }
      if (lane == 0) s_all = exp2_of(all_hi, all_lo);
      if (SUM) total += all;
    }
    lds_barrier();
    if (c0 + C < len) fetch(c0 + C);

    if (!SUM) {
      // weights (q_i . k_j) e^{G_i - G_j}, transposed (rows j, columns i)
      for (int n = wave; n < 3; n += NW) {
        const int i = (n > 0) * 16 + l15, jt = n == 2;
        floatx4 d{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int u = 0; u < KT; ++u) {
          const floatx4 a = *reinterpret_cast<const floatx4*>(&s_k[(jt * 16 + l15) * SK + 16 * u + 4 * g]);
          const floatx4 b = *reinterpret_cast<const floatx4*>(&s_q[i * SK + 16 * u + 4 * g]);
#pragma unroll
          for (int x = 0; x < 4; ++x) d = mfma_f32(a[x], b[x], d);
        }
        const int j0 = jt * 16 + 4 * g;
        const floatx4 jhi = *reinterpret_cast<const floatx4*>(&s_hi[j0]);
        const floatx4 jlo = *reinterpret_cast<const floatx4*>(&s_lo[j0]);
        const float hi = s_hi[i], lo = s_lo[i];
        floatx4 w;
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const float z = d[y] * (p.scale * exp2_between(hi, lo, jhi[y], jlo[y]));
          w[y] = j0 + y <= i ? z : 0.f;
        }
        s_p[n][lane] = w;
      }
      // S^T q
      floatx4 o[2][CT];
#pragma unroll
      for (int it = 0; it < 2; ++it)
#pragma unroll
        for (int c = 0; c < CT; ++c) o[it][c] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) {
        floatx4 q[2];
#pragma unroll
        for (int it = 0; it < 2; ++it)
          q[it] = *reinterpret_cast<const floatx4*>(&s_q[(it * 16 + l15) * SK + 16 * kt + 4 * g]);
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
          for (int it = 0; it < 2; ++it)
#pragma unroll
            for (int c = 0; c < CT; ++c) o[it][c] = mfma_f32(S[kt][c][x], q[it][x], o[it][c]);
      }
#pragma unroll
      for (int it = 0; it < 2; ++it) {
        const float a = s_e[it * 16 + l15];
#pragma unroll
        for (int c = 0; c < CT; ++c) o[it][c] *= a;
      }
      lds_barrier();
#pragma unroll
      for (int n = 0; n < 3; ++n) {
        const floatx4 w = s_p[n][lane];
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
          for (int c = 0; c < CT; ++c) {
            const float v = s_v[((n == 2) * 16 + 4 * g + x) * SV + Sh::value(wave, c, l15)];
            o[n > 0][c] = mfma_f32(v, w[x], o[n > 0][c]);
          }
      }
#pragma unroll
      for (int it = 0; it < 2; ++it) {
        const int i = c0 + it * 16 + l15;
        if (i < len) {
          O* out = static_cast<O*>(p.o) + ((row0 + i) * p.H + h) * DV;
#pragma unroll
          for (int c = 0; c < CT; ++c) store4(out + Sh::value(wave, c, 4 * g), o[it][c]);
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
    for (int jt = 0; jt < 2; ++jt) {
      const floatx4 w = *reinterpret_cast<const floatx4*>(&s_w[jt * 16 + 4 * g]);
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int r = jt * 16 + 4 * g + x;
        float v[CT];
#pragma unroll
        for (int c = 0; c < CT; ++c) v[c] = s_v[r * SV + Sh::value(wave, c, l15)] * w[x];
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) {
          const float k = s_k[r * SK + 16 * kt + l15];
#pragma unroll
          for (int c = 0; c < CT; ++c) S[kt][c] = mfma_f32(k, v[c], S[kt][c]);
        }
      }
    }
  }

  if (SUM) {
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int c = 0; c < CT; ++c) slots[((wave * KT + kt) * CT + c) * 64 + lane] = S[kt][c];
    if (t == 0) decays_of(p)[(int64_t)j.slot * p.H + h] = exp2_of(total);
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
hipError_t launch_f32(const LinPlan& p, hipStream_t stream) {
  const dim3 grid((unsigned)((int64_t)p.jobs * p.H));
  constexpr int threads = ShapeF32<DK, DV>::kThreads;
  launch_before<ShapeF32<DK, DV>>(
      p, stream, [&] { lin_walk_f32_kernel<DK, DV, true, float><<<sums_grid(p), threads, 0, stream>>>(p); });
  if (p.out_bf16)
    lin_walk_f32_kernel<DK, DV, false, uint16_t><<<grid, threads, 0, stream>>>(p);
  else
    lin_walk_f32_kernel<DK, DV, false, float><<<grid, threads, 0, stream>>>(p);
  return hipGetLastError();
}

template <int DK>
hipError_t launch_f32_dk(const LinPlan& p, hipStream_t stream) {
  return p.dv == 32 ? launch_f32<DK, 32>(p, stream)
                    : p.dv == 64 ? launch_f32<DK, 64>(p, stream) : launch_f32<DK, 128>(p, stream);
}

}  // namespace

hipError_t launch_lin_chunk_f32(const LinPlan& p, hipStream_t stream) {
  return p.dk == 32 ? launch_f32_dk<32>(p, stream)
                    : p.dk == 64 ? launch_f32_dk<64>(p, stream) : launch_f32_dk<128>(p, stream);
}

}  // namespace kda
