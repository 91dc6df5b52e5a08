// Linear attention with a decay for each head, token by token:
//
//     S <- e^{g_t} S + k_t v_t^T;   o_t = scale S_t^T q_t
//
// for the new token or the drafts of each sequence. The state is read once and written once, 4 dk dv
// bytes each way per (sequence, head), beside which a token's own rows are nothing: HBM bounds it. (512
// sequences of 32 heads of 128 x 128, 2.15 GB: 374 us, torch's product in place 358; verification,
// which only reads: 161 us.)
//
// One 256-thread workgroup per (n, h). Thread t owns value columns 4 (t % CG) .. + 3 (CG = DV / 4) and
// key rows t / CG + RG i (RG = 256 / CG): 16 bytes at t plus 4 KiB per i, so a wave reads 1 KiB pieces,
// the state stays in registers between the read and the write, and the addresses take one register.
// Fewer registers for more workgroups at a time cost more in spills than they bring (at most 96: 5 us
// more, 72: 96 us). A call of one token has a kernel of its own, which writes a row as soon as it
// is done (385 us as drafts are done). Drafts come four at a time through LDS; their results are summed over
// the row groups there.
//
// All in 32 bits. The state after `accept` tokens is written when it is reached, and the tokens
// behind it go on from it, so results do not depend on what is accepted.
#include "kda_device.h"
#include "kda_internal.h"
#include "kda_lin.h"

namespace kda {

namespace {

constexpr int kTokens = 4;  // at a time

template <int DK, int DV, typename T>
__global__ __launch_bounds__(256) void lin_recurrent_kernel(const LinPlan p) {
  constexpr int CG = DV / 4, RG = 256 / CG, RPT = DK / RG, WR = RG / 4;  // WR: row groups of a wave
  static_assert(RPT >= 1 && WR >= 1, "shape");
  __shared__ float2 s_kq[kTokens][DK];
  __shared__ __align__(16) float s_v[kTokens][DV];
  __shared__ float s_a[kTokens];
  __shared__ __align__(16) float s_o[kTokens][4][DV];

  const int n = blockIdx.x / p.H, h = blockIdx.x % p.H, hk = h / (p.H / p.Hk);
  const int t = threadIdx.x, cg = t % CG, rg = t / CG, wave = t >> 6;
  const int64_t first = (int64_t)n * p.T;
  const int len = p.T;
  const int take = p.accept ? min(max(p.accept[n], 0), len) : len;

  const int64_t at = (int64_t)blockIdx.x * DK * DV;
  floatx4 s[RPT];
  const floatx4* in = reinterpret_cast<const floatx4*>(p.S0 + at);
#pragma unroll
  for (int i = 0; i < RPT; ++i) s[i] = __builtin_nontemporal_load(in + 256 * i + (unsigned)t);
  floatx4* out = reinterpret_cast<floatx4*>(p.S_T + at);

  for (int j0 = 0; j0 < len; j0 += kTokens) {
    const int m = min(kTokens, len - j0);
    if (j0) __syncthreads();
    for (int x = t; x < m * (2 * DK + DV); x += 256) {
      const int j = x / (2 * DK + DV), c = x % (2 * DK + DV);
      const int64_t tok = first + j0 + j;
      if (c < DK) {
        s_kq[j][c].y = ld(reinterpret_cast<const T*>(p.q + tok * p.q_token + hk * p.q_head), c);
      } else if (c < 2 * DK) {
        s_kq[j][c - DK].x = ld(reinterpret_cast<const T*>(p.k + tok * p.k_token + hk * p.k_head), c - DK);
      } else {
        s_v[j][c - 2 * DK] = ld(reinterpret_cast<const T*>(p.v + tok * p.v_token + h * p.v_head), c - 2 * DK);
      }
    }
    if (t < m) s_a[t] = expf(lin_gate(p, first + j0 + t, h));
    __syncthreads();
    floatx4 o[kTokens];
#pragma unroll
    for (int j = 0; j < kTokens; ++j) {
      o[j] = floatx4{0.f, 0.f, 0.f, 0.f};
      if (j >= m) continue;
      const float a = s_a[j];
      const floatx4 v = *reinterpret_cast<const floatx4*>(&s_v[j][4 * cg]);
#pragma unroll
      for (int i = 0; i < RPT; ++i) {
        const float kr = s_kq[j][rg + RG * i].x, qr = s_kq[j][rg + RG * i].y;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          s[i][c] = fmaf(kr, v[c], a * s[i][c]);
          o[j][c] = fmaf(qr, s[i][c], o[j][c]);
        }
      }
      if (j0 + j + 1 == take && p.S_T) {
#pragma unroll
        for (int i = 0; i < RPT; ++i) __builtin_nontemporal_store(s[i], out + 256 * i + (unsigned)t);
      }
    }
    if (!p.o) continue;
    // over the wave's row groups, then over the waves
#pragma unroll
    for (int j = 0; j < kTokens; ++j) {
      if (j >= m) continue;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
#pragma unroll
        for (int x = 32; x >= CG; x >>= 1) o[j][c] += __shfl_xor(o[j][c], x, 64);
      }
      if ((t & 63) < CG) *reinterpret_cast<floatx4*>(&s_o[j][wave][4 * cg]) = o[j];
    }
    __syncthreads();
    for (int x = t; x < m * DV; x += 256) {
      const int j = x / DV, c = x % DV;
      const float y = p.scale * ((s_o[j][0][c] + s_o[j][1][c]) + (s_o[j][2][c] + s_o[j][3][c]));
      const int64_t e = ((first + j0 + j) * p.H + h) * DV + c;
      if (p.out_bf16)
        static_cast<uint16_t*>(p.o)[e] = lin_bf16(y);
      else
        static_cast<float*>(p.o)[e] = y;
    }
  }
}

// One token, committed: the same in less. A row of the state goes out as soon as it is done.
template <int DK, int DV, typename T>
__global__ __launch_bounds__(256) void lin_step_kernel(const LinPlan p) {
  constexpr int CG = DV / 4, RG = 256 / CG, RPT = DK / RG;
  __shared__ float2 s_kq[DK];
  __shared__ __align__(16) float s_o[4][DV];
  const int n = blockIdx.x / p.H, h = blockIdx.x % p.H, hk = h / (p.H / p.Hk);
  const int t = threadIdx.x, cg = t % CG, rg = t / CG;
  floatx4* const S = reinterpret_cast<floatx4*>(p.S_T + (int64_t)blockIdx.x * DK * DV);
  floatx4 s[RPT];
#pragma unroll
  for (int i = 0; i < RPT; ++i) s[i] = __builtin_nontemporal_load(S + 256 * i + (unsigned)t);
  if (t < DK)
    s_kq[t] = float2{ld(reinterpret_cast<const T*>(p.k + n * p.k_token + hk * p.k_head), t),
                     ld(reinterpret_cast<const T*>(p.q + n * p.q_token + hk * p.q_head), t)};
  const T* vp = reinterpret_cast<const T*>(p.v + n * p.v_token + h * p.v_head);
  const floatx4 v{ld(vp, 4 * cg), ld(vp, 4 * cg + 1), ld(vp, 4 * cg + 2), ld(vp, 4 * cg + 3)};
  const float a = expf(lin_gate(p, n, h));
  __syncthreads();
  floatx4 o{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const float2 kq = s_kq[rg + RG * i];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      s[i][c] = fmaf(kq.x, v[c], a * s[i][c]);
      o[c] = fmaf(kq.y, s[i][c], o[c]);
    }
    __builtin_nontemporal_store(s[i], S + 256 * i + (unsigned)t);
  }
  // over the wave's row groups, then over the waves
#pragma unroll
  for (int c = 0; c < 4; ++c) {
#pragma unroll
    for (int x = 32; x >= CG; x >>= 1) o[c] += __shfl_xor(o[c], x, 64);
  }
  if ((t & 63) < CG) *reinterpret_cast<floatx4*>(&s_o[t >> 6][4 * cg]) = o;
  __syncthreads();
  if (t < DV) {
    const float y = p.scale * ((s_o[0][t] + s_o[1][t]) + (s_o[2][t] + s_o[3][t]));
    const int64_t e = (int64_t)blockIdx.x * DV + t;
    if (p.out_bf16)
      static_cast<uint16_t*>(p.o)[e] = lin_bf16(y);
    else
      static_cast<float*>(p.o)[e] = y;
  }
}

template <int DK, int DV>
hipError_t launch(const LinPlan& p, hipStream_t stream) {
  const dim3 grid(p.n_seq * p.H);
  const bool one = p.T == 1 && !p.accept && p.S_T == p.S0 && p.o;
  if (p.act_bf16) {
    if (one)
      lin_step_kernel<DK, DV, uint16_t><<<grid, 256, 0, stream>>>(p);
    else
      lin_recurrent_kernel<DK, DV, uint16_t><<<grid, 256, 0, stream>>>(p);
  } else {
    if (one)
      lin_step_kernel<DK, DV, float><<<grid, 256, 0, stream>>>(p);
    else
      lin_recurrent_kernel<DK, DV, float><<<grid, 256, 0, stream>>>(p);
  }
  return hipGetLastError();
}

template <int DK>
hipError_t launch_dk(const LinPlan& p, hipStream_t stream) {
  return p.dv == 32 ? launch<DK, 32>(p, stream) : p.dv == 64 ? launch<DK, 64>(p, stream) : launch<DK, 128>(p, stream);
}

}  // namespace

hipError_t launch_lin_recurrent(const LinPlan& p, hipStream_t stream) {
  return p.dk == 32 ? launch_dk<32>(p, stream) : p.dk == 64 ? launch_dk<64>(p, stream) : launch_dk<128>(p, stream);
}

}  // namespace kda
