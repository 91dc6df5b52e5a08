// Linear attention with a decay for each head, token by token:
//
//     S <- e^{g_t} S + k_t v_t^T;   o_t = scale S_t^T q_t
//
// for the new token or the drafts of each sequence. The state is read once and written once, 4 dk dv
// bytes each way per (sequence, head), beside which a token's own rows are nothing: HBM bounds it.
//
// One 256-thread workgroup per (n, h). Thread t owns value columns 4 (t % CG) .. + 3 (CG = DV / 4) and
// key rows t / CG + RG i (RG = 256 / CG), so a wave reads whole rows in 1 KiB pieces and the state
// stays in registers between the read and the write. Tokens come four at a time through LDS; their
// results are summed over the row groups there.
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
  __shared__ float s_q[kTokens][DK], s_k[kTokens][DK], s_v[kTokens][DV], s_a[kTokens];
  __shared__ float s_o[kTokens][4][DV];

  const int n = blockIdx.x / p.H, h = blockIdx.x % p.H, hk = h / (p.H / p.Hk);
  const int t = threadIdx.x, cg = t % CG, rg = t / CG, wave = t >> 6;
  int64_t first;
  int len;
  lin_tokens(p, n, &first, &len);
  const int take = p.accept ? min(max(p.accept[n], 0), len) : len;

  const int64_t at = (int64_t)blockIdx.x * DK * DV;
  floatx4 s[RPT];
  const floatx4* in = reinterpret_cast<const floatx4*>(p.S0 + at);
#pragma unroll
  for (int i = 0; i < RPT; ++i)
    s[i] = p.S0 ? __builtin_nontemporal_load(&in[(rg + RG * i) * CG + cg]) : floatx4{0.f, 0.f, 0.f, 0.f};
  floatx4* out = reinterpret_cast<floatx4*>(p.S_T + at);
  // in place nothing changes where no token is taken
  if (take == 0 && p.S_T && p.S_T != p.S0) {
#pragma unroll
    for (int i = 0; i < RPT; ++i) __builtin_nontemporal_store(s[i], &out[(rg + RG * i) * CG + cg]);
  }

  for (int j0 = 0; j0 < len; j0 += kTokens) {
    const int m = min(kTokens, len - j0);
    if (j0) __syncthreads();
    for (int x = t; x < m * (2 * DK + DV); x += 256) {
      const int j = x / (2 * DK + DV), c = x % (2 * DK + DV);
      const int64_t tok = first + j0 + j;
      if (c < DK) {
        s_q[j][c] = ld(reinterpret_cast<const T*>(p.q + tok * p.q_token + hk * p.q_head), c);
      } else if (c < 2 * DK) {
        s_k[j][c - DK] = ld(reinterpret_cast<const T*>(p.k + tok * p.k_token + hk * p.k_head), c - DK);
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
        const float kr = s_k[j][rg + RG * i], qr = s_q[j][rg + RG * i];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          s[i][c] = fmaf(kr, v[c], a * s[i][c]);
          o[j][c] = fmaf(qr, s[i][c], o[j][c]);
        }
      }
      if (j0 + j + 1 == take && p.S_T) {
#pragma unroll
        for (int i = 0; i < RPT; ++i) __builtin_nontemporal_store(s[i], &out[(rg + RG * i) * CG + cg]);
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

template <int DK, int DV>
hipError_t launch(const LinPlan& p, hipStream_t stream) {
  const dim3 grid(p.n_seq * p.H);
  if (p.act_bf16)
    lin_recurrent_kernel<DK, DV, uint16_t><<<grid, 256, 0, stream>>>(p);
  else
    lin_recurrent_kernel<DK, DV, float><<<grid, 256, 0, stream>>>(p);
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
