// Device helpers of linear attention with a decay for each head.
#pragma once

#include "kda_device.h"
#include "kda_internal.h"

namespace kda {

// Sequence n's tokens: the first one's row and their number.
__device__ __forceinline__ void lin_tokens(const LinPlan& p, int n, int64_t* first, int* len) {
  if (p.cu_seqlens) {
    const int a = min(max(p.cu_seqlens[n], 0), p.T), b = min(max(p.cu_seqlens[n + 1], 0), p.T);
    *first = a;
    *len = max(b - a, 0);
  } else {
    *first = (int64_t)n * p.T;
    *len = p.T;
  }
}

// Token row `tok`'s logarithm of the decay at head h.
__device__ __forceinline__ float lin_gate(const LinPlan& p, int64_t tok, int h) {
  const int64_t i = p.fixed ? h : tok * p.H + h;
  return p.gate_bf16 ? ld(static_cast<const uint16_t*>(p.g), i) : ld(static_cast<const float*>(p.g), i);
}

// Round to nearest even; infinities stay, NaN stays NaN.
__device__ __forceinline__ uint16_t lin_bf16(float x) {
  return __builtin_bit_cast(uint16_t, static_cast<__bf16>(x));
}

}  // namespace kda
