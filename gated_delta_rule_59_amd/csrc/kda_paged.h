// Device helpers of the kernels that touch a paged cache.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kda_internal.h"

namespace kda {

constexpr int kF32 = 0, kBF16 = 1, kF8 = 2;  // kda_dtype

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// token / page_size, for 0 <= token < 2^31
__device__ __forceinline__ int div_page(const PageCache& c, unsigned token) {
  return (int)(((uint64_t)token * c.ps_mul) >> c.ps_shift);
}

// Two values rounded to bf16 (nearest even, NaN kept), the first in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const bf16x2 v = {static_cast<__bf16>(lo), static_cast<__bf16>(hi)};
  return __builtin_bit_cast(uint32_t, v);
}

}  // namespace kda
