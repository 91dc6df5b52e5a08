// What the C ABI's entry points share: the last error, and checks of arguments. Nothing here
// touches the device.
#pragma once

#include <cstdarg>
#include <cstddef>
#include <cstdint>
#include <cstdio>
#include <string>

#include "../../include/kda.h"

namespace kda {
namespace api {

inline thread_local std::string g_last_error;

inline kda_status fail(kda_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return s;
}

inline kda_status ok() {
  g_last_error.clear();
  return KDA_OK;
}

// A launch's grid holds at most 2^32 - 1 work-items. The decode kernels run one
// 256-work-item workgroup per (sequence, head).
constexpr int64_t kMaxGridItems = 0xffffffffLL;
constexpr int64_t kMaxDecodePairs = kMaxGridItems / 256;

inline bool head_dim_ok(int d) { return d == 32 || d == 64 || d == 128; }
inline bool dtype_ok(kda_dtype t) { return t == KDA_F32 || t == KDA_BF16; }
inline size_t dsize(kda_dtype t) { return t == KDA_F32 ? 4 : 2; }

struct Range {
  const char* name;
  uintptr_t lo, hi;  // [lo, hi)
};

inline Range range(const char* name, const void* p, size_t bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return Range{name, a, a + bytes};
}

inline bool overlap(const Range& a, const Range& b) {
  return a.lo < b.hi && b.lo < a.hi && a.hi > a.lo && b.hi > b.lo;
}

constexpr int64_t kMaxStride = int64_t(1) << 40;  // bytes; keeps every address below 2^63

// A stride (elements of `es` bytes) of an array read and written 16 bytes at a time.
inline bool stride_ok(int64_t s, size_t es) {
  return s >= 0 && s <= kMaxStride / (int64_t)es && s * (int64_t)es % 16 == 0;
}
inline bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// Rows of [tokens, heads, d] by strides (elements): what they span.
inline size_t span_bytes(int64_t tokens, int64_t token_stride, int heads, int64_t head_stride, int d,
                         size_t es) {
  return tokens ? (size_t)((tokens - 1) * token_stride + (heads - 1) * head_stride + d) * es : 0;
}
inline bool span_ok(int64_t tokens, int64_t token_stride, int heads, int64_t head_stride) {
  return (double)tokens * (double)token_stride + (double)heads * (double)head_stride < 0x1p58;
}

}  // namespace api
}  // namespace kda
