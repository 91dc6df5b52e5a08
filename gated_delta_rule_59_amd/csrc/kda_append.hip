// New keys and values into a paged cache, rotated by position on the way, queries alongside.
//
// A token at position p (start[n] + its index among the new ones) turns channel pair i < rot/2
// by the angle p f_i:  x' = x cos - y sin,  y' = y cos + x sin. Everything is read once and
// written once, so HBM bounds the call; the angles are formed once per token and shared by all
// heads of q and k through LDS.
//
// Angles: p f_i is formed in 64 bits (31 + 24 bits, rounded at 53) and is reduced there to a
// quarter turn, so the 32-bit sine and cosine see |angle| <= pi/4 whatever the position. (In 32
// bits a position of 10^5 would leave an angle off by 10^-2.)
//
// One 256-thread workgroup per token. Work item: two 16-byte chunks of one head that belong
// together (both partners of 8 pairs, or 16 neighbouring channels), so no pair is split
// between threads and q_out may be q itself.
#include "kda_device.h"
#include "kda_internal.h"
#include "kda_paged.h"

namespace kda {

namespace {

// sine and cosine of 2 pi * turns
__device__ __forceinline__ void sincos_turns(double turns, float& s, float& c) {
  const double quarters = 4.0 * turns;
  const double k = rint(quarters);
  float s0, c0;
  sincospif(0.5f * static_cast<float>(quarters - k), &s0, &c0);
  const int quad = static_cast<int>(static_cast<int64_t>(k)) & 3;
  const float a = quad & 1 ? c0 : s0, b = quad & 1 ? s0 : c0;
  s = quad & 2 ? -a : a;
  c = quad == 1 || quad == 2 ? -b : b;
}

// One chunk of E activations (16 bytes) as floats, and back.
template <typename T>
struct Chunk;
template <>
struct Chunk<uint16_t> {
  static constexpr int E = 8;
  static __device__ __forceinline__ void load(const char* p, float* x) {
    const u32x4 w = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
template <>
struct Chunk<float> {
  static constexpr int E = 4;
  static __device__ __forceinline__ void load(const char* p, float* x) {
    const floatx4 w = *reinterpret_cast<const floatx4*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = w[i];
  }
};

// E values as type CACHE (a kda_dtype), rounded to nearest even; streamed (65,536 prompt tokens,
// 1.6 GB read and written: 269 us, 282 with ordinary stores).
template <int CACHE, int E>
__device__ __forceinline__ void store_chunk(char* p, const float* x, float scale) {
  if constexpr (CACHE == kF32) {
    __builtin_nontemporal_store(floatx4{x[0], x[1], x[2], x[3]}, reinterpret_cast<floatx4*>(p));
  } else if constexpr (CACHE == kBF16) {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
    __builtin_nontemporal_store(w, reinterpret_cast<u32x4*>(p));
  } else {
    float y[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
      y[i] = x[i] / scale;  // not times 1 / scale: 175 / 7 is a tie, 175 * (1 / 7) lies above it
      y[i] = y[i] > 448.f ? 448.f : y[i];  // NaN passes both comparisons
      y[i] = y[i] < -448.f ? -448.f : y[i];
    }
    u32x2 w;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      int v = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * i], y[4 * i + 1], 0, false);
      w[i] = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * i + 2], y[4 * i + 3], v, true);
    }
    __builtin_nontemporal_store(w, reinterpret_cast<u32x2*>(p));
  }
}

template <typename TA, int CACHE, int D>
__global__ __launch_bounds__(256) void kv_append_kernel(const KvAppendPlan p) {
  using C = Chunk<TA>;
  constexpr int E = C::E;
  constexpr int ITEMS = D / (2 * E);  // per head
  constexpr int SA = sizeof(TA);
  constexpr int SC = CACHE == kF32 ? 4 : CACHE == kBF16 ? 2 : 1;
  __shared__ float s_cos[D / 2], s_sin[D / 2];

  const int64_t tok = blockIdx.x;
  const int t = threadIdx.x;
  int n;
  int64_t j;
  if (p.cu_seqlens) {
    // sequences that end at or before this token
    int before = 0;
    for (int i = 0; i < p.n_seq; i += 256)
      before += __syncthreads_count(i + t < p.n_seq && p.cu_seqlens[i + t + 1] <= tok);
    n = before;
    if (n >= p.n_seq) return;  // behind the last sequence
    j = tok - p.cu_seqlens[n];
  } else {
    n = (int)(tok / p.T);
    j = tok - (int64_t)n * p.T;
  }
  const int64_t pos = p.start[n] + j;

  if (t < p.rot / 2) {
    const double turns = (double)pos * (double)p.inv_freq[t] * 0.15915494309189535;  // 1 / 2 pi
    sincos_turns(turns, s_sin[t], s_cos[t]);
  }
  // the token's slot
  int page = -1;
  int64_t slot = 0;
  if (pos >= 0 && pos < (int64_t)p.c.max_pages * p.c.page_size && pos <= 0x7fffffff) {
    const int pi = div_page(p.c, (unsigned)pos);
    slot = pos - (int64_t)pi * p.c.page_size;
    page = p.c.table[n * p.c.table_stride + pi];
    if (page >= p.c.num_pages) page = -1;
  }
  __syncthreads();

  const int heads = p.Hq + 2 * p.Hkv;
  for (int it = t + (p.q ? 0 : p.Hq * ITEMS); it < heads * ITEMS; it += 256) {
    const int head = it / ITEMS, sub = it % ITEMS;
    const bool is_q = head < p.Hq, is_v = head >= p.Hq + p.Hkv;
    if (!is_q && page < 0) continue;
    const int h = is_q ? head : is_v ? head - p.Hq - p.Hkv : head - p.Hq;
    const bool turn = !is_v && sub < p.rot / (2 * E);
    const int a = turn && !p.pairs ? sub * E : 2 * sub * E;
    const int b = turn && !p.pairs ? sub * E + p.rot / 2 : a + E;
    const char* src = is_q ? p.q + tok * p.q_token + h * p.q_head
                    : is_v ? p.v + tok * p.v_token + h * p.v_head
                           : p.k + tok * p.k_token + h * p.k_head;
    float x[2 * E];
    C::load(src + a * SA, x);
    C::load(src + b * SA, x + E);
    if (turn) {
      auto turn_pair = [&](int i, float& xu, float& xw) {
        const float cs = s_cos[sub * E + i], sn = s_sin[sub * E + i], u = xu, w = xw;
        xu = u * cs - w * sn;
        xw = w * cs + u * sn;
      };
      if (p.pairs) {
#pragma unroll
        for (int i = 0; i < E; ++i) turn_pair(i, x[2 * i], x[2 * i + 1]);
      } else {
#pragma unroll
        for (int i = 0; i < E; ++i) turn_pair(i, x[i], x[E + i]);
      }
    }
    if (is_q) {
      char* dst = p.q_out + ((tok * p.Hq + h) * D) * SA;
      store_chunk<SA == 4 ? kF32 : kBF16, E>(dst + a * SA, x, 1.f);
      store_chunk<SA == 4 ? kF32 : kBF16, E>(dst + b * SA, x + E, 1.f);
    } else {
      const float* sc = is_v ? p.c.v_scale : p.c.k_scale;
      const float scale = CACHE == kF8 && sc ? sc[h] : 1.f;
      char* dst = is_v ? p.c.v + page * p.c.v_page + slot * p.c.v_token + h * p.c.v_head
                       : p.c.k + page * p.c.k_page + slot * p.c.k_token + h * p.c.k_head;
      store_chunk<CACHE, E>(dst + a * SC, x, scale);
      store_chunk<CACHE, E>(dst + b * SC, x + E, scale);
    }
  }
}

template <typename TA, int CACHE>
hipError_t launch_d(const KvAppendPlan& p, hipStream_t stream) {
  const dim3 grid((unsigned)((int64_t)p.B * p.T));
  if (p.d == 128)
    hipLaunchKernelGGL((kv_append_kernel<TA, CACHE, 128>), grid, dim3(256), 0, stream, p);
  else if (p.d == 64)
    hipLaunchKernelGGL((kv_append_kernel<TA, CACHE, 64>), grid, dim3(256), 0, stream, p);
  else
    hipLaunchKernelGGL((kv_append_kernel<TA, CACHE, 32>), grid, dim3(256), 0, stream, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_append(const KvAppendPlan& p, hipStream_t stream) {
  if ((int64_t)p.B * p.T == 0) return hipSuccess;
  if (!p.act_bf16) return launch_d<float, kF32>(p, stream);
  return p.cache_type == kF8 ? launch_d<uint16_t, kF8>(p, stream)
                             : launch_d<uint16_t, kBF16>(p, stream);
}

}  // namespace kda
