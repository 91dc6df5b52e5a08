// Logits to adjusted logits or probabilities: penalties for tokens that were there, biases, a grammar's
// mask, a temperature, and the softmax.
//
// Every logit is read (twice for probabilities: once for the row's maximum and sum, once for the
// values; of a few rows the second pass reads what the first made of them) and every result written once;
// the second read comes from the caches where the batch fits them. The launches bound one row (4.9 and 3.4 us for
// 32,000 tokens). For 256 sequences of five rows of 131,072, bf16 to fp32, with everything there is, the first
// pass takes 150 us, which its instructions bound (75 where nothing is adjusted), the second 228, of
// which 181 go to reading and writing 1 GB.
//
// A workgroup takes a block of tokens of one sequence, for all of its rows or for one, and has the next
// row's logits on their way while it works on this one's. It first counts in LDS what the history holds of
// its tokens: a word per token, the number of times past the prompt in 31 bits and in the top bit
// whether it is there at all; and of the biases it keeps the last entry's number. Adding whole numbers and
// taking their maximum gives the same whatever the order, so results are the same on every run. Both make
// one word per token that a row's tokens are looked up in: what is added to the logit, +0 for most tokens, which
// nothing is done with; -0, which changes no value, for one that only the repetition factor holds for. Which
// tokens that holds for is a bit each, in a register of the thread that has the token in every row. Row j's
// drafts are the first j: a row counts the one before it.
#include <algorithm>
#include <cfloat>

#include "kda_device.h"
#include "kda_internal.h"
#include "kda_logits_plan.h"

namespace kda {

namespace {

constexpr int kThreads = kLogitsThreads, kE = kLogitsEach;
constexpr unsigned kThere = 0x80000000u;

struct Stat {   // of a wave's part of a row
  float top;    // largest value, NaN aside (-inf if there is none)
  float sum;    // of e^{x - top}; 0 if top is -inf, NaN if a value is
  int at;       // first token that has it (greedy rows only)
  int pad;
};

enum Mode { kAdjust, kStats, kProbs };

// e^{x - top} for values that are not above `top`: off by 2^-22 |x - top| relative, nothing at the top.
__device__ __forceinline__ float exp_finite(float x, float top) {
  return __builtin_amdgcn_exp2f((x - top) * kLog2e);
}
// top is +inf: infinite values share; -inf: there is nothing; NaN stays
__device__ __forceinline__ float exp_infinite(float x) { return x != x ? x : x == INFINITY ? 1.f : 0.f; }
__device__ __forceinline__ float exp_of(float x, float top) {
  return fabsf(top) < INFINITY ? exp_finite(x, top) : exp_infinite(x);
}
// kE neighbouring values as they lie in memory, whatever their alignment, and as floats.
template <typename T>
struct Raw;
template <>
struct Raw<float> {
  float x[kE];
  __device__ __forceinline__ void load(const float* p) {
    typedef float vec __attribute__((ext_vector_type(kE), aligned(4)));
    const vec y = *reinterpret_cast<const vec*>(p);
#pragma unroll
    for (int i = 0; i < kE; ++i) x[i] = y[i];
  }
  __device__ __forceinline__ void put(int i, const float* p) { x[i] = p ? *p : -INFINITY; }
  __device__ __forceinline__ float at(int i) const { return x[i]; }
};
template <>
struct Raw<uint16_t> {
  unsigned x[kE / 2];
  __device__ __forceinline__ void load(const uint16_t* p) {
    typedef unsigned vec __attribute__((ext_vector_type(kE / 2), aligned(2)));
    const vec y = *reinterpret_cast<const vec*>(p);
#pragma unroll
    for (int i = 0; i < kE / 2; ++i) x[i] = y[i];
  }
  __device__ __forceinline__ void put(int i, const uint16_t* p) {
    const unsigned y = p ? *p : 0xff80u;
    x[i / 2] = i % 2 ? (x[i / 2] & 0xffffu) | y << 16 : y;
  }
  __device__ __forceinline__ float at(int i) const {
    return __uint_as_float(i % 2 ? x[i / 2] & 0xffff0000u : x[i / 2] << 16);
  }
};
// Where the bits of m are 1 those of a, else b's. (Written with & and |, the compiler makes comparisons and up to
// six instructions of it.)
__device__ __forceinline__ float choose(unsigned m, float a, float b) {
  return __uint_as_float(__builtin_amdgcn_bitop3_b32(m, __float_as_uint(a), __float_as_uint(b), 0xca));
}
// 1 / d in two parts, the first one below it: x / d is the quotient rounded once (the parts leave 2^-45 of it), so
// that a quotient that is a 32-bit number comes out as it. (With one part 1,365 of 2,048 of them missed at d =
// 1.75.) Both parts are above 0, so infinities stay what they are.
struct Inverse {
  float part, rest;
  __device__ __forceinline__ explicit Inverse(float d) {
    part = __uint_as_float(__float_as_uint(__builtin_amdgcn_rcpf(d)) - 1);  // that instruction is off by less than a step
    rest = fmaxf(fmaf(-d, part, 1.f) * part, 0x1p-149f);
  }
  __device__ __forceinline__ float operator*(float x) const { return fmaf(x, part, x * rest); }
};
// Bit i of x in every bit.
__device__ __forceinline__ unsigned bit(unsigned x, int i) { return (unsigned)__builtin_amdgcn_sbfe((int)x, i, 1); }
__device__ __forceinline__ uint16_t to_bf16(float x) { return __builtin_bit_cast(uint16_t, static_cast<__bf16>(x)); }
__device__ __forceinline__ void store4(float* p, const float* x) {
  typedef float vec __attribute__((ext_vector_type(4), aligned(4)));
  __builtin_nontemporal_store(vec{x[0], x[1], x[2], x[3]}, reinterpret_cast<vec*>(p));
}
__device__ __forceinline__ void store4(uint16_t* p, const float* x) {
  typedef uint16_t vec __attribute__((ext_vector_type(4), aligned(2)));
  __builtin_nontemporal_store(vec{to_bf16(x[0]), to_bf16(x[1]), to_bf16(x[2]), to_bf16(x[3])},
                              reinterpret_cast<vec*>(p));
}
__device__ __forceinline__ void store1(float* p, float x) { *p = x; }
__device__ __forceinline__ void store1(uint16_t* p, float x) { *p = to_bf16(x); }

// The larger of two, of equal ones the first token.
__device__ __forceinline__ void larger(float& top, int& at, float y, int i) {
  if (y > top || (y == top && i < at)) top = y, at = i;
}
// Another lane's value on the way up to lane 63 (16 lanes in four steps, then rows of 16 in two); `none`
// where there is none.
template <int STEP>
__device__ __forceinline__ int lane_below(int none, int x) {
  constexpr int kCtrl[] = {0x111, 0x112, 0x114, 0x118, 0x142, 0x143}, kRows[] = {0xf, 0xf, 0xf, 0xf, 0xa, 0xc};
  return __builtin_amdgcn_update_dpp(none, x, kCtrl[STEP], kRows[STEP], 0xf, false);
}
template <int STEP>
__device__ __forceinline__ float lane_below(float none, float x) {
  return __builtin_bit_cast(float, lane_below<STEP>(__builtin_bit_cast(int, none), __builtin_bit_cast(int, x)));
}
// Over the wave's lanes, as scalars.
__device__ __forceinline__ float wave_max(float x) {
  x = fmaxf(x, lane_below<0>(-INFINITY, x));
  x = fmaxf(x, lane_below<1>(-INFINITY, x));
  x = fmaxf(x, lane_below<2>(-INFINITY, x));
  x = fmaxf(x, lane_below<3>(-INFINITY, x));
  x = fmaxf(x, lane_below<4>(-INFINITY, x));
  x = fmaxf(x, lane_below<5>(-INFINITY, x));
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), 63));
}
__device__ __forceinline__ float wave_sum(float x) {
  x += lane_below<0>(0.f, x);
  x += lane_below<1>(0.f, x);
  x += lane_below<2>(0.f, x);
  x += lane_below<3>(0.f, x);
  x += lane_below<4>(0.f, x);
  x += lane_below<5>(0.f, x);
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), 63));
}
__device__ __forceinline__ int wave_min(int x) {
  x = min(x, lane_below<0>(INT32_MAX, x));
  x = min(x, lane_below<1>(INT32_MAX, x));
  x = min(x, lane_below<2>(INT32_MAX, x));
  x = min(x, lane_below<3>(INT32_MAX, x));
  x = min(x, lane_below<4>(INT32_MAX, x));
  x = min(x, lane_below<5>(INT32_MAX, x));
  return __builtin_amdgcn_readlane(x, 63);
}

// Every stat of a row in one, by one wave; `mine` is the lane's first.
__device__ __forceinline__ Stat join(Stat mine, const Stat* s, int n, bool greedy) {
  const int lane = threadIdx.x & 63;
  for (int i = lane + 64; i < n; i += 64) {
    const Stat x = s[i];
    const float top = fmaxf(mine.top, x.top);
    mine.sum = mine.sum * exp_of(mine.top, top) + x.sum * exp_of(x.top, top);
    larger(mine.top, mine.at, x.top, x.at);
  }
  const float top = wave_max(mine.top);
  Stat all{top, wave_sum(mine.sum * exp_of(mine.top, top)), INT32_MAX, 0};
  if (greedy) all.at = wave_min(mine.top == top ? mine.at : INT32_MAX);
  return all;
}

// Where the first pass may leave the adjusted logits in out for the second: fp32 results of a few rows, which
// stay in the caches (with a history, one row of 32,000 tokens: 9.5 us, so 9.3; five of 131,072: 13.9, 12.6; 48 of
// 32,000: 16.0, 14.8). Large batches would pay for the bytes (16 x 5 of 131,072: 33.9, so 42.5).
template <typename O, int STEPS>
constexpr bool kKeeps = STEPS == 1 && sizeof(O) == sizeof(float);

// STEPS: times kE tokens of each thread are a block. Of large blocks the LDS takes five to a CU, and so shall the
// registers.
template <typename T, typename O, Mode MODE, int STEPS>
__global__ __launch_bounds__(kThreads, STEPS == 4 ? 5 : 1) void logits_kernel(const LogitsPlan p, int blocks, int splits) {
  constexpr int kBlock = STEPS * kThreads * kE;
  extern __shared__ __align__(16) unsigned s_mem[];
  const int t = threadIdx.x;
  const unsigned item = blockIdx.x;  // (sequence, split of its rows, block)
  const int b = item % blocks, part = item / blocks % splits, n = item / blocks / splits;
  const int j0 = splits == 1 ? 0 : part, j1 = splits == 1 ? p.R : part + 1;
  const int base = b * kBlock, here = min(kBlock, p.V - base);
  const bool said = p.history || p.drafts, biased = p.bias_ids;
  unsigned* const s_add = s_mem;              // first the biases' numbers, then what is added
  unsigned* const s_said = s_mem + kBlock;    // only if `said`
  __shared__ int s_found;
  Raw<T> next[STEPS];
  unsigned next_mask[STEPS];
  int next_draft = -1;
  // A zero that the compiler does not know to be the same in all lanes: a draft read at a scalar's address would go
  // to a scalar register, which waits for it, and for the row, where it is asked for.
  int lane_zero;
  asm("v_mov_b32 %0, 0" : "=v"(lane_zero));
  const int stats = blocks * (kThreads / 64);  // of a row: one per wave
  Stat next_stat{-INFINITY, 0.f, INT32_MAX, 0};
#pragma unroll
  for (int c = 0; c < STEPS; ++c) next_mask[c] = ~0u;
  auto fetch = [&](int j) {  // row j's block, tokens past the vocabulary as -inf
    const T* in = static_cast<const T*>(p.logits) + n * p.seq + j * p.row + base;
    const uint32_t* mask = p.mask + n * p.mask_seq + j * p.mask_row + base / 32;
    if (p.drafts && j > 0) next_draft = (p.drafts + (int64_t)n * (p.R - 1) + j - 1)[lane_zero];
    if (MODE == kProbs && (t & 63) < stats)
      next_stat = static_cast<const Stat*>(p.workspace)[((int64_t)n * p.R + j) * stats + (t & 63)];
    if (here == kBlock) {
#pragma unroll
      for (int c = 0; c < STEPS; ++c) next[c].load(in + (c * kThreads + t) * kE);
      if (p.mask) {
#pragma unroll
        for (int c = 0; c < STEPS; ++c) next_mask[c] = mask[(c * kThreads + t) * kE / 32];
      }
    } else {
#pragma unroll
      for (int c = 0; c < STEPS; ++c) {
        const int i = (c * kThreads + t) * kE;
#pragma unroll
        for (int e = 0; e < kE; ++e) next[c].put(e, i + e < here ? in + i + e : nullptr);
        if (p.mask && i < here) next_mask[c] = mask[i / 32];
      }
    }
  };
  fetch(j0);

  const float repetition = p.repetition ? p.repetition[n] : 1.f;
  const float frequency = p.frequency ? p.frequency[n] : 0.f;
  const float presence = p.presence ? p.presence[n] : 0.f;
  // an infinite one would make what is masked (and the end of the last block) a NaN
  const float heat = p.temperature ? p.temperature[n] : 1.f, temperature = heat == INFINITY ? FLT_MAX : heat;
  const bool greedy = !(temperature > 0.f);
  const bool scaled = !greedy && temperature != 1.f && !(MODE == kProbs && p.kept);
  const bool inverse = temperature > 0x1p-60f && temperature < 0x1p60f;  // its parts are far from both ends then
  const Inverse scale(temperature), once(repetition);

  unsigned repeats = 0;  // this thread's tokens that the repetition factor holds for: bit c kE + e
  // What is added to a token that is `w` in the counts and has this bias, and whether it repeats.
  auto adjust = [&](unsigned x, unsigned w, float bias, int i) {
    const unsigned times = w & ~kThere;
    const float less = times ? frequency * (float)times + presence : 0.f;
    const float add = bias - less;
    s_add[x] = add == 0.f ? 0x80000000u : __builtin_bit_cast(unsigned, add);
    // beside an infinite one the factor makes no difference; a product out of range would make it a NaN
    repeats = (repeats & ~(1u << i)) | (w && fabsf(add) < INFINITY ? 1u : 0u) << i;
  };
  if (said || biased) {
    typedef unsigned vec __attribute__((ext_vector_type(4)));
    for (int i = t; i < kBlock / 4 * (said ? 2 : 1); i += kThreads) reinterpret_cast<vec*>(s_mem)[i] = vec{0, 0, 0, 0};
    __syncthreads();
    if (p.history) {
      const int32_t* ids = p.history + n * p.history_stride;
      const int len = min(max(p.history_lens[n], 0), p.max_history);
      const int prompt = p.prompt_lens ? min(max(p.prompt_lens[n], 0), len) : 0;
      auto count = [&](int i, int id) {
        const unsigned x = (unsigned)id - (unsigned)base;
        if (x < (unsigned)here) {
          if (i < prompt) atomicOr(&s_said[x], kThere); else atomicAdd(&s_said[x], 1u);
        }
      };
      typedef int ids4 __attribute__((ext_vector_type(4), aligned(4)));
      for (int i = 4 * t; i < len; i += 4 * kThreads) {
        if (i + 4 <= len) {
          const ids4 x = *reinterpret_cast<const ids4*>(ids + i);
#pragma unroll
          for (int e = 0; e < 4; ++e) count(i + e, x[e]);
        } else {
          for (int e = i; e < len; ++e) count(e, ids[e]);
        }
      }
    }
    if (p.drafts) {  // those before this workgroup's first row
      for (int j = t; j < j0; j += kThreads) {
        const unsigned x = (unsigned)p.drafts[(int64_t)n * (p.R - 1) + j] - (unsigned)base;
        if (x < (unsigned)here) atomicAdd(&s_said[x], 1u);
      }
    }
    if (biased) {
      const int count = p.bias_counts ? min(max(p.bias_counts[n], 0), p.max_bias) : p.max_bias;
      const int32_t* ids = p.bias_ids + (int64_t)n * p.max_bias;
      for (int i = t; i < count; i += kThreads) {
        const unsigned x = (unsigned)ids[i] - (unsigned)base;
        if (x < (unsigned)here) atomicMax(&s_add[x], (unsigned)i + 1);
      }
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < STEPS; ++c) {
      const int i = (c * kThreads + t) * kE;
      const vec w = said ? *reinterpret_cast<const vec*>(&s_said[i]) : vec{0, 0, 0, 0};
      const vec b = *reinterpret_cast<const vec*>(&s_add[i]);
#pragma unroll
      for (int e = 0; e < kE; ++e)
        if (w[e] | b[e]) adjust(i + e, w[e], b[e] ? p.bias[(int64_t)n * p.max_bias + b[e] - 1] : 0.f, c * kE + e);
    }
    __syncthreads();
  }

  for (int j = j0; j < j1; ++j) {
    if (j > j0 && p.drafts) {
      const int draft = __builtin_amdgcn_readfirstlane(next_draft);
      const unsigned x = (unsigned)draft - (unsigned)base;
      if (x < (unsigned)here) {  // the same for all threads
        __syncthreads();
        if (t == 0) s_found = 0;
        __syncthreads();
        if (biased) {
          const int count = p.bias_counts ? min(max(p.bias_counts[n], 0), p.max_bias) : p.max_bias;
          for (int i = t; i < count; i += kThreads)
            if (p.bias_ids[(int64_t)n * p.max_bias + i] == draft) atomicMax(&s_found, i + 1);
        }
        __syncthreads();
        if (t == (int)(x / kE % kThreads))
          adjust(x, s_said[x] += 1, s_found ? p.bias[(int64_t)n * p.max_bias + s_found - 1] : 0.f,
                 x / kE / kThreads * kE + x % kE);
        __syncthreads();
      }
    }
    float x[STEPS][kE];
    unsigned mask[STEPS];
#pragma unroll
    for (int c = 0; c < STEPS; ++c) {
      mask[c] = next_mask[c];
      asm volatile("" : "+v"(mask[c]));  // here, not behind the next row's loads, which the copy would wait for
#pragma unroll
      for (int e = 0; e < kE; ++e) x[c][e] = next[c].at(e);
    }
    const Stat mine = next_stat;
    if (j + 1 < j1) fetch(j + 1);
    Stat row{0.f, 0.f, 0, 0};
    if (MODE == kProbs)  // the row's maximum and sum
      row = join(mine, static_cast<const Stat*>(p.workspace) + ((int64_t)n * p.R + j) * stats, stats, greedy);
#pragma unroll
    for (int c = 0; c < STEPS; ++c) {
      const int i = (c * kThreads + t) * kE;
      typedef unsigned vec __attribute__((ext_vector_type(4)));
      if (said || biased) {
        const vec w = *reinterpret_cast<const vec*>(&s_add[i]);
        if (w[0] | w[1] | w[2] | w[3]) {
#pragma unroll
          for (int e = 0; e < kE; ++e) {
            // no branches: with a history of thousands, some lane has such a token nearly every time
            const float y = x[c][e];
            const float z = choose(bit(__float_as_uint(y), 31), y * repetition, once * y);
            x[c][e] = choose(bit(repeats, c * kE + e), z, y) + __uint_as_float(w[e]);
          }
        }
      }
      if (p.mask) {
        const unsigned allowed = mask[c] >> (i % 32);
#pragma unroll
        for (int e = 0; e < kE; ++e) x[c][e] = choose(bit(allowed, e), x[c][e], -INFINITY);
      }
      if (scaled) {
        if (inverse) {
#pragma unroll
          for (int e = 0; e < kE; ++e) x[c][e] = scale * x[c][e];
        } else {
#pragma unroll
          for (int e = 0; e < kE; ++e) x[c][e] /= temperature;
        }
      }
    }
    O* out = static_cast<O*>(p.out) + n * p.out_seq + j * p.out_row + base;
    if (MODE == kStats) {
      if (kKeeps<O, STEPS> && p.kept) {
#pragma unroll
        for (int e = 0; e < kE; ++e)
          if (t * kE + e < here) store1(out + t * kE + e, x[0][e]);
      }
      Stat s{-INFINITY, 0.f, INT32_MAX, 0};
      float top = -INFINITY;
#pragma unroll
      for (int c = 0; c < STEPS; ++c)
#pragma unroll
        for (int e = 0; e < kE; ++e) top = fmaxf(top, x[c][e]);
      s.top = wave_max(top);
      if (fabsf(s.top) < INFINITY) {
#pragma unroll
        for (int c = 0; c < STEPS; ++c)
#pragma unroll
          for (int e = 0; e < kE; ++e) s.sum += exp_finite(x[c][e], s.top);
      } else {
#pragma unroll
        for (int c = 0; c < STEPS; ++c)
#pragma unroll
          for (int e = 0; e < kE; ++e) s.sum += exp_infinite(x[c][e]);
      }
      s.sum = wave_sum(s.sum);
      if (greedy) {
#pragma unroll
        for (int c = STEPS - 1; c >= 0; --c)
#pragma unroll
          for (int e = kE - 1; e >= 0; --e)
            if (x[c][e] == s.top && s.top > -INFINITY) s.at = base + (c * kThreads + t) * kE + e;
        s.at = wave_min(s.at);
      }
      if ((t & 63) == 0)
        static_cast<Stat*>(p.workspace)[((int64_t)n * p.R + j) * stats + b * (kThreads / 64) + (t >> 6)] = s;
      continue;
    }
    const float share = row.sum == 0.f ? 0.f : 1.f / row.sum;
#pragma unroll
    for (int c = 0; c < STEPS; ++c) {
      const int i = (c * kThreads + t) * kE;
      if (MODE == kProbs) {
        if (greedy) {
#pragma unroll
          for (int e = 0; e < kE; ++e) x[c][e] = base + i + e == row.at ? 1.f : 0.f;
        } else if (fabsf(row.top) < INFINITY) {
#pragma unroll
          for (int e = 0; e < kE; ++e) x[c][e] = exp_finite(x[c][e], row.top) * share;
        } else {
#pragma unroll
          for (int e = 0; e < kE; ++e) x[c][e] = exp_infinite(x[c][e]) * share;
        }
      }
      if (i + kE <= here) {
        store4(out + i, x[c]);
      } else {
#pragma unroll
        for (int e = 0; e < kE; ++e)
          if (i + e < here) store1(out + i + e, x[c][e]);
      }
    }
  }
}

template <typename T, typename O, Mode MODE, int STEPS>
hipError_t launch(const LogitsPlan& p, hipStream_t stream) {
  constexpr int kBlock = STEPS * kThreads * kE;
  const int blocks = (int)logits_blocks(p.V, STEPS), splits = logits_splits(p.N, p.R, blocks);
  const size_t lds = sizeof(unsigned) * kBlock * (p.history || p.drafts ? 2 : p.bias_ids ? 1 : 0);
  logits_kernel<T, O, MODE, STEPS>
      <<<dim3((unsigned)((int64_t)p.N * splits * blocks)), kThreads, lds, stream>>>(p, blocks, splits);
  return hipGetLastError();
}

template <typename T, typename O, int STEPS>
hipError_t launch_steps(const LogitsPlan& p, hipStream_t stream) {
  if (!p.probs) return launch<T, O, kAdjust, STEPS>(p, stream);
  if constexpr (kKeeps<O, STEPS>) {
    if (p.history || p.drafts || p.bias_ids) {
      LogitsPlan q = p;
      q.kept = true;
      const hipError_t e = launch<T, O, kStats, STEPS>(q, stream);
      if (e != hipSuccess) return e;
      q.logits = p.out, q.seq = p.out_seq, q.row = p.out_row;
      q.history = q.drafts = q.bias_ids = nullptr;
      q.mask = nullptr;
      return launch<O, O, kProbs, STEPS>(q, stream);
    }
  }
  const hipError_t e = launch<T, O, kStats, STEPS>(p, stream);
  return e == hipSuccess ? launch<T, O, kProbs, STEPS>(p, stream) : e;
}

template <typename T, typename O>
hipError_t launch_all(const LogitsPlan& p, hipStream_t stream) {
  return logits_steps(p.N, p.R, p.V) == 1 ? launch_steps<T, O, 1>(p, stream) : launch_steps<T, O, 4>(p, stream);
}

}  // namespace

size_t logits_workspace_bytes(int N, int R, int V) {
  return sizeof(Stat) * (kThreads / 64) * (size_t)N * R * logits_blocks(V, logits_steps(N, R, V));
}

hipError_t launch_logits(const LogitsPlan& p, hipStream_t stream) {
  if (p.bf16)
    return p.out_bf16 ? launch_all<uint16_t, uint16_t>(p, stream) : launch_all<uint16_t, float>(p, stream);
  return p.out_bf16 ? launch_all<float, uint16_t>(p, stream) : launch_all<float, float>(p, stream);
}

}  // namespace kda
