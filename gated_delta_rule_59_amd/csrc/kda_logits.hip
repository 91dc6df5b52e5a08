// Logits to adjusted logits or probabilities: penalties for tokens that were there, biases, a grammar's
// mask, a temperature, and the softmax.
//
// Every logit is read (twice for probabilities: once for the row's maximum and sum, once for the
// values) and every result written once; the second read comes from the caches where the batch fits
// them. HBM bounds a batch, the launches one row.
//
// A workgroup takes a block of kBlock tokens of one sequence, for all of its rows or for one. It first
// writes down in LDS what the history holds of its tokens: a word per token, the number of times past
// the prompt in 31 bits and in the top bit whether it is there at all; and of the biases the last
// entry's number. Adding whole numbers and taking their maximum gives the same whatever the order, so
// results are the same on every run. Row j's drafts are the first j: a row adds the one before it.
#include <algorithm>

#include "kda_device.h"
#include "kda_internal.h"

namespace kda {

namespace {

constexpr int kThreads = 256, kE = 4, kBlock = 4096, kSteps = kBlock / (kThreads * kE);
constexpr unsigned kThere = 0x80000000u;

struct Stat {   // of a block of a row
  float top;    // largest value, NaN aside (-inf if there is none)
  float sum;    // of e^{x - top}; 0 if top is -inf, NaN if a value is
  int at;       // first token that has it
  int pad;
};

enum Mode { kAdjust, kStats, kProbs };

// e^x for x <= 0 (below 2^-126: 0): the product with log2 e in two parts, so that its rounding stays
// out of the exponent. (Far below, the first part would be infinite.)
__device__ __forceinline__ float exp_of(float x) {
  x = x < -150.f ? -150.f : x;
  const float hi = x * kLog2e;
  const float lo = fmaf(x, kLog2e, -hi) + x * 1.9259629911e-8f;
  const float y = __builtin_amdgcn_exp2f(hi);
  return fmaf(y, lo * 0.6931471805599453f, y);
}
// e^{x - top}, with infinite ones alike.
__device__ __forceinline__ float exp_from(float x, float top) {
  return x == top ? 1.f : top == INFINITY ? (x == x ? 0.f : x) : x == -INFINITY ? 0.f : exp_of(x - top);
}

// kE neighbouring values, whatever their alignment.
__device__ __forceinline__ void load4(const float* p, float* x) {
  typedef float vec __attribute__((ext_vector_type(4), aligned(4)));
  const vec y = *reinterpret_cast<const vec*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = y[i];
}
__device__ __forceinline__ void load4(const uint16_t* p, float* x) {
  typedef uint16_t vec __attribute__((ext_vector_type(4), aligned(2)));
  const vec y = *reinterpret_cast<const vec*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = bf16_bits_to_f32(y[i]);
}
__device__ __forceinline__ uint16_t to_bf16(float x) { return __builtin_bit_cast(uint16_t, static_cast<__bf16>(x)); }
__device__ __forceinline__ void store4(float* p, const float* x) {
  typedef float vec __attribute__((ext_vector_type(4), aligned(4)));
  *reinterpret_cast<vec*>(p) = vec{x[0], x[1], x[2], x[3]};
}
__device__ __forceinline__ void store4(uint16_t* p, const float* x) {
  typedef uint16_t vec __attribute__((ext_vector_type(4), aligned(2)));
  *reinterpret_cast<vec*>(p) = vec{to_bf16(x[0]), to_bf16(x[1]), to_bf16(x[2]), to_bf16(x[3])};
}
__device__ __forceinline__ void store1(float* p, float x) { *p = x; }
__device__ __forceinline__ void store1(uint16_t* p, float x) { *p = to_bf16(x); }

struct Row {  // what holds for all tokens of a sequence
  float repetition, frequency, presence, temperature;
  bool scaled, greedy;
};

// Two stats of the same row; equal maxima: the first token.
__device__ __forceinline__ void join(Stat& a, float top, float sum, int at) {
  if (top > a.top || (top == a.top && at < a.at)) a.at = at;
  const float m = fmaxf(a.top, top);
  a.sum = (a.sum == 0.f ? 0.f : a.sum * exp_from(a.top, m)) + (sum == 0.f ? 0.f : sum * exp_from(top, m));
  a.top = m;
}
__device__ __forceinline__ void join_lanes(Stat& s) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1)
    join(s, __shfl_xor(s.top, d, 64), __shfl_xor(s.sum, d, 64), __shfl_xor(s.at, d, 64));
}

template <typename T, typename O, Mode MODE>
__global__ __launch_bounds__(kThreads) void logits_kernel(const LogitsPlan p, int blocks, int splits) {
  extern __shared__ unsigned s_mem[];
  __shared__ Stat s_stat[kThreads / 64];
  const int t = threadIdx.x;
  const unsigned item = blockIdx.x;  // (sequence, split of its rows, block)
  const int b = item % blocks, part = item / blocks % splits, n = item / blocks / splits;
  const int j0 = splits == 1 ? 0 : part, j1 = splits == 1 ? p.R : part + 1;
  const int base = b * kBlock, here = min(kBlock, p.V - base);
  const bool said = p.history || p.drafts, biased = p.bias_ids;
  unsigned* const s_said = s_mem;
  unsigned* const s_bias = s_mem + (said ? kBlock : 0);

  Row row;
  row.repetition = p.repetition ? p.repetition[n] : 1.f;
  row.frequency = p.frequency ? p.frequency[n] : 0.f;
  row.presence = p.presence ? p.presence[n] : 0.f;
  row.temperature = p.temperature ? p.temperature[n] : 1.f;
  row.greedy = !(row.temperature > 0.f);
  row.scaled = p.temperature && !row.greedy;

  if (said || biased) {
    for (int i = t; i < kBlock * ((said ? 1 : 0) + (biased ? 1 : 0)); i += kThreads) s_mem[i] = 0;
    __syncthreads();
    if (p.history) {
      const int32_t* ids = p.history + n * p.history_stride;
      const int len = min(max(p.history_lens[n], 0), p.max_history);
      const int prompt = p.prompt_lens ? min(max(p.prompt_lens[n], 0), len) : 0;
      for (int i = t; i < len; i += kThreads) {
        const unsigned x = (unsigned)ids[i] - (unsigned)base;
        if (x < (unsigned)here) {
          if (i < prompt) atomicOr(&s_said[x], kThere); else atomicAdd(&s_said[x], 1u);
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
        if (x < (unsigned)here) atomicMax(&s_bias[x], (unsigned)i + 1);
      }
    }
    __syncthreads();
  }

  for (int j = j0; j < j1; ++j) {
    if (j > j0 && p.drafts) {
      const unsigned x = (unsigned)p.drafts[(int64_t)n * (p.R - 1) + j - 1] - (unsigned)base;
      if (x < (unsigned)here) {  // the same for all threads
        __syncthreads();
        if (t == 0) s_said[x] += 1;
        __syncthreads();
      }
    }
    const T* in = static_cast<const T*>(p.logits) + n * p.seq + j * p.row + base;
    const uint32_t* mask = p.mask ? p.mask + n * p.mask_seq + j * p.mask_row + base / 32 : nullptr;
    Stat whole{-INFINITY, 0.f, INT32_MAX, 0};
    float scale = 0.f;
    if (MODE == kProbs) {  // the row's maximum and sum out of its blocks'
      const Stat* of = static_cast<const Stat*>(p.workspace) + ((int64_t)n * p.R + j) * blocks;
      for (int i = t & 63; i < blocks; i += 64) {
        const Stat x = of[i];
        join(whole, x.top, x.sum, x.at);
      }
      join_lanes(whole);
      scale = 1.f / whole.sum;
    }
    float x[kSteps][kE];
#pragma unroll
    for (int c = 0; c < kSteps; ++c) {
      const int i = (c * kThreads + t) * kE;
      if (i + kE <= here) {
        load4(in + i, x[c]);
      } else {
#pragma unroll
        for (int e = 0; e < kE; ++e) x[c][e] = i + e < here ? ld(in, i + e) : -INFINITY;
      }
    }
#pragma unroll
    for (int c = 0; c < kSteps; ++c) {
      const int i = (c * kThreads + t) * kE;
      const unsigned allowed = mask && i < here ? mask[i / 32] >> (i % 32) : ~0u;
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        float y = x[c][e];
        if (said) {
          const unsigned w = s_said[i + e];
          if (w) y = y > 0.f ? y / row.repetition : y * row.repetition;
          // each operation rounded by itself
          if (w & ~kThere)
            y = __fsub_rn(y, __fadd_rn(__fmul_rn(row.frequency, (float)(w & ~kThere)), row.presence));
        }
        if (biased) {
          const unsigned w = s_bias[i + e];
          if (w) y = __fadd_rn(y, p.bias[(int64_t)n * p.max_bias + w - 1]);
        }
        if (!(allowed >> e & 1)) y = -INFINITY;
        if (row.scaled) y = y / row.temperature;
        if (i + e >= here) y = -INFINITY;
        x[c][e] = y;
      }
    }
    if (MODE == kStats) {
      Stat s{-INFINITY, 0.f, INT32_MAX, 0};
#pragma unroll
      for (int c = 0; c < kSteps; ++c)
#pragma unroll
        for (int e = 0; e < kE; ++e) {
          if (x[c][e] > s.top) s.top = x[c][e], s.at = base + (c * kThreads + t) * kE + e;
        }
#pragma unroll
      for (int c = 0; c < kSteps; ++c)
#pragma unroll
        for (int e = 0; e < kE; ++e) s.sum += x[c][e] == -INFINITY ? 0.f : exp_from(x[c][e], s.top);
      join_lanes(s);
      if ((t & 63) == 0) s_stat[t >> 6] = s;
      __syncthreads();
      if (t == 0) {
#pragma unroll
        for (int w = 1; w < kThreads / 64; ++w) join(s, s_stat[w].top, s_stat[w].sum, s_stat[w].at);
        static_cast<Stat*>(p.workspace)[((int64_t)n * p.R + j) * blocks + b] = s;
      }
      __syncthreads();
      continue;
    }
    O* out = static_cast<O*>(p.out) + n * p.out_seq + j * p.out_row + base;
#pragma unroll
    for (int c = 0; c < kSteps; ++c) {
      const int i = (c * kThreads + t) * kE;
      if (MODE == kProbs) {
#pragma unroll
        for (int e = 0; e < kE; ++e) {
          const float y = x[c][e];
          if (row.greedy)
            x[c][e] = base + i + e == whole.at ? 1.f : 0.f;
          else
            x[c][e] = whole.sum == 0.f ? 0.f : (y == -INFINITY ? 0.f : exp_from(y, whole.top)) * scale;
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

template <typename T, typename O, Mode MODE>
hipError_t launch(const LogitsPlan& p, hipStream_t stream) {
  const int blocks = (p.V + kBlock - 1) / kBlock;
  // one row of a sequence to a workgroup while all rows' blocks fit the card's places at once
  const int splits = (int64_t)p.N * p.R * blocks <= 2048 ? p.R : 1;
  const size_t lds = sizeof(unsigned) * kBlock * ((p.history || p.drafts ? 1 : 0) + (p.bias_ids ? 1 : 0));
  logits_kernel<T, O, MODE><<<dim3((unsigned)((int64_t)p.N * splits * blocks)), kThreads, lds, stream>>>(p, blocks, splits);
  return hipGetLastError();
}

template <typename T, typename O>
hipError_t launch_all(const LogitsPlan& p, hipStream_t stream) {
  if (!p.probs) return launch<T, O, kAdjust>(p, stream);
  const hipError_t e = launch<T, O, kStats>(p, stream);
  return e == hipSuccess ? launch<T, O, kProbs>(p, stream) : e;
}

}  // namespace

size_t logits_workspace_bytes(int N, int R, int V) {
  return sizeof(Stat) * (size_t)N * R * ((V + kBlock - 1) / kBlock);
}

hipError_t launch_logits(const LogitsPlan& p, hipStream_t stream) {
  if (p.bf16)
    return p.out_bf16 ? launch_all<uint16_t, uint16_t>(p, stream) : launch_all<uint16_t, float>(p, stream);
  return p.out_bf16 ? launch_all<float, uint16_t>(p, stream) : launch_all<float, float>(p, stream);
}

}  // namespace kda
