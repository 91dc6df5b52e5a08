// What the prompt kernels of linear attention with a decay for each head share: which workgroup walks
// what, the decays' sums, and the states that enter the segments.
#pragma once

#include "kda_lin.h"

namespace kda {

namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));

// What a workgroup walks: segment s of `segments` of sequence n, head h.
struct Job {
  int n, s, segments, h;
  int slot;        // its state's place in the workspace, where its sequence has several segments
  int64_t first;   // the sequence's first row
  int len;         // its tokens
};
__device__ __forceinline__ int segments_of(const LinPlan& p, int len) { return len ? (len - 1) / p.seg + 1 : 1; }

// Sums over the lanes up to each.
__device__ __forceinline__ int sums_to(int x) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int y = __shfl_up(x, d, 64);
    if ((int)(threadIdx.x & 63) >= d) x += y;
  }
  return x;
}

// Only sequences of several segments have states in the workspace, a slot for each segment; offsets that do not
// overlap give at most 2 (T / seg) of them.
//
// In the workspace behind the states and their decays, for more than 64 packed sequences: the slots of
// the sequences before each, and of each segment its sequence and its number there (-1: there is none).
// (A walk over the offsets in every workgroup, which 64 sequences take, would take longer than the work
// for thousands.)
__device__ __forceinline__ int* starts_of(const LinPlan& p) {
  return reinterpret_cast<int*>(static_cast<char*>(p.workspace) + p.tables);
}
__device__ __forceinline__ int2* jobs_of(const LinPlan& p) {
  return reinterpret_cast<int2*>(starts_of(p) + (p.n_seq + 1) / 2 * 2);
}
__global__ __launch_bounds__(1024) void lin_jobs_kernel(const LinPlan p) {
  __shared__ int s_sum[16], s_slots[16];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  int64_t done = 0, slots = 0;
  for (int n0 = 0; n0 < p.n_seq; n0 += 1024) {
    const int n = n0 + t;
    int64_t first;
    int len = 0, x = 0;
    if (n < p.n_seq) {
      lin_tokens(p, n, &first, &len);
      x = segments_of(p, len);
    }
    const int several = x > 1 ? x : 0, to = sums_to(x), slots_to = sums_to(several);
    if (lane == 63) s_sum[wave] = to, s_slots[wave] = slots_to;
    __syncthreads();
    int64_t at = done + to - x, slot = slots + slots_to - several;
    for (int w = 0; w < 16; ++w) {
      if (w < wave) at += s_sum[w], slot += s_slots[w];
      done += s_sum[w], slots += s_slots[w];
    }
    __syncthreads();
    // offsets that overlap give more
    if (n < p.n_seq) starts_of(p)[n] = (int)min(slot, (int64_t)p.slots);
    for (int s = 0; s < x && at + s < p.jobs; ++s) jobs_of(p)[at + s] = int2{n, s};
  }
  for (int64_t i = done + t; i < p.jobs; i += 1024) jobs_of(p)[i] = int2{-1, 0};
}

// Workgroup b's: false if there is none.
//
// Workgroups b and b + 256 share a CU, where the earlier goes first. Up to 64 packed sequences are taken
// by length: whole segments, then the sequences' last ones from long to short, and where no more than
// 512 workgroups have work, the second half backwards, so that long ones share with short ones (512 pairs of
// 994 .. 15,902 tokens: with the second half forwards 1.60 ms, so 1.46 ms). Where heads share
// queries and keys, an XCD (b mod 8) takes neighbouring ones of a dense batch.
__device__ __forceinline__ bool lin_job(const LinPlan& p, unsigned b, Job* j) {
  if (!p.cu_seqlens) {
    const unsigned all = gridDim.x;
    if (p.H != p.Hk && all % 8 == 0) b = b % 8 * (all / 8) + b / 8;
    j->segments = segments_of(p, p.T);
    j->slot = b / p.H;
    j->h = b % p.H;
    j->n = j->slot / j->segments;
    j->s = j->slot % j->segments;
    lin_tokens(p, j->n, &j->first, &j->len);
    return true;
  }
  const int lane = threadIdx.x & 63;
  if (p.n_seq <= 64) {
    int64_t first;
    int len = 0, x = 0;
    if (lane < p.n_seq) {
      lin_tokens(p, lane, &first, &len);
      x = segments_of(p, len);
    }
    // segments and slots of the sequences up to each: whole segments, and one more of each sequence, or of each
    // that has several. Offsets that overlap give more than there is room for: from the first sequence that
    // finds none on, nothing is done.
    const int whole = sums_to(max(x - 1, 0)), to = whole + lane + 1;
    const uint64_t several = __ballot(x > 1);
    const int slots = whole + __popcll(several & (~0ull >> (63 - lane)));
    const int n_seq = __popcll(__ballot(lane < p.n_seq && to <= p.jobs && slots <= p.slots));
    if (n_seq == 0) return false;
    const int wholes = __shfl(whole, n_seq - 1, 64);
    const unsigned all = (unsigned)min((int64_t)(wholes + n_seq) * p.H, (int64_t)gridDim.x);
    if (b >= all) return false;
    const unsigned place = b < 256 || all > 512 ? b : all - 1 - (b - 256);
    const int k = place / p.H;
    const int rest = lane < n_seq ? len - (x - 1) * p.seg : -1;
    int above = 0;
    for (int m = 0; m < n_seq; ++m) {
      const int y = __shfl(rest, m, 64);
      above += y > rest || (y == rest && m < lane);
    }
    const uint64_t which = k < wholes ? __ballot(whole > k) : __ballot(lane < n_seq && above == k - wholes);
    if (!which) return false;
    const int l = __builtin_ctzll(which);
    j->n = l;
    j->segments = __shfl(x, l, 64);
    j->s = k < wholes ? k - (__shfl(whole, l, 64) - (j->segments - 1)) : j->segments - 1;
    j->slot = __shfl(slots, l, 64) - j->segments + j->s;
    j->h = place % p.H;
    lin_tokens(p, l, &j->first, &j->len);
    return true;
  }
  const int2 which = jobs_of(p)[b / p.H];
  if (which.x < 0) return false;
  j->n = which.x;
  j->s = which.y;
  j->h = b % p.H;
  lin_tokens(p, j->n, &j->first, &j->len);
  j->segments = segments_of(p, j->len);
  j->slot = j->segments > 1 ? starts_of(p)[j->n] + j->s : 0;
  return j->segments == 1 || j->slot < p.slots;
}

// A barrier that orders the LDS only: rows of the next chunk stay on their way across it, and so do
// results. (__syncthreads, which waits for both, takes as long where a chunk's work covers them: 16 prompts of 994 ..
// 15,902 tokens 1.45 ms with either.)
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// Sums over the lanes up to each.
template <int CTRL, int ROWS>
__device__ __forceinline__ double plus_lane(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, ROWS, 0xf, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, ROWS, 0xf, false);
  return x + __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double lane_of(double x, int lane) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)u, lane);
  const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), lane);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double wave_sums(double x) {
  x = plus_lane<0x111, 0xf>(x);  // row_shr: 1, 2, 4, 8: within 16 lanes
  x = plus_lane<0x112, 0xf>(x);
  x = plus_lane<0x114, 0xf>(x);
  x = plus_lane<0x118, 0xf>(x);
  x = plus_lane<0x142, 0xa>(x);  // row_bcast: lane 15 to the next row, lane 31 to the upper half
  return plus_lane<0x143, 0xc>(x);
}

__device__ __forceinline__ void store4(float* p, const floatx4& x) { *reinterpret_cast<floatx4*>(p) = x; }
__device__ __forceinline__ void store4(uint16_t* p, const floatx4& x) {
  s16x4 y;
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] = (short)lin_bf16(x[i]);
  *reinterpret_cast<s16x4*>(p) = y;
}

// 2^(x + rest), rest next to nothing. Rounding the exponent to 32 bits alone would leave a decay of 2^-30 off by 2^-20.5.
__device__ __forceinline__ float exp2_of(float x, float rest) {
  return __builtin_amdgcn_exp2f(x) * fmaf(rest, 0.693147181f, 1.f);
}
// A sum of logarithms in two parts.
struct Log {
  float hi, lo;
  __device__ __forceinline__ explicit Log(double x) : hi((float)x), lo((float)(x - (double)hi)) {}
};
__device__ __forceinline__ float exp2_of(double x) {
  const Log y(x);
  return exp2_of(y.hi, y.lo);
}
__device__ __forceinline__ float lane_of(float x, int lane) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), lane));
}
// 2^((hi + lo) - (jhi + jlo)). What the difference of the first parts is rounded by is had back (exactly where |hi| is
// not below |jhi|, as for sums of decays up to a token and up to one before it).
__device__ __forceinline__ float exp2_between(float hi, float lo, float jhi, float jlo) {
  const float x = hi - jhi;
  return exp2_of(x, ((hi - x) - jhi) + (lo - jlo));
}

// A state in the workspace: [wave][key tile][value tile][lane] of four key rows each.
template <typename Sh>
__device__ __forceinline__ int64_t slot_of(const LinPlan& p, int64_t slot, int h) {
  return (slot * p.H + h) * (Sh::kState / 4);
}
__device__ __forceinline__ float* decays_of(const LinPlan& p) {
  return static_cast<float*>(p.workspace) + (int64_t)p.slots * p.H * p.dk * p.dv;
}

// From the sums of a sequence's segments to the states that enter them, in the sums' place. A thread
// takes four key rows of a value channel through all segments, kAhead of them on their way at a time.
template <typename Sh>
__global__ __launch_bounds__(256) void lin_entries_kernel(const LinPlan p) {
  constexpr int CT = Sh::kTiles, KT = Sh::kDK / 16, kAhead = 16;
  constexpr int kGroups = (Sh::kState / 4 + 255) / 256;
  const int64_t items = (int64_t)p.n_seq * p.H * kGroups;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int64_t nh = item / kGroups;
    const int part = (int)(item % kGroups), n = (int)(nh / p.H), h = (int)(nh % p.H);
    const int i = part * 256 + threadIdx.x;
    int64_t first;
    int len, slot = 0;
    lin_tokens(p, n, &first, &len);
    const int segments = segments_of(p, len);
    if (segments == 1) continue;
    if (!p.cu_seqlens) {
      slot = n * segments;
    } else if (p.n_seq > 64) {
      slot = starts_of(p)[n];
    } else {
      const int m = threadIdx.x & 63;
      if (m < n) {
        lin_tokens(p, m, &first, &len);
        const int x = segments_of(p, len);
        slot = x > 1 ? x : 0;
      }
#pragma unroll
      for (int d = 32; d >= 1; d >>= 1) slot += __shfl_xor(slot, d, 64);
    }
    const int there = min(segments, p.slots - slot);  // offsets that overlap give more segments than slots
    if (i >= Sh::kState / 4) continue;
    floatx4 e{0.f, 0.f, 0.f, 0.f};
    if (p.S0) {
      const int lane = i % 64, tile = i / 64, c = tile % CT, kt = tile / CT % KT, wave = tile / CT / KT;
      const float* in = p.S0 + nh * Sh::kState;
#pragma unroll
      for (int x = 0; x < 4; ++x)
        e[x] = in[Sh::key(kt >> 1, kt & 1, 4 * (lane >> 4) + x) * Sh::kDV + Sh::value(wave, c, lane & 15)];
    }
    floatx4* at = static_cast<floatx4*>(p.workspace) + i;
    const float* decays = decays_of(p);
    for (int s0 = 0; s0 < there; s0 += kAhead) {
      floatx4 z[kAhead];
      float a[kAhead];
#pragma unroll
      for (int s = 0; s < kAhead; ++s) {
        z[s] = floatx4{0.f, 0.f, 0.f, 0.f};
        a[s] = 1.f;
        if (s0 + s < there && s0 + s + 1 < segments) {
          z[s] = at[slot_of<Sh>(p, slot + s0 + s, h)];
          a[s] = decays[(int64_t)(slot + s0 + s) * p.H + h];
        }
      }
#pragma unroll
      for (int s = 0; s < kAhead; ++s) {
        if (s0 + s < there) {
          at[slot_of<Sh>(p, slot + s0 + s, h)] = e;
          e = e * a[s] + z[s];
        }
      }
    }
  }
}

// Workgroups that sum up segments. Up to 64 packed sequences give whole segments the first places, of which
// there are no more than T / seg. (64 sequences of 4,096 tokens together, 32 heads: 146 us, so 133.)
inline dim3 sums_grid(const LinPlan& p) {
  return dim3((unsigned)((int64_t)(p.cu_seqlens && p.n_seq <= 64 ? p.T / p.seg : p.jobs) * p.H));
}

// What comes before the walks: the jobs' table, and with segments their sums (`sum` launches them) and
// the states that enter them.
template <typename Sh, typename Sum>
void launch_before(const LinPlan& p, hipStream_t stream, Sum sum) {
  if (p.cu_seqlens && p.n_seq > 64) lin_jobs_kernel<<<1, 1024, 0, stream>>>(p);
  if (p.T <= p.seg) return;
  sum();
  constexpr int groups = (Sh::kState / 4 + 255) / 256;
  const int64_t items = (int64_t)p.n_seq * p.H * groups;
  // 2,048 are the card's places; sequences of one segment, which have nothing here, would cost a workgroup each
  // part (300 packed sequences of 32 heads: 455 us, so 396).
  lin_entries_kernel<Sh><<<dim3((unsigned)(items < 2048 ? items : 2048)), 256, 0, stream>>>(p);
}

}  // namespace

}  // namespace kda
