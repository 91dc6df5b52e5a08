// Verification of drafted tokens: which of them stand, and the token that follows.
//
// With p_j the target's and q_j the drafting distribution, draft x_j stands with probability
// min(1, p_j(x_j) / q_j(x_j)), here: u_j q_j(x_j) < p_j(x_j) for the uniform number u_j. At the
// first that falls, a, the following token is drawn from max(p_a - q_a, 0) normalised, which
// makes the sum of both ways p_a: min(p, q) + max(p - q, 0) = p. If all stand, it is drawn from
// p_a as it is. The draw inverts the cumulative sum: the smallest i with C_i > u C_V.
//
// What has to be read is one row of p and, where a draft fell, one of q: HBM bounds it for a
// batch, latency for one sequence. Two launches: in the first, every wave finds out which drafts
// stand (a few gathered values) and sums the weights of its blocks of 1024 tokens; in the second,
// one wave per sequence finds the block in the blocks' prefix sums and the token within the block.
// No wave waits for another there, so there are no barriers and no LDS.
//
// Sums are 64 bit in a fixed order: a token's share can be 10^-8 of the sum, less than 32 bits
// resolve next to it, and the result is the same on every run. Small vocabularies take one launch
// (verify_alone_kernel).
#include <algorithm>

#include "kda_device.h"
#include "kda_internal.h"

namespace kda {

namespace {

constexpr int kBlock = 1024;  // tokens per block sum: 16 of each lane

__device__ __forceinline__ float weight_of(float x) { return x > 0.f && x < INFINITY ? x : 0.f; }
__device__ __forceinline__ float uniform_of(float u) { return u > 0.f ? u < 1.f ? u : 0x1.fffffep-1f : 0.f; }

__device__ __forceinline__ int draft_count(const VerifyPlan& v, int n) {
  return v.n_drafts ? min(max(v.n_drafts[n], 0), v.m) : v.m;
}

// Drafts of sequence n that stand; one wave, 64 drafts at a time.
template <typename T>
__device__ __forceinline__ int standing(const VerifyPlan& v, int n, int count) {
  const T* p = static_cast<const T*>(v.p) + n * v.p_seq;
  const T* q = v.q ? static_cast<const T*>(v.q) + n * v.q_seq : nullptr;
  for (int j0 = 0; j0 < v.m; j0 += 64) {
    const int j = j0 + (threadIdx.x & 63);
    bool falls = false;
    if (j < v.m) {  // also those that are none: their number then arrives meanwhile
      const int x = v.drafts[(int64_t)n * v.m + j];
      const float u = uniform_of(v.uniform[(int64_t)n * (v.m + 1) + j]);
      falls = x < 0 || x >= v.V;
      if (!falls) {
        const float px = ld(p, j * v.p_row + x), qx = q ? ld(q, j * v.q_row + x) : 1.f;
        falls = !(fabsf(px) < INFINITY && fabsf(qx) < INFINITY && (double)u * (double)qx < (double)px);
      }
    }
    const uint64_t fallen = __ballot(falls && j < count);
    if (fallen) return j0 + __builtin_ctzll(fallen);
    if (j0 + 64 >= count) break;
  }
  return count;
}

// N neighbouring values of a row as floats, whatever the row's alignment (streamed).
template <int N>
__device__ __forceinline__ void load_row(const float* p, float* x) {
  typedef float vec __attribute__((ext_vector_type(4), aligned(4)));
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const vec y = __builtin_nontemporal_load(reinterpret_cast<const vec*>(p + i));
    x[i] = y[0], x[i + 1] = y[1], x[i + 2] = y[2], x[i + 3] = y[3];
  }
}
template <int N>
__device__ __forceinline__ void load_row(const uint16_t* p, float* x) {
  typedef uint16_t vec __attribute__((ext_vector_type(N < 8 ? N : 8), aligned(2)));
  constexpr int W = N < 8 ? N : 8;
#pragma unroll
  for (int i = 0; i < N; i += W) {
    const vec y = __builtin_nontemporal_load(reinterpret_cast<const vec*>(p + i));
#pragma unroll
    for (int k = 0; k < W; ++k) x[i + k] = bf16_bits_to_f32(y[k]);
  }
}

// The weights that decide: w = max(p - q, 0), and p in case they are all zero.
template <typename T>
struct Weights {
  const T *p, *q;  // rows; q NULL: nothing to take off, except 1 at token x
  int x;           // the draft that fell, if it was picked; -1 otherwise
  int V;
  // of tokens i .. i + N - 1 (0 past the vocabulary)
  template <int N>
  __device__ __forceinline__ void at(int i, double* w, double* all) const {
    float a[N], b[N];
#pragma unroll
    for (int k = 0; k < N; ++k) a[k] = b[k] = 0.f;
    if (i + N <= V) {
      load_row<N>(p + i, a);
      if (q) load_row<N>(q + i, b);
    } else {
#pragma unroll
      for (int k = 0; k < N; ++k) {
        if (i + k < V) {
          a[k] = ld(p, i + k);
          if (q) b[k] = ld(q, i + k);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const double pk = weight_of(a[k]);
      const double d = pk - (double)(i + k == x ? 1.f : weight_of(b[k]));
      w[k] = d > 0.0 ? d : 0.0;
      all[k] = pk;
    }
  }
};

template <typename T>
__device__ __forceinline__ Weights<T> weights(const VerifyPlan& v, int n, int a, int count) {
  Weights<T> w;
  w.p = static_cast<const T*>(v.p) + n * v.p_seq + a * v.p_row;
  w.q = a < count && v.q ? static_cast<const T*>(v.q) + n * v.q_seq + a * v.q_row : nullptr;
  w.x = a < count && !v.q ? v.drafts[(int64_t)n * v.m + a] : -1;
  w.V = v.V;
  return w;
}

__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) x += __shfl_xor(x, m, 64);
  return x;
}

// A wave's sums over block b: of w and of p, in every lane.
template <typename T>
__device__ __forceinline__ void block_sums(const Weights<T>& row, int b, double* w_sum, double* p_sum) {
  // Tokens per lane and step: 16 bytes, so a load instruction covers 1 KiB in one piece. (Eight fp32
  // values per lane, two instructions that each skip every other 16 bytes: 53 us where this takes 46.)
  constexpr int N = 16 / sizeof(T);
  const int lane = threadIdx.x & 63;
  double w = 0.0, all = 0.0;
#pragma unroll
  for (int c = 0; c < kBlock; c += 64 * N) {
    double wk[N], pk[N];
    row.template at<N>(b * kBlock + c + lane * N, wk, pk);
#pragma unroll
    for (int k = 0; k < N; ++k) {
      w += wk[k];
      all += pk[k];
    }
  }
  *w_sum = wave_sum(w);
  *p_sum = wave_sum(all);
}

// Four waves per workgroup, `waves` per sequence; wave i of a sequence sums blocks i, i + waves, ...
// into sums[n][block] = {sum of w, sum of p}.
template <typename T>
__global__ __launch_bounds__(256) void verify_sums_kernel(const VerifyPlan v, int blocks, int waves) {
  const int lane = threadIdx.x & 63;
  const int64_t wave = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = (int)(wave / waves), first = (int)(wave - (int64_t)n * waves);
  if (n >= v.N) return;
  const int count = draft_count(v, n);
  const int a = __builtin_amdgcn_readfirstlane(standing<T>(v, n, count));
  if (first == 0 && lane == 0) v.accept[n] = a;
  const Weights<T> row = weights<T>(v, n, a, count);
  double* out = static_cast<double*>(v.workspace) + (int64_t)n * blocks * 2;
  for (int b = first; b < blocks; b += waves) {
    double w, all;
    block_sums(row, b, &w, &all);
    if (lane < 2) out[2 * (int64_t)b + lane] = lane ? all : w;
  }
}

// Where a wave's running sum passes a threshold: the first lane with a positive x and base + x_0 +
// ... + x_lane > threshold; if rounding lets none pass, the last with a positive x; -1 if there
// is none. *before: base and the sum ahead of that lane.
__device__ __forceinline__ int find_lane(double x, double base, double threshold, double* before) {
  const int lane = threadIdx.x & 63;
  double incl = x;
#pragma unroll
  for (int s = 1; s < 64; s <<= 1) {
    const double y = __shfl_up(incl, s, 64);
    if (lane >= s) incl += y;
  }
  const uint64_t some = __ballot(x > 0.0), past = __ballot(x > 0.0 && base + incl > threshold);
  if (!some) return -1;
  const int found = past ? __builtin_ctzll(past) : 63 - __builtin_clzll(some);
  const double ahead = __shfl(incl, max(found - 1, 0), 64);
  *before = base + (found ? ahead : 0.0);
  return found;
}

// The tokens of sequence n, by one wave, from the blocks' sums.
template <typename T>
__device__ __forceinline__ void pick(const VerifyPlan& v, int n, int a, const Weights<T>& row,
                                     const double* sums, int blocks) {
  constexpr int K = kBlock / 64;
  constexpr int kKept = 2;  // blocks of a lane up to 131,072 tokens
  const int lane = threadIdx.x & 63;
  const float u = uniform_of(v.uniform[(int64_t)n * (v.m + 1) + v.m]);

  // each lane a run of blocks, the first kKept of which it keeps
  const int per = (blocks + 63) / 64, b0 = min(lane * per, blocks), b1 = min(b0 + per, blocks);
  double kept_w[kKept], kept_all[kKept], w = 0.0, all = 0.0;
#pragma unroll
  for (int k = 0; k < kKept; ++k) {
    const bool mine = b0 + k < b1;
    const int b = mine ? b0 + k : 0;
    kept_w[k] = mine ? sums[2 * (int64_t)b] : 0.0;
    kept_all[k] = mine ? sums[2 * (int64_t)b + 1] : 0.0;
  }
#pragma unroll
  for (int k = 0; k < kKept; ++k) {
    w += kept_w[k];
    all += kept_all[k];
  }
  for (int b = b0 + kKept; b < b1; ++b) {
    w += sums[2 * (int64_t)b];
    all += sums[2 * (int64_t)b + 1];
  }
  const double total_w = wave_sum(w), total_p = wave_sum(all);
  const int which = total_w > 0.0 ? 0 : 1;  // 1: no weight is positive, p itself
  const double threshold = (double)u * (which ? total_p : total_w);

  int next = -1;
  double base;
  const int owner = find_lane(which ? all : w, 0.0, threshold, &base);
  if (owner >= 0) {
    // the block among that lane's
    int block = -1;
    double block_base = base;
    bool passed_block = false;
    auto look = [&](int b, double s) {
      if (!passed_block && s > 0.0) {
        block = b;
        block_base = base;
        passed_block = base + s > threshold;
      }
      base += s;
    };
#pragma unroll
    for (int k = 0; k < kKept; ++k) look(owner * per + k, __shfl(which ? kept_all[k] : kept_w[k], owner, 64));
    for (int b = owner * per + kKept; b < min((owner + 1) * per, blocks) && !passed_block; ++b)
      look(b, sums[2 * (int64_t)b + which]);
    // the token within it: each lane K neighbouring ones
    double wk[K], pk[K], sum = 0.0;
    row.template at<K>(block * kBlock + lane * K, wk, pk);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      wk[k] = which ? pk[k] : wk[k];
      sum += wk[k];
    }
    const int at = find_lane(sum, block_base, threshold, &base);
    int mine = -1;
    bool passed = false;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (!passed && wk[k] > 0.0) {
        mine = k;
        passed = base + wk[k] > threshold;
      }
      base += wk[k];
    }
    next = block * kBlock + at * K + __shfl(mine, max(at, 0), 64);
  }
  for (int j = lane; j <= v.m; j += 64)
    v.tokens[(int64_t)n * (v.m + 1) + j] =
        j < a ? v.drafts[(int64_t)n * v.m + j] : j == a ? next : -1;
}

// One wave per sequence.
template <typename T>
__global__ __launch_bounds__(64) void verify_pick_kernel(const VerifyPlan v, int blocks) {
  const int n = blockIdx.x, a = v.accept[n];
  const Weights<T> row = weights<T>(v, n, a, draft_count(v, n));
  pick(v, n, a, row, static_cast<const double*>(v.workspace) + (int64_t)n * blocks * 2, blocks);
}

// All of it in one launch: a workgroup per sequence with a wave per block, whose sums meet in LDS.
constexpr int kAloneBlocks = 16;
template <typename T>
__global__ __launch_bounds__(64 * kAloneBlocks) void verify_alone_kernel(const VerifyPlan v, int blocks) {
  __shared__ double sums[2 * kAloneBlocks];
  const int n = blockIdx.x, lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int count = draft_count(v, n);
  const int a = __builtin_amdgcn_readfirstlane(standing<T>(v, n, count));
  const Weights<T> row = weights<T>(v, n, a, count);
  double w, all;
  block_sums(row, wave, &w, &all);
  if (lane < 2) sums[2 * wave + lane] = lane ? all : w;
  __syncthreads();
  if (wave) return;
  if (lane == 0) v.accept[n] = a;
  pick(v, n, a, row, sums, blocks);
}

int64_t row_blocks(int V) { return ((int64_t)V + kBlock - 1) / kBlock; }

template <typename T>
hipError_t launch_t(const VerifyPlan& p, hipStream_t stream) {
  const int blocks = (int)row_blocks(p.V);
  // One launch for small vocabularies and no more sequences than CUs: 4 drafts over 8,000 tokens 7.1 us
  // (two launches 8.3), 256 sequences 9.7 (11.8), 512 sequences 17.2 (14.9); with two blocks to a wave
  // it loses, one sequence over 32,000 tokens 10.8 us (8.2).
  if (blocks <= kAloneBlocks && p.N <= 256) {
    hipLaunchKernelGGL(verify_alone_kernel<T>, dim3((unsigned)p.N), dim3(64 * blocks), 0, stream, p, blocks);
    return hipGetLastError();
  }
  // A wave per block, up to 65,536 of them, eight times what the CUs hold: waves that begin while others
  // wait for their row keep HBM busy (512 x 4 drafts over 131,072 tokens 79 us, 87 with 8,192 waves).
  const int waves = (int)std::min<int64_t>(blocks, std::max<int64_t>(1, 65536 / p.N));
  hipLaunchKernelGGL(verify_sums_kernel<T>, dim3((unsigned)(((int64_t)waves * p.N + 3) / 4)), dim3(256), 0,
                     stream, p, blocks, waves);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(verify_pick_kernel<T>, dim3((unsigned)p.N), dim3(64), 0, stream, p, blocks);
  return hipGetLastError();
}

}  // namespace

size_t verify_workspace_bytes(int N, int V) { return (size_t)(row_blocks(V) * N) * 2 * sizeof(double); }
hipError_t launch_verify(const VerifyPlan& p, hipStream_t stream) {
  return p.bf16 ? launch_t<uint16_t>(p, stream) : launch_t<float>(p, stream);
}

}  // namespace kda
