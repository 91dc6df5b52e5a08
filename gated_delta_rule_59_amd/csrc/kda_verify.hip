// Verification of drafted tokens: which of them stand, and the token that follows.
//
// With p_j the target's and q_j the drafting distribution, draft x_j stands with probability
// min(1, p_j(x_j) / q_j(x_j)), here: u_j q_j(x_j) < p_j(x_j) for the uniform number u_j. At the
// first that falls, a, the following token is drawn from max(p_a - q_a, 0) normalised, which
// makes the sum of both ways p_a: min(p, q) + max(p - q, 0) = p. If all stand, it is drawn from
// p_a as it is. The draw inverts the cumulative sum: the smallest i with C_i > u C_V.
//
// What has to be read is one row of p and, where a draft fell, one of q: HBM bounds it for a
// batch, latency for one sequence. Two launches: the first sums the weights of every block of
// kBlock tokens (grid over blocks and sequences, 64-bit sums), the second, one workgroup per
// sequence, finds the block in the blocks' prefix sums and the token within the block.
//
// Sums are 64 bit in a fixed order: a token's share can be 10^-8 of the sum, less than 32 bits
// resolve next to it, and the result is the same on every run.
#include "kda_device.h"
#include "kda_internal.h"

namespace kda {

namespace {

constexpr int kBlock = 2048;  // tokens per block sum: 8 of each of 256 threads

__device__ __forceinline__ float weight_of(float x) { return x > 0.f && x < INFINITY ? x : 0.f; }

// Drafts of sequence n that stand; every thread of the workgroup gets it. (Threads take drafts
// t, t + 256, ...; the first that falls counts.)
template <typename T>
__device__ __forceinline__ int standing(const VerifyPlan& v, int n, int count, int* s_first) {
  const T* p = static_cast<const T*>(v.p) + n * v.p_seq;
  const T* q = static_cast<const T*>(v.q);
  if (threadIdx.x == 0) *s_first = count;
  __syncthreads();
  for (int j = threadIdx.x; j < count; j += 256) {
    const int x = v.drafts[(int64_t)n * v.m + j];
    bool stands = x >= 0 && x < v.V;
    if (stands) {
      const float px = ld(p, j * v.p_row + x);
      const float qx = q ? ld(q + n * v.q_seq, j * v.q_row + x) : 1.f;
      float u = v.uniform[(int64_t)n * (v.m + 1) + j];
      u = u > 0.f ? u < 1.f ? u : 0x1.fffffep-1f : 0.f;
      stands = fabsf(px) < INFINITY && fabsf(qx) < INFINITY && (double)u * (double)qx < (double)px;
    }
    if (!stands) atomicMin(s_first, j);
  }
  __syncthreads();
  return *s_first;
}

// The weights that decide: w = max(p - q, 0), and p in case they are all zero.
template <typename T>
struct Weights {
  const T *p, *q;  // rows; q NULL: nothing to take off, except at token x
  int x;           // the draft that fell, if it was picked; -1 otherwise
  __device__ __forceinline__ void at(int i, double& w, double& all) const {
    const float pi = weight_of(ld(p, i));
    all = pi;
    if (q) {
      const double d = (double)pi - (double)weight_of(ld(q, i));
      w = d > 0.0 ? d : 0.0;
    } else {
      w = i == x ? fmax((double)pi - 1.0, 0.0) : (double)pi;
    }
  }
};

template <typename T>
__device__ __forceinline__ Weights<T> weights(const VerifyPlan& v, int n, int a, int count) {
  Weights<T> w;
  w.p = static_cast<const T*>(v.p) + n * v.p_seq + a * v.p_row;
  w.q = a < count && v.q ? static_cast<const T*>(v.q) + n * v.q_seq + a * v.q_row : nullptr;
  w.x = a < count && !v.q ? v.drafts[(int64_t)n * v.m + a] : -1;
  return w;
}

__device__ __forceinline__ int draft_count(const VerifyPlan& v, int n) {
  return v.n_drafts ? min(max(v.n_drafts[n], 0), v.m) : v.m;
}

__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) x += __shfl_xor(x, m, 64);
  return x;
}

// Grid: x over blocks of kBlock tokens, then sequences. sums[n][block] = {sum w, sum p}.
template <typename T>
__global__ __launch_bounds__(256) void verify_sums_kernel(const VerifyPlan v, int blocks) {
  __shared__ int s_first;
  __shared__ double s_part[2][4];
  const int n = blockIdx.x / blocks, b = blockIdx.x % blocks;
  const int t = threadIdx.x;
  const int count = draft_count(v, n);
  const int a = standing<T>(v, n, count, &s_first);
  const Weights<T> row = weights<T>(v, n, a, count);
  double w = 0.0, all = 0.0;
#pragma unroll
  for (int c = 0; c < kBlock / 256; ++c) {
    const int i = b * kBlock + c * 256 + t;
    if (i < v.V) {
      double wi, pi;
      row.at(i, wi, pi);
      w += wi;
      all += pi;
    }
  }
  w = wave_sum(w);
  all = wave_sum(all);
  if ((t & 63) == 0) {
    s_part[0][t >> 6] = w;
    s_part[1][t >> 6] = all;
  }
  __syncthreads();
  if (t < 2) {
    double* out = static_cast<double*>(v.workspace) + ((int64_t)n * blocks + b) * 2;
    out[t] = (s_part[t][0] + s_part[t][1]) + (s_part[t][2] + s_part[t][3]);
  }
}

// The first index i < count (in order) whose running sum base + x_0 + ... + x_i exceeds the
// threshold; thread t holds elements [t * K, t * K + K). If none does, the last positive one; -1
// if none is positive. *base_out: the sum before it. Every thread gets the result.
template <int K>
__device__ int find_first(const double* x, double base, double threshold, double* s_w, int* s_idx,
                          double* base_out) {
  const int t = threadIdx.x, lane = t & 63, wv = t >> 6;
  double own = 0.0;
#pragma unroll
  for (int k = 0; k < K; ++k) own += x[k];
  double incl = own;
#pragma unroll
  for (int s = 1; s < 64; s <<= 1) {
    const double y = __shfl_up(incl, s, 64);
    if (lane >= s) incl += y;
  }
  if (lane == 63) s_w[wv] = incl;
  if (t == 0) s_idx[0] = 0x7fffffff, s_idx[1] = -1;
  __syncthreads();
  double run = base;
  for (int i = 0; i < wv; ++i) run += s_w[i];
  run += incl - own;
  double prev = run;
  int hit = 0x7fffffff, lastpos = -1;
  double hit_base = 0.0, last_base = 0.0;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (x[k] > 0.0) {
      lastpos = t * K + k;
      last_base = prev;
      if (hit == 0x7fffffff && prev + x[k] > threshold) {
        hit = t * K + k;
        hit_base = prev;
      }
    }
    prev += x[k];
  }
  if (hit != 0x7fffffff) atomicMin(&s_idx[0], hit);
  if (lastpos >= 0) atomicMax(&s_idx[1], lastpos);
  __syncthreads();
  const int found = s_idx[0] != 0x7fffffff ? s_idx[0] : s_idx[1];
  if (found >= 0 && found / K == t) s_w[4] = s_idx[0] != 0x7fffffff ? hit_base : last_base;
  __syncthreads();
  *base_out = s_w[4];
  return found;
}

// One workgroup per sequence.
template <typename T>
__global__ __launch_bounds__(256) void verify_pick_kernel(const VerifyPlan v, int blocks) {
  __shared__ int s_first, s_idx[2];
  __shared__ double s_w[5];
  const int n = blockIdx.x, t = threadIdx.x;
  const int count = draft_count(v, n);
  const int a = standing<T>(v, n, count, &s_first);
  const Weights<T> row = weights<T>(v, n, a, count);
  const double* sums = static_cast<const double*>(v.workspace) + (int64_t)n * blocks * 2;

  // totals, and whether w has anything
  double w = 0.0, all = 0.0;
  for (int i = t; i < blocks; i += 256) {
    w += sums[2 * i];
    all += sums[2 * i + 1];
  }
  w = wave_sum(w);
  all = wave_sum(all);
  if ((t & 63) == 0) s_w[t >> 6] = w;
  __syncthreads();
  const double total_w = (s_w[0] + s_w[1]) + (s_w[2] + s_w[3]);
  __syncthreads();
  if ((t & 63) == 0) s_w[t >> 6] = all;
  __syncthreads();
  const double total_p = (s_w[0] + s_w[1]) + (s_w[2] + s_w[3]);
  __syncthreads();
  const int which = total_w > 0.0 ? 0 : 1;
  const double total = which ? total_p : total_w;

  int next = -1;
  if (total > 0.0) {
    float u = v.uniform[(int64_t)n * (v.m + 1) + v.m];
    u = u > 0.f ? u < 1.f ? u : 0x1.fffffep-1f : 0.f;
    const double threshold = (double)u * total;
    // the block: 256 blocks at a time, each thread one. The first whose running sum passes the
    // threshold, or (if rounding lets none pass) the last that has any weight.
    double base = 0.0, block_base = 0.0;
    int block = -1;
    for (int b0 = 0; b0 < blocks; b0 += 256) {
      const double x = b0 + t < blocks ? sums[2 * (b0 + t) + which] : 0.0;
      double before;
      const int f = find_first<1>(&x, base, threshold, s_w, s_idx, &before);
      if (f < 0) continue;
      block = b0 + f;
      block_base = before;
      base = before + sums[2 * block + which];
      if (base > threshold) break;
    }
    // the token within it
    if (block >= 0) {
      constexpr int K = kBlock / 256;
      double x[K];
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int i = block * kBlock + t * K + k;
        double wi = 0.0, pi = 0.0;
        if (i < v.V) row.at(i, wi, pi);
        x[k] = which ? pi : wi;
      }
      double before;
      next = find_first<K>(x, block_base, threshold, s_w, s_idx, &before);
      if (next >= 0) next += block * kBlock;
    }
  }
  if (t == 0) v.accept[n] = a;
  for (int j = t; j <= v.m; j += 256)
    v.tokens[(int64_t)n * (v.m + 1) + j] =
        j < a ? v.drafts[(int64_t)n * v.m + j] : j == a ? next : -1;
}

int64_t row_blocks(int V) { return ((int64_t)V + kBlock - 1) / kBlock; }

template <typename T>
hipError_t launch_t(const VerifyPlan& p, hipStream_t stream) {
  const int blocks = (int)row_blocks(p.V);
  hipLaunchKernelGGL(verify_sums_kernel<T>, dim3((unsigned)((int64_t)blocks * p.N)), dim3(256), 0,
                     stream, p, blocks);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(verify_pick_kernel<T>, dim3((unsigned)p.N), dim3(256), 0, stream, p, blocks);
  return hipGetLastError();
}

}  // namespace

int64_t verify_blocks(int N, int V) { return row_blocks(V) * N; }
size_t verify_workspace_bytes(int N, int V) {
  return (size_t)verify_blocks(N, V) * 2 * sizeof(double);
}
hipError_t launch_verify(const VerifyPlan& p, hipStream_t stream) {
  return p.bf16 ? launch_t<uint16_t>(p, stream) : launch_t<float>(p, stream);
}

}  // namespace kda
