// Pages, offsets, positions and slots of a step's new tokens.
//
// Prefix sums over the sequences say which pages of the free ring and which rows of the step are whose;
// then every new page, every token and every page that comes back is one independent item that finds
// its sequence by bisection. A few KiB are read and written: the launch and a chain of dependent
// loads bound it.
//
// One launch, no workspace: every workgroup forms the sums over all sequences for itself (some
// microseconds' worth of adds for hundreds of sequences, which two launches or a wait between workgroups
// would exceed) and takes its share of the items. Workgroups do not see each other's writes: what the
// call updates and what it reads lie apart. Held and ring are written elsewhere; table entries below
// held are read, those from held on written; ring entries below count are read, those from count on
// written.
#include <algorithm>

#include "kda_device.h"
#include "kda_internal.h"

namespace kda {

namespace {

constexpr int kThreads = 256, kPer = 4, kTile = kThreads * kPer;  // sequences at a time

// Sums that stop at 2^32 - 1, which is above every bound here.
__device__ __forceinline__ unsigned plus(unsigned a, unsigned b) { return __builtin_elementwise_add_sat(a, b); }

template <int CTRL, int ROWS>
__device__ __forceinline__ unsigned plus_lane(unsigned x) {
  return plus(x, (unsigned)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, ROWS, 0xf, false));
}
// Sums over the wave's lanes up to each (16 lanes in four steps, then rows of 16 in two).
__device__ __forceinline__ unsigned wave_sums(unsigned x) {
  x = plus_lane<0x111, 0xf>(x);
  x = plus_lane<0x112, 0xf>(x);
  x = plus_lane<0x114, 0xf>(x);
  x = plus_lane<0x118, 0xf>(x);
  x = plus_lane<0x142, 0xa>(x);
  return plus_lane<0x143, 0xc>(x);
}
// Sums over the workgroup's threads before each, of M numbers at once, and the totals. `s` is scratch that
// nothing else uses until the next barrier but one.
template <int M>
__device__ __forceinline__ void sums_before(unsigned (&x)[M], unsigned (&total)[M], unsigned (*s)[M]) {
  const int wave = threadIdx.x >> 6;
  unsigned to[M];
#pragma unroll
  for (int m = 0; m < M; ++m) to[m] = wave_sums(x[m]);
  if ((threadIdx.x & 63) == 63) {
#pragma unroll
    for (int m = 0; m < M; ++m) s[wave][m] = to[m];
  }
  __syncthreads();
#pragma unroll
  for (int m = 0; m < M; ++m) {
    unsigned before = (unsigned)__builtin_amdgcn_update_dpp(0, (int)to[m], 0x138, 0xf, 0xf, false);  // the lane below
    unsigned below = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w) {
      if (w < wave) below = plus(below, s[w][m]);
      all = plus(all, s[w][m]);
    }
    x[m] = plus(before, below);
    total[m] = all;
  }
}

// kPer neighbouring numbers, 0 past the end.
__device__ __forceinline__ void load_per(const int32_t* p, int n, int N, int* x) {
  typedef int vec __attribute__((ext_vector_type(kPer), aligned(4)));
#pragma unroll
  for (int i = 0; i < kPer; ++i) x[i] = 0;
  if (n + kPer <= N) {
    const vec y = *reinterpret_cast<const vec*>(p + n);
#pragma unroll
    for (int i = 0; i < kPer; ++i) x[i] = y[i];
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (n + i < N) x[i] = p[n + i];
  }
}

// The last of n ascending numbers that is not above x (the first one is not).
__device__ __forceinline__ int last_at_most(const int* a, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ __launch_bounds__(kThreads) void page_plan_kernel(const PagePlan p, unsigned ps_mul, int ps_shift) {
  __shared__ int s_page[kTile], s_token[kTile], s_back[kTile], s_held[kTile], s_len[kTile];
  const int t = threadIdx.x;
  const bool first = blockIdx.x == 0;
  const unsigned step = gridDim.x * kThreads, mine = blockIdx.x * kThreads + t;
  const unsigned cap = p.cap;
  const unsigned head = (unsigned)max(p.ring[0], 0) % cap;
  const int count = min(max(p.ring[1], 0), p.cap);
  auto place = [&](unsigned i) {  // entry i < cap of the ring, counted from its head
    const unsigned x = head + i;
    return x >= cap ? x - cap : x;
  };

  auto page_of = [&](unsigned pos) { return (unsigned)(((uint64_t)pos * ps_mul) >> ps_shift); };

  __shared__ unsigned s_asked[kThreads / 64][2], s_served[kThreads / 64][3];
  unsigned asked[2] = {0, 0};       // pages, tokens of the tiles so far
  unsigned done[3] = {0, 0, 0};     // pages and tokens served, pages that come back
  const unsigned pages_there = count, tokens_there = p.max_tokens;
  for (int base = 0; base < p.N; base += kTile) {
    int held[kPer], len[kPer], need[kPer], fresh[kPer];
    bool ends[kPer];
    const int n0 = base + t * kPer;
    load_per(p.held, n0, p.N, held);
    load_per(p.lens, n0, p.N, len);
    load_per(p.new_lens, n0, p.N, fresh);
    unsigned before[2] = {0, 0}, all[2];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      held[i] = min(max(held[i], 0), p.max_pages);
      len[i] = max(len[i], 0);
      ends[i] = fresh[i] < 0;
      const unsigned end = (unsigned)len[i] + (unsigned)max(fresh[i], 0);  // below 2^32
      const int pages = end ? (int)page_of(min(end, (unsigned)INT32_MAX) - 1) + 1 : 0;
      // masks, not branches: see below
      const int fits = (n0 + i < p.N) & !ends[i] & (end <= (unsigned)INT32_MAX) & (pages <= p.max_pages);
      need[i] = max(0, pages - held[i]) & -fits;
      fresh[i] &= -fits;
      before[0] = plus(before[0], need[i]);
      before[1] = plus(before[1], fresh[i]);
    }
    sums_before(before, all, s_asked);
    unsigned pages_to = plus(asked[0], before[0]), tokens_to = plus(asked[1], before[1]);
    asked[0] = plus(asked[0], all[0]);
    asked[1] = plus(asked[1], all[1]);
    // who is served; their sums (at most count pages and max_tokens tokens), and what comes back
    unsigned at[3] = {0, 0, 0}, more[3];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      pages_to = plus(pages_to, need[i]);
      tokens_to = plus(tokens_to, fresh[i]);
      // Masks, not branches: with `if (!served) need[i] = fresh[i] = 0` the compiler (ROCm 7.2) leaves the
      // first sequence of a thread served that passes the first condition and fails the second.
      const int served = ((need[i] == 0) | (pages_to <= pages_there)) & ((fresh[i] == 0) | (tokens_to <= tokens_there));
      need[i] &= -served;
      fresh[i] &= -served;
      at[0] += need[i];
      at[1] += fresh[i];
      at[2] = plus(at[2], ends[i] ? held[i] : 0);
    }
    sums_before(at, more, s_served);
#pragma unroll
    for (int m = 0; m < 3; ++m) at[m] = plus(at[m], done[m]);
    const int n_tile = min(kTile, p.N - base);
    const unsigned used = done[0], tokens = done[1], back = done[2];
    const unsigned all_need = more[0], all_fresh = more[1], all_back = more[2];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int x = t * kPer + i, n = n0 + i;
      s_page[x] = at[0];
      s_token[x] = at[1];
      s_back[x] = min(at[2], (unsigned)INT32_MAX);
      s_held[x] = held[i];
      s_len[x] = len[i];
      if (first && n < p.N) {
        p.held_out[n] = ends[i] ? 0 : held[i] + need[i];
        p.seq_lens[n] = ends[i] ? 0 : len[i] + fresh[i];
        p.cu_seqlens[n] = at[1];
      }
      at[0] += need[i];
      at[1] += fresh[i];
      at[2] = plus(at[2], ends[i] ? held[i] : 0);
    }
    __syncthreads();
    // pages from the ring into the table
    for (unsigned i = used + mine; i < used + all_need; i += step) {
      const int x = last_at_most(s_page, n_tile, i);
      p.table[(base + x) * p.table_stride + s_held[x] + (i - s_page[x])] = p.free_pages[place(i)];
    }
    // slots and positions
    if (p.slots || p.positions) {
      for (unsigned i = tokens + mine; i < tokens + all_fresh; i += step) {
        const int x = last_at_most(s_token, n_tile, i);
        const int pos = s_len[x] + (i - s_token[x]);
        if (p.positions) p.positions[i] = pos;
        if (p.slots) {
          const int page = (int)page_of(pos);
          const int id = page < s_held[x] ? p.table[(base + x) * p.table_stride + page]
                                          : p.free_pages[place(s_page[x] + (page - s_held[x]))];
          p.slots[i] = id < 0 ? -1 : (int64_t)id * p.page_size + (pos - page * p.page_size);
        }
      }
    }
    // pages of ended sequences into the ring, as far as it has room
    const int64_t room = (int64_t)p.cap - count;
    const int64_t back_end = min((int64_t)back + all_back, room);
    for (int64_t i = (int64_t)back + mine; i < back_end; i += step) {
      const int x = last_at_most(s_back, n_tile, (int)i);
      p.free_pages[place((unsigned)(count + i))] = p.table[(base + x) * p.table_stride + (i - s_back[x])];
    }
#pragma unroll
    for (int m = 0; m < 3; ++m) done[m] = plus(done[m], more[m]);
    if (base + kTile < p.N) __syncthreads();
  }
  for (int64_t i = (int64_t)done[1] + mine; i < p.max_tokens; i += step) {
    if (p.slots) p.slots[i] = -1;
    if (p.positions) p.positions[i] = -1;
  }
  if (first && t == 0) {
    p.cu_seqlens[p.N] = done[1];
    p.ring_out[0] = (int)(((int64_t)head + done[0]) % cap);
    p.ring_out[1] = count - (int)done[0] + (int)min((int64_t)done[2], (int64_t)p.cap - count);
  }
}

}  // namespace

hipError_t launch_page_plan(const PagePlan& p, hipStream_t stream) {
  unsigned mul;
  int shift;
  divide_by(p.page_size, &mul, &shift);
  // A token per thread, and 16 workgroups at least, which the pages that come back are shared by too (512
  // sequences of which 9 end: 9.8 us with one workgroup, 5.9 with 16).
  const int groups = std::min(512, std::max(16, (int)(((int64_t)p.max_tokens + kThreads - 1) / kThreads)));
  page_plan_kernel<<<groups, kThreads, 0, stream>>>(p, mul, shift);
  return hipGetLastError();
}

}  // namespace kda
