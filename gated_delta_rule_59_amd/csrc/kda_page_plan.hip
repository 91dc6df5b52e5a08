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

// Inclusive sums over the workgroup's threads; the total too.
template <typename T>
__device__ __forceinline__ T block_scan(T x, T* total) {
  __shared__ T s_wave[kThreads / 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const T y = __shfl_up(x, d, 64);
    if (lane >= d) x += y;
  }
  if (lane == 63) s_wave[wave] = x;
  __syncthreads();
  T all = 0, before = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) {
    if (w < wave) before += s_wave[w];
    all += s_wave[w];
  }
  __syncthreads();
  *total = all;
  return x + before;
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

  int64_t asked_pages = 0, asked_tokens = 0, back = 0;  // of the tiles so far
  int used = 0, tokens = 0;
  for (int base = 0; base < p.N; base += kTile) {
    int held[kPer], len[kPer], need[kPer], fresh[kPer];
    bool ends[kPer], fits[kPer];
    int64_t pages_sum = 0, tokens_sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int n = base + t * kPer + i;
      const bool real = n < p.N;
      held[i] = real ? min(max(p.held[n], 0), p.max_pages) : 0;
      len[i] = real ? max(p.lens[n], 0) : 0;
      const int x = real ? p.new_lens[n] : 0;
      ends[i] = x < 0;
      const unsigned end = (unsigned)len[i] + (unsigned)max(x, 0);  // below 2^32
      const int pages = end ? (int)page_of(min(end, (unsigned)INT32_MAX) - 1) + 1 : 0;
      fits[i] = real && !ends[i] && end <= (unsigned)INT32_MAX && pages <= p.max_pages;
      need[i] = fits[i] ? max(0, pages - held[i]) : 0;
      fresh[i] = fits[i] ? x : 0;
      pages_sum += need[i];
      tokens_sum += fresh[i];
    }
    int64_t all_pages, all_tokens;
    int64_t pages_to = block_scan(pages_sum, &all_pages) - pages_sum + asked_pages;
    int64_t tokens_to = block_scan(tokens_sum, &all_tokens) - tokens_sum + asked_tokens;
    asked_pages += all_pages;
    asked_tokens += all_tokens;
    // who is served; their sums (at most count pages and max_tokens tokens), and what comes back
    int need_sum = 0, fresh_sum = 0;
    int64_t back_sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      pages_to += need[i];
      tokens_to += fresh[i];
      // Masks, not branches: with `if (!served) need[i] = fresh[i] = 0` the compiler (ROCm 7.2) leaves the
      // first sequence of a thread served that passes the first condition and fails the second.
      const int served = ((need[i] == 0) | (pages_to <= count)) & ((fresh[i] == 0) | (tokens_to <= p.max_tokens));
      need[i] &= -served;
      fresh[i] &= -served;
      need_sum += need[i];
      fresh_sum += fresh[i];
      back_sum += ends[i] ? held[i] : 0;
    }
    int64_t all_back;
    int all_need, all_fresh;
    int page_at = block_scan(need_sum, &all_need) - need_sum + used;
    int token_at = block_scan(fresh_sum, &all_fresh) - fresh_sum + tokens;
    int64_t back_at = block_scan(back_sum, &all_back) - back_sum + back;
    const int n_tile = min(kTile, p.N - base);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int x = t * kPer + i, n = base + x;
      s_page[x] = page_at;
      s_token[x] = token_at;
      s_back[x] = (int)min(back_at, (int64_t)INT32_MAX);
      s_held[x] = held[i];
      s_len[x] = len[i];
      if (first && n < p.N) {
        p.held_out[n] = ends[i] ? 0 : held[i] + need[i];
        p.seq_lens[n] = ends[i] ? 0 : len[i] + fresh[i];
        p.cu_seqlens[n] = token_at;
      }
      page_at += need[i];
      token_at += fresh[i];
      back_at += ends[i] ? held[i] : 0;
    }
    __syncthreads();
    // pages from the ring into the table
    for (unsigned i = used + mine; i < (unsigned)(used + all_need); i += step) {
      const int x = last_at_most(s_page, n_tile, i);
      p.table[(base + x) * p.table_stride + s_held[x] + (i - s_page[x])] = p.free_pages[place(i)];
    }
    // slots and positions
    if (p.slots || p.positions) {
      for (unsigned i = tokens + mine; i < (unsigned)(tokens + all_fresh); i += step) {
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
    const int64_t back_end = min(back + all_back, room);
    for (int64_t i = back + mine; i < back_end; i += step) {
      const int x = last_at_most(s_back, n_tile, (int)i);
      p.free_pages[place((unsigned)(count + i))] = p.table[(base + x) * p.table_stride + (i - s_back[x])];
    }
    used += all_need;
    tokens += all_fresh;
    back += all_back;
    __syncthreads();
  }
  for (int64_t i = (int64_t)tokens + mine; i < p.max_tokens; i += step) {
    if (p.slots) p.slots[i] = -1;
    if (p.positions) p.positions[i] = -1;
  }
  if (first && t == 0) {
    p.cu_seqlens[p.N] = tokens;
    p.ring_out[0] = (int)(((int64_t)head + used) % cap);
    p.ring_out[1] = count - used + (int)min(back, (int64_t)p.cap - count);
  }
}

}  // namespace

hipError_t launch_page_plan(const PagePlan& p, hipStream_t stream) {
  unsigned mul;
  int shift;
  divide_by(p.page_size, &mul, &shift);
  const int groups = std::min(256, std::max(1, (p.max_tokens + 4 * kThreads - 1) / (4 * kThreads)));
  page_plan_kernel<<<groups, kThreads, 0, stream>>>(p, mul, shift);
  return hipGetLastError();
}

}  // namespace kda
