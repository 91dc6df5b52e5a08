// Launch shape of the attention over a paged cache.
#include <algorithm>

#include "kda_internal.h"
#include "kda_paged_decode.h"

namespace kda {

namespace {

// Workgroups that share the work evenly: those that the 256 CUs hold at once, two each. Twice as
// many measured 5 to 8 % slower, and three each on an e4m3 cache (where the registers allow it) 4 %:
// each has its own start and leaves its own parts.
constexpr int64_t kShared = 256 * 2;
// Up to this many 128-token units, a (sequence, row block, head) is done by one workgroup, four
// waves to a head, with nothing left to join.
constexpr int64_t kAlone = 4;

size_t parts(const PagedDecodePlan& p) { return (size_t)p.split * 2 * p.heads * p.part_rows; }

}  // namespace

size_t plan_paged_decode(PagedDecodePlan* p) {
  p->group = p->Hq / p->Hkv;
  p->rows = p->m * p->group;
  p->tiles = p->rows > 16 ? 2 : 1;
  p->row_blocks = (p->rows + 16 * p->tiles - 1) / (16 * p->tiles);
  p->part_rows = std::min(p->rows, 16 * p->tiles);
  p->heads = 1;
  p->split = 0;
  int64_t span = p->max_len;
  if (p->window) span = std::min<int64_t>(span, (int64_t)p->window + p->m - 1 + 127);
  const int64_t units = (span + 127) / 128, all = (int64_t)p->N * p->row_blocks * p->Hkv;
  if (units <= kAlone) return 0;
  // Neighbouring heads together where every workgroup still has four units (of 128 tokens of one
  // head) or more; below that, the four waves of one head finish sooner.
  if (all * units >= 4 * kShared) p->heads = p->Hkv % 4 == 0 ? 4 : p->Hkv % 2 == 0 ? 2 : 1;
  p->split = (int)std::min(kShared, all * units);
  return parts(*p) * (p->d + 2) * sizeof(float) + (size_t)(all / p->heads) * 2 * sizeof(int);
}

void paged_decode_workspace(PagedDecodePlan* p, void* workspace) {
  p->part_o = static_cast<float*>(workspace);
  p->part_ml = p->part_o + parts(*p) * p->d;
  p->part_of = reinterpret_cast<int*>(p->part_ml + parts(*p) * 2);
}

hipError_t launch_paged_decode(const PagedDecodePlan& p, hipStream_t stream) {
  if (p.cache_type == kF32) return launch_paged_decode_f32(p, stream);
  return p.cache_type == kBF16 ? launch_paged_decode_bf16(p, stream)
                               : launch_paged_decode_e4m3(p, stream);
}

}  // namespace kda
