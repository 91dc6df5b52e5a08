// Launch shape of the attention over a paged cache.
#include <algorithm>

#include "kda_internal.h"
#include "kda_paged_decode.h"

namespace kda {

namespace {
// Workgroups that share the work evenly: those that the 256 CUs hold at once (three each with
// one row tile, two with two).
constexpr int kShared1 = 256 * 2, kShared2 = 256 * 2;
// Up to this many units of 128 tokens a (sequence, row block, head) is done by one workgroup.
constexpr int64_t kAlone = 4;
}  // namespace

size_t plan_paged_decode(PagedDecodePlan* p) {
  p->group = p->Hq / p->Hkv;
  p->rows = p->m * p->group;
  p->tiles = p->rows > 16 ? 2 : 1;
  p->row_blocks = (p->rows + 16 * p->tiles - 1) / (16 * p->tiles);
  int64_t span = p->max_len;
  if (p->window) span = std::min<int64_t>(span, (int64_t)p->window + p->m - 1 + paged::kUnit - 1);
  const int64_t units = (span + paged::kUnit - 1) / paged::kUnit;
  const int64_t all = (int64_t)p->N * p->row_blocks * p->Hkv;
  if (units <= kAlone) {
    p->split = 0;
    return 0;
  }
  p->split = (int)std::min<int64_t>(p->tiles == 1 ? kShared1 : kShared2, all * units);
  return (size_t)p->split * 2 * 16 * p->tiles * (p->d + 2) * sizeof(float);
}

hipError_t launch_paged_decode(const PagedDecodePlan& p, hipStream_t stream) {
  if (p.cache_type == kF32) return launch_paged_decode_f32(p, stream);
  return p.cache_type == kBF16 ? launch_paged_decode_bf16(p, stream)
                               : launch_paged_decode_e4m3(p, stream);
}

}  // namespace kda
