// Launch shape of the attention over a paged cache.
#include <algorithm>

#include "kda_internal.h"
#include "kda_paged_decode.h"

namespace kda {

namespace {

// Workgroups that share the work evenly: one per CU, whose four waves have 32 to 64 KiB of keys
// and values in flight, or two where 32 tokens are only 4 KiB or less. More measured slower (each has a start
// and leaves parts of its own, and more places of memory are open at a time): 4 contexts of 65k tokens
// 178 us with 256 workgroups, 190 with 512; e4m3 heads of 64 channels 241 us with 512, 281 with 256.
int tile_bytes(const PagedDecodePlan& p) {
  return 2 * 32 * p.d * (p.cache_type == kF32 ? 4 : p.cache_type == kBF16 ? 2 : 1);
}
int64_t shared_workgroups(const PagedDecodePlan& p) { return 256 * (tile_bytes(p) >= 8192 ? 1 : 2); }
// What beginning a (sequence, row block, head group) costs a workgroup (its queries and first keys have
// to arrive, its rows are finished) before it is back to reading, in units: the time in which a CU
// reads 128 KiB. Counted where a workgroup has several; where several workgroups share one, it would
// leave the others more. 512 contexts, 8 heads of 128 channels, e4m3: of up to 600 tokens 105.8 us
// without, 89 with 2 units, 86 with 3 or 4, 89 with 6; of up to 4096 tokens 364, 353, 348, 349. bf16,
// of up to 600 tokens: 124 without, 118 with 1 or 2, 123 with 4.
int start_units(const PagedDecodePlan& p) {
  const int64_t groups = (int64_t)p.N * p.row_blocks * p.groups;
  return groups < p.split ? 0 : std::max(1, (int)(32768 / (tile_bytes(p) * (shared_workgroups(p) / 256))));
}
// Up to this many (sequence, row block, head)s, of this many 128-token units each and together, are
// done by one workgroup each, four waves to a head, with nothing left to join. Beyond, sharing wins
// (us alone and shared, 8 heads, bf16): one context of 512 tokens 10.2 and 11.1, of 1,024 tokens 16.5 and
// 12.2 (a CU reads only some 55 GB/s); 64 contexts of up to 200 tokens 11.4 and 17.7, of up to 512
// 21.2 and 20.5; 128 contexts of up to 128 tokens 18.7 and 19.7, of up to 200 22.9 and 22.0, of up to 512
// 38 and 31; 256 contexts of up to 60 tokens 27.8 and 23.9.
constexpr int64_t kAloneUnits = 4, kAlonePairs = 1024, kAloneAll = 2048;

size_t parts(const PagedDecodePlan& p) { return (size_t)p.split * 2 * p.heads * p.part_rows; }

}  // namespace

size_t plan_paged_decode(PagedDecodePlan* p) {
  p->group = p->Hq / p->Hkv;
  p->rows = p->m * p->group;
  p->tiles = p->rows > 16 ? 2 : 1;
  p->row_blocks = (p->rows + 16 * p->tiles - 1) / (16 * p->tiles);
  p->part_rows = std::min(p->rows, 16 * p->tiles);
  p->heads = 1;
  p->groups = p->Hkv;
  p->unit_log = 7;
  divide_by(p->group, &p->group_mul, &p->group_shift);
  p->split = 0;
  p->hold = 0;
  p->start = 0;
  int64_t span = p->max_len;
  if (p->window) span = std::min<int64_t>(span, (int64_t)p->window + p->m - 1 + 127);
  const int64_t units = (span + 127) / 128, all = (int64_t)p->N * p->row_blocks * p->Hkv;
  if (units <= kAloneUnits && all <= kAlonePairs && all * units <= kAloneAll) return 0;
  // Neighbouring heads together where every workgroup still has four units (of 128 tokens of one
  // head) or more; below that, the four waves of one head finish sooner.
  const int64_t shared = shared_workgroups(*p);
  if (all * units >= 4 * shared) {
    const int log = p->Hkv % 4 == 0 ? 2 : p->Hkv % 2 == 0 ? 1 : 0;
    p->heads = 1 << log;
    p->groups = p->Hkv >> log;
    p->unit_log = 7 - log;
  }
  p->split = (int)std::min(shared, all * units);
  p->start = start_units(*p);
  if (p->heads == 4) {
    // room for a workgroup's share of the pairs, one more that it shares at either end, and one that
    // is uneven; at most what the CU has (160 KiB for its one or two workgroups, less 512 B that they
    // use otherwise and a scratch of 32 tokens x rows), which is one result at least: e4m3 heads of 64
    // channels with 32 rows have room for one fp32 result (8,736 of 16,256 B), others for two or more
    const int64_t entry = sizeof(paged::Held) + p->part_rows * (p->d * (int64_t)sizeof(float) + paged::kHeldPad);
    const int64_t room = (160 * 1024 * 256 / shared - 512) / 4 - 32 * 16 * p->tiles * (int64_t)sizeof(float);
    const int64_t pairs = (int64_t)p->N * p->row_blocks * p->groups;
    p->hold = (int)std::min(room, entry * ((pairs + p->split - 1) / p->split + 2)) & ~15;
  }
  // Grows with the units, so a window or a smaller max_len never needs more: split does; and where heads
  // grows instead, at all * units = 4 * shared, the further heads' parts (1 KiB and more for each
  // workgroup) are more than the shorter table of parts saves (32 B for each at most).
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
