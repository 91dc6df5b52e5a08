// Attention over a paged cache of type f32 (the kernels are in kda_paged_decode.h).
#include "kda_paged_decode.h"

namespace kda {

hipError_t launch_paged_decode_f32(const PagedDecodePlan& p, hipStream_t stream) {
  return paged::launch_cache<kF32>(p, stream);
}

}  // namespace kda
