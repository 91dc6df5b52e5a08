// Attention over a paged cache of type e4m3 (the kernels are in kda_paged_decode.h).
#include "kda_paged_decode.h"

namespace kda {

hipError_t launch_paged_decode_e4m3(const PagedDecodePlan& p, hipStream_t stream) {
  return paged::launch_cache<kF8>(p, stream);
}

}  // namespace kda
