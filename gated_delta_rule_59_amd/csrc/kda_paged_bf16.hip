// Attention over a paged cache of type bf16 (the kernels are in kda_paged_decode.h).
#include "kda_paged_decode.h"

namespace kda {

hipError_t launch_paged_decode_bf16(const PagedDecodePlan& p, hipStream_t stream) {
  return paged::launch_cache<kBF16>(p, stream);
}

}  // namespace kda
