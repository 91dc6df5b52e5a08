// Linear attention with a decay for each head, over whole prompts.
#include "kda_lin.h"

namespace kda {

size_t plan_lin_chunk(LinPlan* p) {
  p->seg = p->T;
  p->jobs = p->n_seq;
  return 0;
}

hipError_t launch_lin_chunk(const LinPlan& p, hipStream_t stream) { return launch_lin_recurrent(p, stream); }

}  // namespace kda
