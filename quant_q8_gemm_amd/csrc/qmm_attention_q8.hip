// qmm_attention_q8.hip -- the attention kernels of caches that hold q8 blocks.
#include "qmm_attention_kernels.h"

namespace qmm {

hipError_t launch_attention_q8(const AttnArgs& a, const Pools& p, const Batch& b, const AttnPlan& plan, hipStream_t s) {
  return launch_type<QMM_Q8>(a, p, b, plan, s);
}

}  // namespace qmm
