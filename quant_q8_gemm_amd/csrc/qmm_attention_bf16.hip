// qmm_attention_bf16.hip -- the attention kernels of caches that hold bf16.
#include "qmm_attention_kernels.h"

namespace qmm {

hipError_t launch_attention_bf16(const AttnArgs& a, const Pools& p, const Batch& b, const AttnPlan& plan, hipStream_t s) {
  return launch_type<QMM_BF16>(a, p, b, plan, s);
}

}  // namespace qmm
