// qmm_rope.h -- the checked arguments of qmm_rope_cache as its kernel takes them.
#pragma once

#include "qmm_cache.h"

namespace qmm {

struct Rows {
  const void* p;
  int64_t stride, head_stride;  // elements
};

struct RopeArgs {
  Rows q, q_out, k, v;
  const double* frequencies;
  const int32_t* positions;
  int32_t type, out_type, q_heads, layout, n_rot;
  float magnitude;
  int32_t q_heads_per_job, heads_per_job, q_jobs, k_jobs;  // set by the launcher
};

hipError_t launch_rope(RopeArgs r, const Pools& p, const Batch& b, int64_t max_new, hipStream_t s);
hipError_t launch_cache_read(const Pools& p, const Batch& b, int64_t max_new, int type, void* k, void* v, hipStream_t s);

}  // namespace qmm
