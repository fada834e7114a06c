// qmm_attention.h -- the checked arguments of qmm_attention as its kernels take
// them, and its launch plan.
#pragma once

#include "qmm_cache.h"

namespace qmm {

// Division of numbers below 2^30 by a divisor of up to 2^12: with m = ceil(2^42 / d), n m 2^-42
// is past n/d by less than n 2^-42 <= 2^-12, which does not reach the next whole number.
struct Divisor {
  uint64_t m;
  Divisor(int d = 1) : m(((1ull << 42) + d - 1) / d) {}
  __host__ __device__ int of(int n) const { return (int)(((uint64_t)(uint32_t)n * m) >> 42); }
};

struct AttnArgs {
  const void* q;
  int64_t q_stride, q_head_stride;  // elements
  void* out;                        // 16-bit rows, or a qact buffer
  int64_t out_stride;
  float* part;                      // partial results [split][row * heads + head][dim], or nullptr
  float2* sums;                     // their (maximum, sum), [split][row * heads + head]
  int64_t window;                   // 0: none
  int32_t heads, group;             // heads per head of the cache
  Divisor by_group;
  int32_t causal, q8_out, splits, columns, tiles;
  int32_t share;                    // tiles of a split at least; splits * share cover max_length
  int64_t t_pad;                    // rows of the qact buffer
  float scale2;                     // scale / ln 2: the exponentials are powers of two
};

// Work-groups that a launch's tiles are given at most (but for one a sequence and head).
constexpr int64_t kMostTiles = 1 << 18;

// Plan of a launch (qmm_attention_plan).  Its work-groups are below 2^30: 65535 sequences of 4096
// heads, two tiles each, and splits only where there are few.
struct AttnPlan {
  bool few;
  int columns, tiles, splits, share, groups;
  int64_t work_groups;
  size_t work_bytes;
};
AttnPlan plan_attention(int type, int heads, int kv_heads, int dim, int64_t n_seq, int64_t n_tok, int64_t max_new,
                        int64_t max_length, int64_t window, int num_cus);

// The product kernels of one cache type (a source file each), on a checked plan;
// and the kernel that joins the splits.
typedef hipError_t AttnLaunch(const AttnArgs& a, const Pools& p, const Batch& b, const AttnPlan& plan, hipStream_t s);
AttnLaunch launch_attention_f16, launch_attention_bf16, launch_attention_q8;
hipError_t launch_attention(const AttnArgs& a, const Pools& p, const Batch& b, const AttnPlan& plan, hipStream_t s);

}  // namespace qmm
