// qmm_attention.hip -- the launch plan of attention over the paged cache, and the
// kernel that joins the splits of its keys:
//
//   out = sum_k o_k w_k / sum_k l_k w_k,  w_k = 2^(scale2 * (top_k - top))
//
// over the splits' partial results (o, top, l), in their order.
#include "qmm_attention_parts.h"
#include "qmm_internal.h"

#include <algorithm>

namespace qmm {

namespace {

template <int TYPE>
__global__ __launch_bounds__(256) void join_kernel(AttnArgs a, Batch batch, int dim) {
  const int64_t thread = (int64_t)blockIdx.x * 256 + threadIdx.x, threads = (int64_t)gridDim.x * 256;
  if (a.q8_out) zero_padding(a, dim, batch.n_tok, thread, threads);
  const int first = clamped(batch.starts[0], 0, batch.n_tok), end = clamped(batch.starts[batch.n_seq], first, batch.n_tok);
  const int per_head = dim >> 2;
  const int64_t rows = (int64_t)batch.n_tok * a.heads, items = (int64_t)(end - first) * a.heads * per_head;
  for (int64_t i = thread; i < items; i += threads) {
    const int64_t row = (int64_t)first * a.heads + i / per_head;
    const int d = 4 * (int)(i % per_head);
    float top = kNone;
    for (int k = 0; k < a.splits; ++k) top = fmaxf(top, a.sums[k * rows + row].x);
    float total = 0.0f;
    float4 x = make_float4(0, 0, 0, 0);
    for (int k = 0; k < a.splits; ++k) {
      const float2 m = a.sums[k * rows + row];
      const float by = m.x == kNone ? 0.0f : __builtin_amdgcn_exp2f((m.x - top) * a.scale2);
      const float4 v = *(const float4*)(a.part + (k * rows + row) * dim + d);
      total = fmaf(m.y, by, total);
      x.x = fmaf(v.x, by, x.x), x.y = fmaf(v.y, by, x.y), x.z = fmaf(v.z, by, x.z), x.w = fmaf(v.w, by, x.w);
    }
    const float by = total == 0.0f ? 0.0f : 1.0f / total;
    store_four<TYPE>(a, dim, (int)(row / a.heads), (int)(row % a.heads), d,
                     make_float4(x.x * by, x.y * by, x.z * by, x.w * by));
  }
}

}  // namespace

AttnPlan plan_attention(int type, int heads, int kv_heads, int dim, int64_t n_seq, int64_t n_tok, int64_t max_new,
                        int64_t max_length, int num_cus) {
  AttnPlan plan{};
  const int64_t group = heads / kv_heads, flats = std::clamp<int64_t>(max_new, 1, n_tok) * group;
  plan.few = flats <= 64;
  plan.columns = plan.few ? (int)std::min<int64_t>(flats, 32) : 128;
  plan.tiles = (int)((flats + plan.columns - 1) / plan.columns);
  // Splits: enough work-groups for the compute units, each with some tiles for every wave.
  const int64_t base = n_seq * kv_heads * plan.tiles, tiles = (max_length + kTileSlots - 1) / kTileSlots;
  const int64_t want = (2 * (int64_t)num_cus + base - 1) / base, most = tiles / (plan.few ? 16 : 32);
  plan.splits = (int)std::clamp<int64_t>(std::min(want, most), 1, 256);
  plan.work_groups = base * plan.splits;
  plan.work_bytes = plan.splits == 1 ? 0 : (size_t)plan.splits * n_tok * heads * ((size_t)dim * 4 + 8);
  return plan;
}

hipError_t launch_attention(const AttnArgs& a, const Pools& p, const Batch& b, const AttnPlan& plan, hipStream_t s) {
  const hipError_t e = (p.type == QMM_Q8    ? launch_attention_q8
                        : p.type == QMM_F16 ? launch_attention_f16
                                            : launch_attention_bf16)(a, p, b, plan, s);
  if (e != hipSuccess || plan.splits == 1) return e;
  const int64_t items = (int64_t)b.n_tok * a.heads * (p.dim / 4);
  const unsigned grid = (unsigned)std::min<int64_t>((items + 255) / 256, 1 << 16);
  if (p.type == QMM_BF16) join_kernel<QMM_BF16><<<grid, 256, 0, s>>>(a, b, p.dim);
  else join_kernel<QMM_F16><<<grid, 256, 0, s>>>(a, b, p.dim);
  return hipGetLastError();
}

}  // namespace qmm
