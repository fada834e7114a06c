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

// A work-group takes the rows (token, head) that its threads cover with dim/4 threads each
// and LANES such sets for a row, which share its splits and are joined in LDS.  Loads go out
// four splits at a time: there are few threads when this kernel matters, and a load after
// the other would be all of its time.  Latency bounds it then: 64 rows of 24 splits 5.1 us, 32 of 13
// 4.0 us; of many rows the partial results' bytes: 81920 rows of two splits 34.4 us (3.0 TB/s).
template <int TYPE, int LANES>
__global__ __launch_bounds__(256) void join_kernel(AttnArgs a, Batch batch, int dim) {
  __shared__ float4 parts[256];
  __shared__ float2 sums[256];
  if (a.q8_out)
    zero_padding(a, dim, batch.n_tok, (int64_t)blockIdx.x * 256 + threadIdx.x, (int64_t)gridDim.x * 256);
  const int first = clamped(uniform_load(batch.starts, 0), 0, batch.n_tok);
  const int end = first_row(batch, batch.n_seq);
  const int quads = dim >> 2, per_row = quads * LANES, rows_here = 256 / per_row;
  const int lane = threadIdx.x / quads % LANES, d = 4 * (threadIdx.x % quads), mine = threadIdx.x / per_row;
  const int64_t all = (int64_t)batch.n_tok * a.heads;
  for (int64_t row0 = (int64_t)first * a.heads + (int64_t)blockIdx.x * rows_here; row0 < (int64_t)end * a.heads;
       row0 += (int64_t)gridDim.x * rows_here) {
    const int64_t row = row0 + mine;
    const bool real = mine < rows_here && row < (int64_t)end * a.heads;
    float top = kNone, total = 0.0f;
    float4 x = make_float4(0, 0, 0, 0);
    if (real) {
      for (int k0 = lane; k0 < a.splits; k0 += 4 * LANES) {
        float2 m[4];
        float4 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int k = k0 + j * LANES;
          const int64_t at = (k < a.splits ? k : k0) * all + row;
          m[j] = a.sums[at];
          v[j] = *(const float4*)(a.part + at * dim + d);
          if (k >= a.splits || m[j].y == 0.0f) {  // not there, or nothing was seen in it
            m[j] = make_float2(kNone, 0.0f);
            v[j] = make_float4(0, 0, 0, 0);
          }
        }
        const float now = fmaxf(fmaxf(fmaxf(m[0].x, m[1].x), fmaxf(m[2].x, m[3].x)), top);
        const float4 so_far = x;
        const float sum = total;
        x = make_float4(0, 0, 0, 0), total = 0.0f;
        add_part(x, total, so_far, top, sum, now, a.scale2);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          add_part(x, total, v[j], m[j].x, m[j].y, now, a.scale2);
        top = now;
      }
    }
    if (LANES > 1) {
      parts[threadIdx.x] = x;
      sums[threadIdx.x] = make_float2(top, total);
      __syncthreads();
      if (real && lane == 0) {
        float now = top;
#pragma unroll
        for (int l = 1; l < LANES; ++l) now = fmaxf(now, sums[threadIdx.x + l * quads].x);
        x = make_float4(0, 0, 0, 0), total = 0.0f;
#pragma unroll
        for (int l = 0; l < LANES; ++l) {
          const float2 m = sums[threadIdx.x + l * quads];
          add_part(x, total, parts[threadIdx.x + l * quads], m.x, m.y, now, a.scale2);
        }
      }
    }
    if (real && lane == 0) {
      store_four<TYPE>(a, dim, (int)(row / a.heads), (int)(row % a.heads), d, divided(x, total));
    }
    if (LANES > 1) __syncthreads();
  }
}

template <int TYPE, int LANES>
hipError_t launch_join(const AttnArgs& a, const Pools& p, const Batch& b, hipStream_t s) {
  const int rows_here = 256 / (p.dim / 4 * LANES);
  const int64_t blocks = ((int64_t)b.n_tok * a.heads + rows_here - 1) / rows_here;
  join_kernel<TYPE, LANES><<<(unsigned)std::min<int64_t>(blocks, 1 << 16), 256, 0, s>>>(a, b, p.dim);
  return hipGetLastError();
}

}  // namespace

AttnPlan plan_attention(int type, int heads, int kv_heads, int dim, int64_t n_seq, int64_t n_tok, int64_t max_new,
                        int64_t max_length, int64_t window, int num_cus) {
  AttnPlan plan{};
  const int64_t group = heads / kv_heads, flats = std::clamp<int64_t>(max_new, 1, n_tok) * group;
  plan.few = flats <= 64;
  plan.columns = plan.few ? (int)std::min<int64_t>(flats, 32) : 128;
  plan.tiles = (int)((flats + plan.columns - 1) / plan.columns);
  // Work-groups without columns end at once, but thousands of sequences with max_new unknown would
  // have millions of them, for some milliseconds: fewer take turns over a sequence's tiles then.
  plan.tiles = (int)std::min<int64_t>(plan.tiles, std::max<int64_t>(kMostTiles / (n_seq * kv_heads), plan.few ? 2 : 1));
  // the most tiles of 32 slots that a tile of columns reads
  int64_t keys = max_length;
  if (window > 0 && window < keys) keys = std::min(keys, window + plan.columns / group + kTileSlots);  // 2^63 - 1 is a window too
  const int64_t tiles = std::max<int64_t>((keys + kTileSlots - 1) / kTileSlots, 1);
  // work-groups of a split, and how many of them have columns at most: sequences with fewer
  // tokens than max_new leave some without
  const int64_t grid = n_seq * kv_heads * plan.tiles, slots = 2 * (int64_t)num_cus;
  const int64_t base = std::min(grid, kv_heads * (n_tok * group / plan.columns + n_seq));
  // The number of splits that needs the least time, in microseconds: rounds of work-groups over
  // the GPU, each with a start and its share's tiles, and for more than one split the join
  // and the partial results' way through memory.  A tile takes a work-group of many columns
  // about 1 us, or 0.6 with two groups of waves, and of heads past 128 by as much more; one of few
  // what the active ones' tiles take from memory, 0.3 at least.  Measured:
  // one token of 32 heads over 3314 slots with 1, 4, 16 splits 21.6, 15.9, 16.5 us; 16 sequences of
  // 20 heads of 64 over up to 1500 with 1, 2, 4: 15.4, 17.8, 19.7; one token of 64/8 heads over 131072
  // with 8, 16, 32: 167, 109, 106; 2048 tokens of 40/8 heads over 32768 with 1, 2, 4: 1605, 1339, 1301;
  // 100 tokens of 16/4 heads over 3000 in q8 with 1, 2, 4, 8, 16: 65.1, 40.8, 29.2, 25.9, 26.3, of 256
  // 196, 106, 62, 46, 41.
  const double start = plan.few ? 3.0 : 8.0, join = plan.few ? 4.5 : 10.0, partial_mb = (double)n_tok * heads * dim * 8e-6;
  const int64_t least = plan.few ? 4 : 8, unit = plan.few ? 4 : 2;
  int64_t share = tiles;
  double best = 0.0;
  for (int64_t n = 1; n <= 256 && (n == 1 || (tiles / n >= least && grid < 16 * slots)); n += n < 16 ? 1 : n / 8) {
    const int64_t each = ((tiles + n - 1) / n + unit - 1) / unit * unit, rounds = (base * n + slots - 1) / slots;
    const double active = (double)std::clamp<int64_t>(base * n, 192, slots);  // fewer do not take all of the bandwidth
    const double tile = plan.few ? std::max(0.3, active * 2.0 * tile_bytes(type, dim) / 5e6)
                                 : (base * n > num_cus ? 1.0 : 0.6) * std::max(dim / 128.0, 1.0);
    const double cost = (double)rounds * ((double)each * tile + start) + (n > 1 ? join + partial_mb * (double)n / 4.0 : 0.0);
    if (n == 1 || cost < 0.97 * best) best = cost, share = each;
  }
  share = std::max(share, (tiles + 255) / 256);
  plan.splits = (int)((tiles + share - 1) / share);
  plan.share = (int)share;
  plan.work_groups = grid * plan.splits;
  plan.groups = !plan.few && base * plan.splits <= num_cus ? 2 : 1;
  plan.work_bytes = plan.splits == 1 ? 0 : (size_t)plan.splits * n_tok * heads * ((size_t)dim * 4 + 8);
  return plan;
}

hipError_t launch_attention(const AttnArgs& a, const Pools& p, const Batch& b, const AttnPlan& plan, hipStream_t s) {
  const hipError_t e = (p.type == QMM_Q8    ? launch_attention_q8
                        : p.type == QMM_F16 ? launch_attention_f16
                                            : launch_attention_bf16)(a, p, b, plan, s);
  if (e != hipSuccess || plan.splits == 1) return e;
  // four splits in flight for each thread, as far as a row's threads go
  const bool wide = plan.splits > 4;
  if (p.type == QMM_BF16) return (wide ? launch_join<QMM_BF16, 4> : launch_join<QMM_BF16, 1>)(a, p, b, s);
  return (wide ? launch_join<QMM_F16, 4> : launch_join<QMM_F16, 1>)(a, p, b, s);
}

}  // namespace qmm
