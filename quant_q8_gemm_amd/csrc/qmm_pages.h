// qmm_pages.h -- where the attention kernels find a sequence's tiles; compiled for the host too, where it is
// tested.
#pragma once

#include "qmm_cache.h"
#if defined(__HIP_DEVICE_COMPILE__)
#include "qmm_common.h"
#endif

namespace qmm {

// 64 columns of a row of the table: on the GPU in a register of the wave, a column a lane; a
// lookup is then a v_readlane, where a load would be waited for with every tile.
struct Columns {
#if defined(__HIP_DEVICE_COMPILE__)
  int32_t held;
  __device__ __forceinline__ void fetch(const int32_t* row, int columns, int base) {
    held = row[min(base + (int)(threadIdx.x & 63), columns - 1)];
  }
  __device__ __forceinline__ void wait() { pin(held); }
  __device__ __forceinline__ uint32_t at(int i) const { return (uint32_t)__builtin_amdgcn_readlane(held, i); }
#else
  int32_t held[64];
  void fetch(const int32_t* row, int columns, int base) {
    for (int i = 0; i < 64; ++i) held[i] = row[base + i < columns ? base + i : columns - 1];
  }
  void wait() {}
  uint32_t at(int i) const { return (uint32_t)held[i]; }
#endif
};

struct Pages {
  const int32_t* row;
  int columns, base, shift, n_pages, tile;
  Columns held;
  int64_t page, head;  // bytes of a page, and to the head in it
  // (before anything else of a kernel, so that the columns are there when the lengths are)
  __host__ __device__ inline __attribute__((always_inline)) Pages(const Batch& b, const Pools& p, int s, int h)
      : row(b.table + s * b.table_stride), columns(b.columns), base(0), shift(p.page_shift - 5), n_pages(p.n_pages) {
    held.fetch(row, columns, 0);
    tile = tile_bytes(p.type, p.dim);
    head = (int64_t)tile * (h << shift);
    page = (int64_t)tile * (p.heads << shift);
  }
  // Tile t's place in both pools, or -1; t is the same in every lane, from 0 on, and the sequence's
  // tiles (end and those before it) have a column.
  __host__ __device__ inline __attribute__((always_inline)) int64_t place(int t, int end) {
    if (t >= end) return -1;
    const int i = t >> shift;
    if ((unsigned)(i - base) >= 64u) {
      base = i;
      held.fetch(row, columns, i);
      held.wait();  // here, and not where lookups without a load come by
    }
    const uint32_t at = held.at(i - base);
    if (at >= (uint32_t)n_pages) return -1;
    return head + (int64_t)((uint64_t)at * (uint64_t)page) + (uint32_t)((t & ((1 << shift) - 1)) * tile);
  }
};

// Where the tiles of a stage are.
template <int KB>
struct Places {
  int64_t at[KB];
  // t is a multiple of KB: two tiles are on one page but for pages of 32 slots
  __host__ __device__ inline __attribute__((always_inline)) void find(Pages& pages, int t, int end) {
    at[0] = pages.place(t, end);
    if (KB > 1) at[KB - 1] = pages.shift == 0 ? pages.place(t + 1, end) : t + 1 < end && at[0] >= 0 ? at[0] + pages.tile : -1;
  }
  // a bit for each tile that is somewhere
  __host__ __device__ inline __attribute__((always_inline)) uint32_t here() const {
    uint32_t r = 0;
#pragma unroll
    for (int k = 0; k < KB; ++k) r |= (uint32_t)(at[k] >= 0) << k;
    return r;
  }
};

}  // namespace qmm
