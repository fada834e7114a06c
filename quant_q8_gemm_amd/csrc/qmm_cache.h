// qmm_cache.h -- where the paged cache keeps what, and which rows and slots a
// sequence of a batch has: shared by the kernels that write and read it, and
// compiled for the host too, where its bounds are tested.
//
// A head's 32 slots form a tile in the order in which the matrix instructions'
// left operand (32 rows by 16, eight values a lane) wants it: keys with slots as
// rows, values with channels as rows and slots along the sum.  One 16-byte load a
// lane then moves a whole operand of 1 KiB, with nothing to transpose between
// memory and the matrix core.  The keys' rows are slots with bits 2 and 3
// exchanged, so that the scores leave the first product as a lane's eight
// consecutive slots, which is how the second one wants its right operand.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/qmm.h"

namespace qmm {

constexpr int kTileSlots = 32;

__host__ __device__ constexpr int tile_bytes(int type, int dim) { return type == QMM_Q8 ? 34 * dim : 64 * dim; }

__host__ __device__ constexpr int key_row(int r) { return (r & ~12) | ((r & 4) << 1) | ((r & 8) >> 1); }

// Element (16 bits) or byte (q8) of slot r and channel d in a tile.
__host__ __device__ constexpr int key_at(int r, int d) {
  return (((d >> 4) * 2 + ((d >> 3) & 1)) * 32 + key_row(r)) * 8 + (d & 7);
}
__host__ __device__ constexpr int value_at(int r, int d) { return (((d >> 5) * 4 + (r >> 3)) * 32 + (d & 31)) * 8 + (r & 7); }
__host__ __device__ constexpr int key_code_at(int r, int d) {
  return (d >> 5) * 1024 + (((d >> 3) & 1) * 32 + key_row(r)) * 16 + ((d >> 4) & 1) * 8 + (d & 7);
}
__host__ __device__ constexpr int value_code_at(int r, int d) {
  return (d >> 5) * 1024 + (((r >> 3) & 1) * 32 + (d & 31)) * 16 + (r >> 4) * 8 + (r & 7);
}
// Byte of the scale of block d/32 of slot r.
__host__ __device__ constexpr int scale_at(int dim, int r, int block) { return 32 * dim + (block * 32 + r) * 2; }

// The sequences of a call as the kernels take them (qmm_batch, checked).
struct Batch {
  const int32_t* starts;
  const int32_t* lengths;
  const int32_t* table;
  int64_t table_stride;
  int32_t n_seq, columns, n_tok;
};

// The pools of a call; a page is 1 << page_shift slots.
struct Pools {
  uint8_t *k, *v;
  int32_t heads, dim, page_shift, type;
  int32_t n_pages;
};

// A sequence: its rows [first, first + count) and slots [0, length).  Whatever the
// arrays hold, the rows are rows of the call and the slots have a column.
struct Sequence {
  int first, count, length;
};

__host__ __device__ inline int clamped(int v, int low, int high) { return v < low ? low : v > high ? high : v; }

// One of the batch's numbers, at an index that is the same in every lane.  On the GPU a
// scalar load: a vector load's wait would be one for every load before it, those of
// the tiles ahead among them.
__host__ __device__ inline int32_t uniform_load(const int32_t* p, int64_t i) {
#if defined(__HIP_DEVICE_COMPILE__)
  return ((const __attribute__((address_space(4))) int32_t*)(uintptr_t)p)[i];
#else
  return p[i];
#endif
}

// The row that sequence s begins at: the highest start up to its own, so that starts which go
// down give no row to two sequences.  All lanes of a wave call it with the same s.  Starts that are
// in order cost a load of the earlier ones and a comparison: of 64 by one load, issued before
// anything is waited for (24 chunks into q8, with the cache read back: 23.1 us without it, 24.1 behind the
// scalar loads, 23.4 so), of more by four of 256 in flight.  One token each of n sequences of up to 64 slots, 16/4 heads
// of 64: n = 1024 35.6 us without it and 38.1 with it, 4096 141 and 164, 16384 539 and 819; 400 of up to
// 2000 slots 95.7 and 96.5.
__host__ __device__ inline int first_row(const Batch& b, int s) {
#if defined(__HIP_DEVICE_COMPILE__)
  int earlier = INT32_MIN;
  if (s > 0) earlier = b.starts[min((int)(threadIdx.x & 63), s - 1)];
  const int own = clamped(uniform_load(b.starts, s), 0, b.n_tok);
  if (s > 64) {
    typedef int32_t v4 __attribute__((ext_vector_type(4), aligned(4)));
    v4 most = {earlier, earlier, earlier, earlier};
    for (int i = 64; i < s; i += 1024) {
#pragma unroll
      for (int j = 0; j < 1024; j += 256) {
        const v4 x = *(const v4*)(b.starts + min(i + j + 4 * (int)(threadIdx.x & 63), s - 4));
#pragma unroll
        for (int k = 0; k < 4; ++k) most[k] = max(most[k], x[k]);
      }
    }
    earlier = max(max(most[0], most[1]), max(most[2], most[3]));
  }
  if (!__any(earlier > own)) return own;
  for (int step = 32; step > 0; step >>= 1) earlier = max(earlier, __shfl_xor(earlier, step));
  return clamped(__builtin_amdgcn_readfirstlane(earlier), own, b.n_tok);
#else
  int top = clamped(b.starts[s], 0, b.n_tok);
  for (int i = 0; i < s; ++i) top = clamped(b.starts[i], top, b.n_tok);
  return top;
#endif
}

__host__ __device__ inline Sequence sequence(const Batch& b, int page_shift, int s) {
  const int length = clamped(uniform_load(b.lengths, s), 0, b.columns << page_shift), next = uniform_load(b.starts, s + 1);
  const int first = first_row(b, s);
  return {first, clamped(next, first, b.n_tok) - first, length};
}

// Byte offset in a pool of the tile of head h that holds slots 32*tile .. on `page`; -1 where
// the page is none of the pool's.
__host__ __device__ inline int64_t offset_on_page(const Pools& p, int page, int h, int tile) {
  const int tiles_shift = p.page_shift - 5;
  if (page < 0 || page >= p.n_pages) return -1;
  const int64_t at = (((int64_t)page * p.heads + h) << tiles_shift) + (tile & ((1 << tiles_shift) - 1));
  return at * tile_bytes(p.type, p.dim);
}

// The same by the table, of sequence s; 0 <= 32*tile < columns * page.  UNIFORM: s and tile
// are the same in every lane.
template <bool UNIFORM = false>
__host__ __device__ inline int64_t tile_offset(const Batch& b, const Pools& p, int s, int h, int tile) {
  const int64_t i = s * b.table_stride + (tile >> (p.page_shift - 5));
  return offset_on_page(p, UNIFORM ? uniform_load(b.table, i) : b.table[i], h, tile);
}

}  // namespace qmm
