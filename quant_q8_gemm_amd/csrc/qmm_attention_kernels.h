// qmm_attention_kernels.h -- attention over the paged cache: the kernel for few
// columns (decode steps) and the kernel for many (chunks and prompts), instantiated
// per cache type in a source file each.
#pragma once

#include "qmm_attention_parts.h"
#include "qmm_internal.h"
#include "qmm_pages.h"

namespace qmm {

namespace {

// ---- few columns ----
//
// The cache's bytes bound it.  The waves of a work-group take turns over a split's
// 32-slot tiles, each with a running softmax of its own, straight from memory into the
// operands' registers: a tile's keys and values are on their way while the one before
// is worked on.  The waves' results are joined in LDS, the splits' by a second kernel.
// Measured: one token of 64/8 heads of 128 over 131072 bf16 slots 91.4 us (5.9 TB/s); of 32/32 over
// 3314 f16 slots 12.6 us (4.3 TB/s); 32 sequences of up to 8192 q8 slots, 32/8 heads, 78.3 us (4.2 TB/s;
// of 8192 each 5.2).

// A tile's keys or values as loaded.
template <int TYPE, int DB>
struct Loaded {
  typedef typename Math<TYPE>::v8 v8;
  v8 f[2 * DB];
  __device__ __forceinline__ void load(const uint8_t* tile, int lane) {
#pragma unroll
    for (int i = 0; i < 2 * DB; ++i) f[i] = *(const v8*)(tile + i * 1024 + lane * 16);
  }
  __device__ __forceinline__ void load_keys(const uint8_t* tile, int lane) { load(tile, lane); }
  __device__ __forceinline__ void load_values(const uint8_t* tile, int lane) { load(tile, lane); }
  __device__ __forceinline__ void clean() {
#pragma unroll
    for (int i = 0; i < 2 * DB; ++i) f[i] = finite<TYPE>(f[i]);
  }
  __device__ __forceinline__ v8 key(int i) const { return f[i]; }
  __device__ __forceinline__ v8 value(int i) const { return f[i]; }
};
template <int DB>
struct Loaded<QMM_Q8, DB> {
  v4i w[DB];
  _Float16 k[DB];      // keys: the scales of this lane's slot
  f16x8 v[2 * DB];     // values: of the eight slots of each step
  __device__ __forceinline__ void load(const uint8_t* tile, int lane) {
#pragma unroll
    for (int i = 0; i < DB; ++i) w[i] = *(const v4i*)(tile + i * 1024 + lane * 16);
  }
  __device__ __forceinline__ void load_keys(const uint8_t* tile, int lane) {
    load(tile, lane);
    const int r = key_row(lane & 31);  // its own inverse
#pragma unroll
    for (int i = 0; i < DB; ++i) k[i] = *(const _Float16*)(tile + scale_at(32 * DB, r, i));
  }
  __device__ __forceinline__ void load_values(const uint8_t* tile, int lane) {
    load(tile, lane);
#pragma unroll
    for (int i = 0; i < 2 * DB; ++i)
      v[i] = *(const f16x8*)(tile + scale_at(32 * DB, 16 * (i & 1) + 8 * (lane >> 5), i >> 1));
  }
  __device__ __forceinline__ f16x8 codes(int i, const f16x8& s) const {
    return (i & 1) ? codes8(w[i >> 1].z, w[i >> 1].w, s) : codes8(w[i >> 1].x, w[i >> 1].y, s);
  }
  // A scale that is no finite number becomes zero, and with a finite one the codes whose
  // product with it is none: leftovers of a pool may be any bits.
  __device__ __forceinline__ void clean() {
#pragma unroll
    for (int i = 0; i < 2 * DB; ++i) {
      const u16x8 u = __builtin_bit_cast(u16x8, codes(i, v[i]));
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int four = 2 * (i & 1) + (j >> 2), shift = 8 * (j & 3);
        if ((u[j] & 0x7c00) == 0x7c00) w[i >> 1][four] = (w[i >> 1][four] & ~(255 << shift)) | (128 << shift);
      }
      v[i] = finite<QMM_Q8>(v[i]);
    }
  }
  __device__ __forceinline__ f16x8 key(int i) const { return codes(i, splat8(k[i >> 1])); }
  __device__ __forceinline__ f16x8 value(int i) const { return codes(i, v[i]); }
};

template <int TYPE, int DB, int WAVES>
__global__ __launch_bounds__(64 * WAVES) __attribute__((amdgpu_waves_per_eu(DB <= 4 ? 2 : 1, DB <= 4 ? 2 : 1))) void few_kernel(
    AttnArgs a, Pools pools, Batch batch) {
  constexpr int kDim = 32 * DB, kRow = kDim + 4;
  extern __shared__ float lds[];
  typedef typename Math<TYPE>::v8 v8;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, half = lane >> 5;
  const int h = blockIdx.x % pools.heads, rest = blockIdx.x / pools.heads, split = rest % a.splits, s = blockIdx.y;
  if (a.q8_out && a.splits == 1)
    zero_padding(a, kDim, batch.n_tok, ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * blockDim.x + threadIdx.x,
                 (int64_t)gridDim.x * gridDim.y * blockDim.x);
  Pages pages(batch, pools, s, h);
  const Sequence seq = sequence(batch, pools.page_shift, s);
  const int flats = seq.count * a.group;
  float* const tops = lds;                    // [WAVES][32]
  float* const sums = lds + WAVES * 32;       // [WAVES][32]
  float* const parts = lds + 2 * WAVES * 32;  // [WAVES][columns][kRow]

  for (int tile = rest / a.splits; (int64_t)tile * a.columns < flats; tile += a.tiles) {
    const int first = tile * a.columns, last = min(first + a.columns, flats) - 1;
    const Column c = column(a, seq, h, first + min(lane & 31, a.columns - 1));
    int low, high, all_low, all_high, unused;
    seen(a, seq, a.by_group.of(first), a.by_group.of(last), low, high);
    seen(a, seq, a.by_group.of(first), a.by_group.of(first), unused, all_high);
    seen(a, seq, a.by_group.of(last), a.by_group.of(last), all_low, unused);
    const int begin = low >> 5, tiles = max(0, ((high + 31) >> 5) - begin), share = max(a.share, (tiles + a.splits - 1) / a.splits);
    const int from = begin + split * share, end = min(begin + tiles, from + share);
    if (split > 0 && from >= end) {  // nothing left for this split
      no_part(a, seq, batch.n_tok, h, split, first, last);
      continue;
    }

    for (bool safe = false;; safe = true) {
      // A tile's loads are issued whether it is there or not (the pool's first instead, which
      // then counts for nothing): behind a branch the wait for one tile would be one for
      // the next as well.
      Loaded<TYPE, DB> keys, values;
      int t = from + wave;
      int64_t at = pages.place(t, end), next = pages.place(t + WAVES, end);
      keys.load_keys(pools.k + max(at, (int64_t)0), lane);
      values.load_values(pools.v + max(at, (int64_t)0), lane);
      v8 q[2 * DB];
      load_queries<TYPE, DB>(a, c, lane, q);
#pragma unroll
      for (int i = 0; i < 2 * DB; ++i) pin(q[i]);
      v16f o[DB];
#pragma unroll
      for (int d = 0; d < DB; ++d) o[d] = v16f{};
      Running run;
      for (; t < end; t += WAVES) {
        const bool here = at >= 0;
        at = next;
        next = pages.place(t + 2 * WAVES, end);
        v16f score[1] = {v16f{}};
#pragma unroll
        for (int i = 0; i < 2 * DB; ++i) score[0] = Math<TYPE>::mma(keys.key(i), q[i], score[0]);
        keys.load_keys(pools.k + max(at, (int64_t)0), lane);
        const int slot0 = 32 * t;
        const bool inside = here && slot0 >= all_low && slot0 + 32 <= all_high;
        if (!inside) hide(score[0], slot0, half, c.low, here ? c.high : 0);
        v8 p[2];
        soften<TYPE, DB, 1>(score, a.scale2, run, o, p);
        if (safe && !inside) values.clean();
#pragma unroll
        for (int i = 0; i < 2 * DB; ++i) o[i >> 1] = Math<TYPE>::mma(values.value(i), p[i & 1], o[i >> 1]);
        values.load_values(pools.v + max(at, (int64_t)0), lane);
      }

      const float sum = both_sum(run.sum);
      if (lane < a.columns && lane < 32) tops[wave * 32 + lane] = run.top, sums[wave * 32 + lane] = sum;
      if ((lane & 31) < a.columns) {
        float* const to = parts + (wave * a.columns + (lane & 31)) * kRow + 4 * half;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *(float4*)(to + 32 * d + 8 * i) = make_float4(o[d][4 * i], o[d][4 * i + 1], o[d][4 * i + 2], o[d][4 * i + 3]);
      }
      __syncthreads();
      bool odd = false;
      for (int i = threadIdx.x; i < a.columns * (kDim / 4); i += 64 * WAVES) {
        const int n = i / (kDim / 4), d = 4 * (i % (kDim / 4));
        const Column to = column(a, seq, h, first + n);
        if (!to.real) continue;
        float top = tops[n];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) top = fmaxf(top, tops[w * 32 + n]);
        float total = 0.0f;
        float4 x = make_float4(0, 0, 0, 0);
#pragma unroll
        for (int w = 0; w < WAVES; ++w)
          add_part(x, total, *(const float4*)(parts + (w * a.columns + n) * kRow + d), tops[w * 32 + n], sums[w * 32 + n], top,
                   a.scale2);
        odd |= !(fabsf(x.x + x.y) + fabsf(x.z + x.w) < __builtin_inff());
        if (safe) add_edges<TYPE>(pools, batch, s, h, {from, end, all_low, all_high}, to, d, x);
        store_part<TYPE>(a, kDim, batch.n_tok, split, to, d, x, top, total);
      }
      // again, safely, where a result is no finite number (a barrier that the next round needs too)
      if (!__syncthreads_or(odd) || safe) break;
    }
  }
}

// ---- many columns ----
//
// The matrix core and the softmax's vector instructions bound it.  A work-group's four
// waves take 32 columns each and share the keys and values, which pass through LDS
// in a ring of stages of 32*KB slots: while one is worked on the next are copied, 16-bit tiles
// straight from memory to LDS, q8 tiles through registers, where they become f16 once for
// all waves.  Where there is at most one work-group for a compute unit it has two groups of
// four waves, which take turns over the keys with stages of their own: a wave of a
// SIMD by itself leaves it idle for half of the time (scores, powers and the second product
// of a tile wait for each other), and a second one fills that.
// Measured: 2048 tokens of 40/8 heads of 128 over 32768 bf16 slots 1,262 us (1.05 PFLOP/s, the matrix core
// busy for 54% of the cycles; the softmax's vector instructions add to its time); a prompt of 4096 of
// 32/8 heads of 256 in f16 278 us (0.99), of 3314 of 32/32 of 128 115 us (0.79); with two groups
// 4 x 448 tokens over 1501 states, 16 heads of 96, 36.5 -> 31 us.

// N consecutive 1 KiB copies from base + 16*lane to LDS; M0 is set by each run itself, and
// nothing else in these kernels reads it.
template <int N>
__device__ __forceinline__ void copy_run(const void* base, uint32_t lane_off, uint32_t lds) {
  static_assert(N >= 1 && N <= 4, "13-bit offsets");
  if constexpr (N == 1)
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(lane_off), "s"(base), "s"(lds)
                 : "memory");
  else if constexpr (N == 2)
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1\n\t"
                 "global_load_lds_dwordx4 %0, %1 offset:1024" ::"v"(lane_off), "s"(base), "s"(lds)
                 : "memory");
  else if constexpr (N == 3)
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1\n\t"
                 "global_load_lds_dwordx4 %0, %1 offset:1024\n\tglobal_load_lds_dwordx4 %0, %1 offset:2048" ::"v"(lane_off),
                 "s"(base), "s"(lds)
                 : "memory");
  else
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1\n\t"
                 "global_load_lds_dwordx4 %0, %1 offset:1024\n\tglobal_load_lds_dwordx4 %0, %1 offset:2048\n\t"
                 "global_load_lds_dwordx4 %0, %1 offset:%3" ::"v"(lane_off), "s"(base), "s"(lds), "n"(3 * 1024)
                 : "memory");
}

template <int N>
__device__ __forceinline__ void copy_kib(const uint8_t* base, uint32_t lane_off, uint32_t lds) {
  if constexpr (N > 4) {
    copy_run<4>(base, lane_off, lds);
    copy_kib<N - 4>(base + 4096, lane_off, lds + 4096);
  } else {
    copy_run<N>(base, lane_off, lds);
  }
}

// N products whose left operands come from LDS (1 KiB each, at(i) bytes from base), step by
// step: while G of them run the next G operands are on their way.  The scheduling
// barriers keep that order; by itself the compiler reads each operand right before its
// product, which then waits for it.
template <class V, int N, int G, class At, class Mma>
__device__ __forceinline__ void products(const uint8_t* base, At&& at, Mma&& mma) {
  static_assert(N % G == 0, "whole groups");
  V buffer[2][G];
#pragma unroll
  for (int j = 0; j < G; ++j) buffer[0][j] = *(const V*)(base + at(j));
#pragma unroll
  for (int g = 0; g < N / G; ++g) {
    if (g + 1 < N / G) {
#pragma unroll
      for (int j = 0; j < G; ++j) buffer[(g + 1) & 1][j] = *(const V*)(base + at((g + 1) * G + j));
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < G; ++j) mma(g * G + j, buffer[g & 1][j]);
    __builtin_amdgcn_sched_barrier(0);
  }
}

// What the lanes of a wave have written to LDS is there for all of them.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Waits until at most N of the wave's loads are on their way: the copies to LDS, which the
// compiler does not count.
template <int N>
__device__ __forceinline__ void wait_loads() {
  static_assert(N >= 0 && N < 64, "a 6-bit count");
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// A wave's part of staging: waves 0 and 1 the keys, 2 and 3 the values; of two tiles one
// each, of one tile half each.
template <int TYPE, int DB, int KB>
struct Stager {
  static constexpr int kLoads = KB * DB;  // of a stage, for each wave
  static __device__ __forceinline__ int64_t from(const Places<KB>& at, int wave) {
    const int64_t first = at.at[0], second = at.at[KB - 1];
    return KB == 2 && (wave & 1) ? second : first;
  }
  // a tile that is nowhere: the pool's first, whose numbers are then not used
  __device__ __forceinline__ void load(const Pools& p, const Places<KB>& at, int wave, int lane, uint8_t* lds) {
    const int64_t off = from(at, wave);
    const uint8_t* const base = (const uint8_t*)uniform_ptr((wave < 2 ? p.k : p.v) + (off < 0 ? 0 : off) +
                                                            (KB == 1 && (wave & 1) ? DB * 1024 : 0));
    // the stage: keys of tile 0, of tile 1, values of tile 0, of tile 1
    const uint32_t to = __builtin_amdgcn_readfirstlane(
        (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)(lds + wave * (KB * DB * 1024)));
    copy_kib<KB * DB>(base, lane * 16, to);
  }
  __device__ __forceinline__ void store(int, int, uint8_t*) {}
};
template <int DB, int KB>
struct Stager<QMM_Q8, DB, KB> {
  static constexpr int kLoads = 0;
  static constexpr int kBlocks = KB == 2 ? DB : DB / 2;  // blocks of 32 channels of a tile
  v4i w[kBlocks];
  f16x8 s[2 * kBlocks];
  __device__ __forceinline__ void load(const Pools& p, const Places<KB>& at, int wave, int lane, uint8_t*) {
    const int64_t off = Stager<QMM_F16, DB, KB>::from(at, wave);
    const uint8_t* const tile = (wave < 2 ? p.k : p.v) + (off < 0 ? 0 : off);
    const int block0 = KB == 1 && (wave & 1) ? kBlocks : 0;
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) w[i] = *(const v4i*)(tile + (block0 + i) * 1024 + lane * 16);
    if (wave < 2) {
      const int r = key_row(lane & 31);
#pragma unroll
      for (int i = 0; i < kBlocks; ++i)
        s[2 * i] = s[2 * i + 1] = splat8(*(const _Float16*)(tile + scale_at(32 * DB, r, block0 + i)));
    } else {
#pragma unroll
      for (int i = 0; i < 2 * kBlocks; ++i)
        s[i] = *(const f16x8*)(tile + scale_at(32 * DB, 16 * (i & 1) + 8 * (lane >> 5), block0 + (i >> 1)));
    }
  }
  __device__ __forceinline__ void store(int wave, int lane, uint8_t* lds) {
    uint8_t* const to = lds + wave * (KB * DB * 1024) + lane * 16;
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) {
      *(f16x8*)(to + 2 * i * 1024) = codes8(w[i].x, w[i].y, s[2 * i]);
      *(f16x8*)(to + (2 * i + 1) * 1024) = codes8(w[i].z, w[i].w, s[2 * i + 1]);
    }
  }
};

// A column's result from the lane's accumulators: 16 of each 32 channels, four in a row,
// the others in the lane of the other half.
template <int TYPE, int DB>
__device__ __forceinline__ void store_column(const AttnArgs& a, const Column& c, int split, int n_tok, int half, float top,
                                             float total, const v16f (&o)[DB]) {
  constexpr int kDim = 32 * DB, T = TYPE == QMM_BF16 ? QMM_BF16 : QMM_F16;
  if (!a.q8_out || a.splits > 1) {
    if (!c.real) return;
    if (a.splits > 1) {
#pragma unroll
      for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          store_part<TYPE>(a, kDim, n_tok, split, c, 32 * d + 8 * i + 4 * half,
                           make_float4(o[d][4 * i], o[d][4 * i + 1], o[d][4 * i + 2], o[d][4 * i + 3]), top, total);
      return;
    }
    const int64_t to = c.row * a.out_stride + (int64_t)c.head * kDim + 4 * half;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        store4<T>(a.out, to + 32 * d + 8 * i,
                  divided(make_float4(o[d][4 * i], o[d][4 * i + 1], o[d][4 * i + 2], o[d][4 * i + 3]), total));
    return;
  }
  const int64_t id = (int64_t)a.heads * kDim;
#pragma unroll
  for (int d = 0; d < DB; ++d) {
    float largest = 0.0f;
    float4 x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = divided(make_float4(o[d][4 * i], o[d][4 * i + 1], o[d][4 * i + 2], o[d][4 * i + 3]), total);
      largest = larger(larger(largest, larger(x[i].x, x[i].y)), larger(x[i].z, x[i].w));
    }
    const Halves both = halves(largest);
    const Q8Scale sc(larger(both.a, both.b));
    const int64_t block = (int64_t)(c.row >> 5) * (id >> 5) + c.head * DB + d;
    uint8_t* const to = (uint8_t*)a.out + block * 1024 + (c.row & 31) * 16 + 4 * half;
    int S = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      int q[4];
      quant4(x[i], sc.dhf, sc.inv, q);
      S += q[0] + q[1] + q[2] + q[3];
      if (c.real) *(uint32_t*)(to + (i >> 1) * 512 + (i & 1) * 8) = pack4(q);
    }
    S += __shfl_xor(S, 32);
    if (c.real && half == 0) *(uint32_t*)((uint8_t*)a.out + a.t_pad * id + block * 128 + (c.row & 31) * 4) = sc.pair(S);
  }
}

// Two waves a SIMD, but for q8 heads of 256: their accumulators, queries and the tile on its way
// from q8 to f16 need more than 256 registers (a prompt of 4096, 32/8 heads: 568 us so, 675 with two
// waves that reload some in every step).
constexpr bool alone(int type, int db) { return type == QMM_Q8 && db == 8; }

template <int TYPE, int DB, int KB, int STAGES, int GROUPS>
__global__ __launch_bounds__(256 * GROUPS) __attribute__((
    amdgpu_waves_per_eu(alone(TYPE, DB) ? 1 : 2, alone(TYPE, DB) ? 1 : 2))) void many_kernel(
    AttnArgs a, Pools pools, Batch batch) {
  constexpr int kDim = 32 * DB, kStage = 4 * KB * DB * 1024, kColumns = 128;
  // operands read ahead: of heads of 256 two, as many as leave everything else in registers
  // (the same prompt in f16: 303 us with four, 278 with two)
  constexpr int kRead = DB == 8 && !alone(TYPE, DB) ? 2 : 4;
  __shared__ __attribute__((aligned(16))) uint8_t all_lds[GROUPS * STAGES * kStage];
  typedef typename Math<TYPE>::v8 v8;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) & 3, lane = threadIdx.x & 63, half = lane >> 5;
  const int group = GROUPS == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x >> 8);
  uint8_t* const lds = all_lds + group * (STAGES * kStage);
  const int h = blockIdx.x % pools.heads, rest = blockIdx.x / pools.heads, split = rest % a.splits, s = blockIdx.y;
  if (a.q8_out && a.splits == 1)
    zero_padding(a, kDim, batch.n_tok, ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * blockDim.x + threadIdx.x,
                 (int64_t)gridDim.x * gridDim.y * blockDim.x);
  Pages pages(batch, pools, s, h);
  const Sequence seq = sequence(batch, pools.page_shift, s);
  const int flats = seq.count * a.group;

  // the last columns see the most keys: they start first
  for (int tile = a.tiles - 1 - rest / a.splits; (int64_t)tile * kColumns < flats; tile += a.tiles) {
    const int first = tile * kColumns, last = min(first + kColumns, flats) - 1;
    // what any and what all of the columns see, and the same of this wave's own
    int low, high, all_low, all_high, my_low, my_high, my_all_low, my_all_high, unused;
    const int mine = a.by_group.of(min(first + 32 * wave, last)), mine_end = a.by_group.of(min(first + 32 * wave + 31, last));
    seen(a, seq, a.by_group.of(first), a.by_group.of(last), low, high);
    seen(a, seq, a.by_group.of(first), a.by_group.of(first), unused, all_high);
    seen(a, seq, a.by_group.of(last), a.by_group.of(last), all_low, unused);
    seen(a, seq, mine, mine_end, my_low, my_high);
    seen(a, seq, mine, mine, unused, my_all_high);
    seen(a, seq, mine_end, mine_end, my_all_low, unused);
    const bool idle = first + 32 * wave > last;
    const Column c = column(a, seq, h, first + 32 * wave + (lane & 31));
    const int begin = low >> 5 & -KB, tiles = max(0, ((high + 31) >> 5) - begin);
    const int share = max(a.share, (tiles + a.splits * KB - 1) / (a.splits * KB) * KB);
    const int from = begin + split * share, end = min(begin + tiles, from + share);
    if (split > 0 && from >= end) {  // nothing left for this split
      no_part(a, seq, batch.n_tok, h, split, first, last);
      continue;
    }

    for (bool safe = false;; safe = true) {
      v8 q[2 * DB];
      load_queries<TYPE, DB>(a, c, lane, q);
      v16f o[DB];
#pragma unroll
      for (int d = 0; d < DB; ++d) o[d] = v16f{};
      Running run;
      // The stages are a ring: while tile t is worked on, the ones up to t + kAhead are on their
      // way.  `here` of each, oldest first: whether its tiles are somewhere.
      constexpr int kAhead = STAGES - 1;
      Places<KB> next;
      Stager<TYPE, DB, KB> stager;
      uint32_t here_of[kAhead];
      constexpr int kStep = KB * GROUPS;  // a group's tiles are KB of every kStep
      const int mine_from = from + group * KB;
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        next.find(pages, mine_from + i * kStep, end);
        here_of[i] = next.here();
        if (mine_from + i * kStep < end) {
          stager.load(pools, next, wave, lane, lds + i * kStage);
          stager.store(wave, lane, lds + i * kStage);
        }
      }
      next.find(pages, mine_from + kAhead * kStep, end);
#pragma unroll
      for (int i = 0; i < 2 * DB; ++i) pin(q[i]);  // here, not in the loop, where the wait would be for the loads ahead too
      int stage = 0, free_stage = kAhead;
      for (int round = from; round < end; round += kStep) {
        const int t = round + group * KB;  // may lie behind the end for the last group
        // this wave's loads of tile t, which are older than those of the tiles ahead
        if (kAhead > 1 && t + (kAhead - 1) * kStep < end)
          wait_loads<(kAhead - 1) * Stager<TYPE, DB, KB>::kLoads>();
        else
          wait_loads<0>();
        __syncthreads();
        const uint32_t here_bits = here_of[0];
        const bool more = t + kAhead * kStep < end;
        uint8_t* const other = lds + free_stage * kStage;
#pragma unroll
        for (int i = 0; i + 1 < kAhead; ++i) here_of[i] = here_of[i + 1];
        here_of[kAhead - 1] = next.here();
        if (more) stager.load(pools, next, wave, lane, other);
        next.find(pages, t + (kAhead + 1) * kStep, end);
        const int slot0 = 32 * t;
        const bool here = here_bits == (1u << KB) - 1;
        if (safe) {
          constexpr int kPieces = kStage / 32 / KB;  // of 16 bytes, of a tile's values
#pragma unroll
          for (int k = 0; k < KB; ++k) {
            const int slot = slot0 + 32 * k;
            if (t < end && ((here_bits >> k & 1) == 0 || slot < all_low || slot + 32 > all_high)) {
              v8* const values = (v8*)(lds + stage * kStage + kStage / 2) + k * kPieces;
              for (int i = threadIdx.x & 255; i < kPieces; i += 256) values[i] = finite<TYPE>(values[i]);
            }
          }
          __syncthreads();
        }
        if (!idle && t < end && slot0 < my_high && slot0 + 32 * KB > my_low) {
          const uint8_t* const keys = lds + stage * kStage + lane * 16;
          const uint8_t* const values = keys + kStage / 2;
          v16f score[KB];
#pragma unroll
          for (int k = 0; k < KB; ++k) score[k] = v16f{};
          products<v8, 2 * DB * KB, kRead>(
              keys, [](int i) { return (i % KB * 2 * DB + i / KB) * 1024; },
              [&](int i, const v8& k) { score[i % KB] = Math<TYPE>::mma(k, q[i / KB], score[i % KB]); });
          if (!here || slot0 < my_all_low || slot0 + 32 * KB > my_all_high) {
#pragma unroll
            for (int k = 0; k < KB; ++k)  // a tile that is nowhere is seen by nobody
              hide(score[k], slot0 + 32 * k, half, c.low, (here_bits >> k & 1) != 0 ? c.high : 0);
          }
          v8 p[2 * KB];
          // ahead of the other wave of the SIMD, whose matrix instructions take a while each
          // (a prompt of 3314: 122.8 -> 120.2 us)
          __builtin_amdgcn_s_setprio(1);
          soften<TYPE, DB, KB>(score, a.scale2, run, o, p);
          __builtin_amdgcn_s_setprio(0);
          products<v8, 2 * DB * KB, kRead>(
              values, [](int i) { return (i / DB / 2 * 2 * DB + 2 * (i % DB) + i / DB % 2) * 1024; },
              [&](int i, const v8& v) { o[i % DB] = Math<TYPE>::mma(v, p[i / DB], o[i % DB]); });
        }
        if (more) stager.store(wave, lane, other);
        free_stage = stage;
        stage = stage + 1 == STAGES ? 0 : stage + 1;
      }
      if constexpr (GROUPS > 1) {
        // the second group's sums join the first's, lane by lane through the second's stages, as
        // many channels at a time as these hold
        constexpr int kMoved = 16 * DB * 1024 <= STAGES * kStage ? DB : DB / 2;
        static_assert(16 * kMoved * 1024 <= STAGES * kStage, "the sums fit the stages");
        v4f* const moved = (v4f*)(all_lds + STAGES * kStage + wave * (kMoved * 4096)) + lane;
        float2* const state = (float2*)(all_lds + wave * 512) + lane;
        float by = 0.0f, by2 = 0.0f;
#pragma unroll
        for (int from_block = 0; from_block < DB; from_block += kMoved) {
          __syncthreads();
          if (group == 1) {
#pragma unroll
            for (int i = 0; i < 4 * kMoved; ++i) {
              const v16f& x = o[from_block + (i >> 2)];
              moved[64 * i] = v4f{x[4 * (i & 3)], x[4 * (i & 3) + 1], x[4 * (i & 3) + 2], x[4 * (i & 3) + 3]};
            }
            if (from_block == 0) *state = make_float2(run.top, run.sum);
          }
          __syncthreads();
          if (group == 0) {
            if (from_block == 0) {
              const float2 m = *state;
              const float top = fmaxf(run.top, m.x);
              by = run.top == kNone ? 0.0f : __builtin_amdgcn_exp2f((run.top - top) * a.scale2);
              by2 = m.x == kNone ? 0.0f : __builtin_amdgcn_exp2f((m.x - top) * a.scale2);
              run.top = top;
              run.sum = fmaf(m.y, by2, run.sum * by);
            }
#pragma unroll
            for (int i = 0; i < 4 * kMoved; ++i) {
              const v4f v = moved[64 * i];
              v16f& x = o[from_block + (i >> 2)];
#pragma unroll
              for (int j = 0; j < 4; ++j) x[4 * (i & 3) + j] = fmaf(v[j], by2, x[4 * (i & 3) + j] * by);
            }
          }
        }
      }
      const bool out_here = !idle && group == 0;
      bool odd = false;
#pragma unroll
      for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) odd |= !(fabsf(o[d][i]) < __builtin_inff());
      // again, safely, where a result is no finite number; the stages are read
      if (__syncthreads_or(odd) && !safe) continue;

      const float total = both_sum(run.sum);
      if (!safe) {
        if (out_here) store_column<TYPE, DB>(a, c, split, batch.n_tok, half, run.top, total, o);
        __syncthreads();  // the stages are free again
        break;
      }
      // Where values are added that the product left out, the columns' results pass through
      // the wave's quarter of the stages, kBlocks blocks of 32 channels at a time, so that this
      // is one loop; 16-byte pieces are exchanged by column, or all columns' would be in the
      // same banks.
      constexpr int kBlocks = KB * DB / 2, kSwap = kBlocks % 2 == 0 ? 15 : 7;
      float* const out = (float*)(lds + wave * (kStage / 2));
#pragma unroll
      for (int pass = 0; pass < DB; pass += kBlocks) {
        if (!out_here) break;
#pragma unroll
        for (int d = 0; d < kBlocks; ++d)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *(float4*)(out + (lane & 31) * (32 * kBlocks) + 4 * ((8 * d + 2 * i + half) ^ (lane & kSwap))) =
                make_float4(o[pass + d][4 * i], o[pass + d][4 * i + 1], o[pass + d][4 * i + 2], o[pass + d][4 * i + 3]);
        wave_sync();
#pragma unroll 1
        for (int i = lane; i < 32 * 8 * kBlocks; i += 64) {  // whole groups of eight lanes have a column
          const int n = i / (8 * kBlocks), piece = i % (8 * kBlocks);
          const float top = __shfl(run.top, n), all = __shfl(total, n);
          const Column to = column(a, seq, h, first + 32 * wave + n);
          float4 x = *(const float4*)(out + n * (32 * kBlocks) + 4 * (piece ^ (n & kSwap)));
          if (!to.real) continue;
          const int d = 32 * pass + 4 * piece;
          add_edges<TYPE>(pools, batch, s, h, {from, end, all_low, all_high}, to, d, x);
          store_part<TYPE>(a, kDim, batch.n_tok, split, to, d, x, top, all);
        }
        wave_sync();
      }
      __syncthreads();  // the stages are free again
      break;
    }
  }
}

constexpr int few_waves(int db) { return db <= 4 ? 4 : 2; }

// Stages of many_kernel: as many as leave two work-groups, or a group's two halves, on a CU
// (160 KiB of LDS); q8 tiles pass through registers, one ahead.
constexpr int stages(int type, int db) { return type == QMM_Q8 ? 2 : db == 2 ? 4 : db == 3 ? 3 : db == 4 ? 2 : db == 6 ? 3 : 2; }

template <int TYPE, int DB>
hipError_t launch_dim(const AttnArgs& a, const Pools& p, const Batch& b, const AttnPlan& plan, hipStream_t s) {
  const dim3 grid((unsigned)(plan.work_groups / b.n_seq), (unsigned)b.n_seq);
  constexpr int KB = DB <= 4 ? 2 : 1;
  if (plan.few) {
    constexpr int W = few_waves(DB);
    const size_t lds = sizeof(float) * W * (64 + (size_t)plan.columns * (32 * DB + 4));
    few_kernel<TYPE, DB, W><<<grid, 64 * W, lds, s>>>(a, p, b);
    return hipGetLastError();
  }
  if constexpr (!alone(TYPE, DB)) {
    if (plan.groups == 2) {
      many_kernel<TYPE, DB, KB, stages(TYPE, DB), 2><<<grid, 512, 0, s>>>(a, p, b);
      return hipGetLastError();
    }
  }
  many_kernel<TYPE, DB, KB, stages(TYPE, DB), 1><<<grid, 256, 0, s>>>(a, p, b);
  return hipGetLastError();
}

template <int TYPE>
hipError_t launch_type(const AttnArgs& a, const Pools& p, const Batch& b, const AttnPlan& plan, hipStream_t s) {
  switch (p.dim) {
    case 64: return launch_dim<TYPE, 2>(a, p, b, plan, s);
    case 96: return launch_dim<TYPE, 3>(a, p, b, plan, s);
    case 128: return launch_dim<TYPE, 4>(a, p, b, plan, s);
    case 192: return launch_dim<TYPE, 6>(a, p, b, plan, s);
    default: return launch_dim<TYPE, 8>(a, p, b, plan, s);
  }
}

}  // namespace

}  // namespace qmm
