// qmm_rope.hip -- rotary positions of the new tokens' queries and keys, and keys and
// values kept in the paged cache; and the cache read back.
//
//   (a, b) at position p -> m*(a cos t - b sin t, a sin t + b cos t),  t = p*f
//
// t in turns is formed in 64 bits and modulo one: at position 10^6 the product in 32
// bits would be off by up to 0.03 radians.  Sine and cosine of what is left (f32) are
// formed once for a work-group's tokens and used for all of its heads.
//
// Memory bounds it: q, k and v are read once, q and the cache written once.  A
// work-group takes 16 slots that lie in one tile of the cache, so that keys leave as runs of
// 256 bytes (a lane's eight channels are one piece of the tile) and values as
// runs of 512 (a lane gathers eight tokens of a channel, so that only the first
// and last slots of a chunk are written one by one).
// Measured: 3314 tokens of 32 + 32 heads of 128 from f32 50.1 us (4.9 TB/s, a copy's rate); 24 chunks of
// 1674 tokens, 40 + 8 heads, into q8 16.2 us (2.5 TB/s), where work-groups' starts bound it; one token
// 4.9 us, all of it a work-group's path.
#include "qmm_cache.h"
#include "qmm_common.h"
#include "qmm_internal.h"
#include "qmm_quant.h"
#include "qmm_rope.h"

#include <algorithm>

namespace qmm {

namespace {

constexpr int kSlots = 16;      // slots of a work-group
constexpr int kThreads = 256;

template <int TYPE>
__device__ __forceinline__ void load8(const void* p, int64_t i, float (&x)[8]) {
  const float4 a = load4<TYPE>(p, i), b = load4<TYPE>(p, i + 4);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
  x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

template <int TYPE>
__device__ __forceinline__ void store8(void* p, int64_t i, const float (&x)[8]) {
  typedef elem_t<TYPE> T;
  if constexpr (TYPE == QMM_F32) {
    store4<TYPE>(p, i, make_float4(x[0], x[1], x[2], x[3]));
    store4<TYPE>(p, i + 4, make_float4(x[4], x[5], x[6], x[7]));
  } else {
    typedef T v8 __attribute__((ext_vector_type(8)));
    *(v8*)((T*)p + i) = v8{(T)x[0], (T)x[1], (T)x[2], (T)x[3], (T)x[4], (T)x[5], (T)x[6], (T)x[7]};
  }
}

__device__ __forceinline__ void store8_any(int type, void* p, int64_t i, const float (&x)[8]) {
  if (type == QMM_F32) store8<QMM_F32>(p, i, x);
  else if (type == QMM_F16) store8<QMM_F16>(p, i, x);
  else store8<QMM_BF16>(p, i, x);
}

// A frequency as turns per position, whole ones left out (a position has whole numbers of
// them), in units of 2^-64: a position times it, modulo 2^64, is the angle's place in its
// turn, with nothing lost at any position but the rounding of the frequency itself.
__device__ __forceinline__ uint64_t turns_of(double radians) {
  const double t = fabs(radians) * 0.15915494309189533577;  // 1/(2 pi)
  const double high = (t - floor(t)) * 4294967296.0, whole = floor(high);
  const uint64_t step = ((uint64_t)(uint32_t)whole << 32) + (uint64_t)((high - whole) * 4294967296.0);
  return radians < 0.0 ? 0 - step : step;
}

// (cos, sin) at a position.  The nearest quarter turn is taken off as an integer; of the
// rest, |x| <= pi/4 once in f32, the Taylor polynomials to x^9 and x^10 (their remainders
// are below 3e-9 and 2e-10).  The sum of the roundings is below 4 * 2^-24.  With the
// angle in 64-bit floating point and the library's sincospi, sine and cosine took more of a
// work-group's time than four heads' rotation.
__device__ __forceinline__ float2 turned(int position, uint64_t step) {
  const uint32_t at = (uint32_t)(((uint64_t)(int64_t)position * step) >> 32);
  const uint32_t quarter = (at + (1u << 29)) >> 30;
  const float x = (float)(int32_t)(at - (quarter << 30)) * 1.4629180792671596e-9f, x2 = x * x;  // 2 pi / 2^32
  float s = fmaf(x2, 2.75573192e-6f, -1.98412698e-4f);
  s = fmaf(x2, s, 8.33333333e-3f);
  s = fmaf(x2, s, -1.66666667e-1f);
  s = fmaf(x * x2, s, x);
  float c = fmaf(x2, -2.75573192e-7f, 2.48015873e-5f);
  c = fmaf(x2, c, -1.38888889e-3f);
  c = fmaf(x2, c, 4.16666667e-2f);
  c = fmaf(x2, c, -0.5f);
  c = fmaf(x2, c, 1.0f);
  const float a = (quarter & 1) != 0 ? s : c, b = (quarter & 1) != 0 ? c : s;
  return make_float2(((quarter + 1) & 2) != 0 ? -a : a, (quarter & 2) != 0 ? -b : b);
}

// What a thread rotates at a time: 16 channels of a token's head as two runs of
// eight.  Half layout: the runs at `u`*8 in both halves; interleaved, and where
// nothing turns: 16 channels in a row.
struct Unit {
  int a, b;    // first channel of each run
  int pair;    // first pair, < 0: nothing turns
};

__device__ __forceinline__ Unit unit(const RopeArgs& r, int u) {
  const int half = r.n_rot >> 1;
  if (16 * u >= r.n_rot) return {16 * u, 16 * u + 8, -1};
  if (r.layout == QMM_ROPE_HALF) return {8 * u, half + 8 * u, 8 * u};
  return {16 * u, 16 * u + 8, 8 * u};
}

// turn: the eight pairs' (cos, sin), times the magnitude
__device__ __forceinline__ void rotate(const RopeArgs& r, const float2* turn, float (&a)[8], float (&b)[8]) {
  if (r.layout == QMM_ROPE_HALF) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 t = turn[i];
      const float x = a[i], y = b[i];
      a[i] = fmaf(x, t.x, -(y * t.y));
      b[i] = fmaf(x, t.y, y * t.x);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 t = turn[i], s = turn[4 + i];
      const float x = a[2 * i], y = a[2 * i + 1], z = b[2 * i], w = b[2 * i + 1];
      a[2 * i] = fmaf(x, t.x, -(y * t.y));
      a[2 * i + 1] = fmaf(x, t.y, y * t.x);
      b[2 * i] = fmaf(z, s.x, -(w * s.y));
      b[2 * i + 1] = fmaf(z, s.y, w * s.x);
    }
  }
}

// A thread's unit of a head as loaded: 16 values, still of their type.
template <int IN>
struct Loaded16 {
  typedef elem_t<IN> v8 __attribute__((ext_vector_type(8)));
  v8 a, b;
  __device__ __forceinline__ void load(const void* p, int64_t i, const Unit& at) {
    a = *(const v8*)((const elem_t<IN>*)p + i + at.a);
    b = *(const v8*)((const elem_t<IN>*)p + i + at.b);
  }
  __device__ __forceinline__ void get(float (&x)[8], float (&y)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (float)a[i], y[i] = (float)b[i];
  }
};

// Eight channels' codes of a q8 key, and the block's scale from the lane that has its first.
__device__ __forceinline__ void store_codes(uint8_t* tile, int dim, int r, int d, bool first, const Q8Part<8>& q) {
  *(uint2*)(tile + key_code_at(r, d)) = make_uint2(q.codes[0] ^ 0x80808080u, q.codes[1] ^ 0x80808080u);
  if (first) *(uint16_t*)(tile + scale_at(dim, r, d >> 5)) = (uint16_t)q.pair;
}

__device__ __forceinline__ Q8Part<16> quant_sixteen(const float (&a)[8], const float (&b)[8]) {
  float v[16];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = a[i], v[8 + i] = b[i];
  return quant_part<16>(v);
}

// IN: type of q, k and v; CACHE: of the cache.  blockIdx: x the 16 slots (in steps of
// the grid, where the sequence has more), y the job (some heads of q, k or v), z the
// sequence.  A thread keeps its token and channels and goes from head to head, the
// next head's values on their way while it works on one.
template <int IN, int CACHE>
__global__ __launch_bounds__(kThreads, CACHE == QMM_Q8 ? 3 : 4) void rope_kernel(RopeArgs r, Pools pools, Batch batch) {
  extern __shared__ float lds[];
  const int s = blockIdx.z, job = blockIdx.y;
  const Sequence seq = sequence(batch, pools.page_shift, s);
  if (seq.count == 0) return;
  // which tensor, and which of its heads
  const int kind = job < r.q_jobs ? 0 : job < r.q_jobs + r.k_jobs ? 1 : 2;
  const int per_job = kind == 0 ? r.q_heads_per_job : r.heads_per_job;
  const int head0 = (job - (kind == 0 ? 0 : kind == 1 ? r.q_jobs : r.q_jobs + r.k_jobs)) * per_job;
  const int head_end = min(head0 + per_job, kind == 0 ? r.q_heads : pools.heads);
  const int dim = pools.dim, units = dim >> 4, half = r.n_rot >> 1;
  const int slot0 = seq.length - seq.count;  // of the first new token; below 0: tokens without a slot
  float2* const turns = (float2*)lds;                               // [16][half]
  float* const stage = lds + 2 * kSlots * half;                     // q8 keys: [16][dim + 4] values of a head
  uint8_t* const codes = (uint8_t*)lds;                             // q8 values: [heads][16][dim + 4] codes

  for (int block = blockIdx.x;; block += gridDim.x) {
    const int base = ((slot0 >> 4) + block) * kSlots;
    if (base >= seq.length) break;
    const int from = max(0, slot0 - base), to = min(kSlots, seq.length - base), count = to - from;
    const int row0 = seq.first + base - slot0;  // row of slot `base`
    if (kind > 0 && base < 0) continue;         // keys and values of slots below 0: there is none
    const int in_tile = base & 31;
    // the tile of head 0, and the bytes from head to head
    const int64_t tile0 = kind > 0 ? tile_offset<true>(batch, pools, s, 0, base >> 5) : 0;
    const int64_t tile_step = (int64_t)tile_bytes(CACHE, dim) << (pools.page_shift - 5);
    if (tile0 < 0) continue;  // a page outside the pool
    const Rows& x = kind == 0 ? r.q : kind == 1 ? r.k : r.v;
    // Token and unit of a thread (at most 16 * 16 of them), and as many heads side by side
    // as there are threads for.  The first head's values are on their way while the turns
    // are computed.
    const int places = count * units, side = kThreads / places;
    int h = head0 + (int)threadIdx.x / places;
    const bool turning = kind == 0 || (kind == 1 && CACHE != QMM_Q8), mine = (int)threadIdx.x < side * places;
    // q8 keys: whether the lanes of a token's units hold whole blocks of 32 channels
    const bool whole_blocks =
        r.n_rot == 0 || r.layout == QMM_ROPE_INTERLEAVED || (r.n_rot % 64 == 0 && units % 4 == 0);
    const int t = from + (int)threadIdx.x % places / units;
    const Unit at = kind == 2 ? Unit{16 * ((int)threadIdx.x % units), 16 * ((int)threadIdx.x % units) + 8, -1}
                              : unit(r, (int)threadIdx.x % units);
    const int64_t in = (row0 + t) * x.stride;
    Loaded16<IN> now;
    if ((turning || CACHE == QMM_Q8) && mine && h < head_end) now.load(x.p, in + h * x.head_stride, at);
    if (kind < 2) {
      if (half > 0) {  // a thread keeps its pair and goes from token to token
        const int abreast = kThreads / half, pair = (int)threadIdx.x % half;
        int token = (int)threadIdx.x / half;
        const auto position = [&](int i) {
          return i >= count ? 0 : r.positions != nullptr ? r.positions[row0 + from + i] : base + from + i;
        };
        if (token < abreast) {
          const uint64_t step = turns_of(r.frequencies[pair]);
          int p = position(token);
          for (; token < count; token += abreast) {
            const int next = position(token + abreast);
            const float2 turn = turned(p, step);
            turns[(from + token) * half + pair] = make_float2(turn.x * r.magnitude, turn.y * r.magnitude);
            p = next;
          }
        }
      }
      __syncthreads();
    }
    if (turning) {
      if (mine) {
        float2 turn[8];
        if (at.pair >= 0) {
#pragma unroll
          for (int i = 0; i < 8; ++i) turn[i] = turns[t * half + at.pair + i];
        }
        const int64_t out = (row0 + t) * r.q_out.stride;
        for (; h < head_end; h += side) {
          float a[8], b[8];
          now.get(a, b);
          if (h + side < head_end) now.load(x.p, in + (h + side) * x.head_stride, at);
          if (at.pair >= 0) rotate(r, turn, a, b);
          if (kind == 0) {
            const int64_t o = out + h * r.q_out.head_stride;
            store8_any(r.out_type, (void*)r.q_out.p, o + at.a, a);
            store8_any(r.out_type, (void*)r.q_out.p, o + at.b, b);
          } else if constexpr (CACHE != QMM_Q8) {
            uint8_t* const to_tile = pools.k + tile0 + h * tile_step;
            store8<CACHE>(to_tile, key_at(in_tile + t, at.a), a);
            store8<CACHE>(to_tile, key_at(in_tile + t, at.b), b);
          }
        }
      }
    } else if constexpr (CACHE != QMM_Q8) {
      typedef elem_t<CACHE> T;
      typedef T v8 __attribute__((ext_vector_type(8)));
      // eight slots of a channel
      const int runs = 2 * dim, beside = max(1, kThreads / runs);
      for (int run = threadIdx.x % min(runs, kThreads); run < runs; run += kThreads) {
        int h = head0 + (runs < kThreads ? (int)threadIdx.x / runs : 0);
        if (runs < kThreads && (int)threadIdx.x >= beside * runs) break;
        const int d = run % dim, g = run >= dim ? 8 : 0;
        if (g + 8 <= from || g >= to) continue;
        const elem_t<IN>* const in = (const elem_t<IN>*)x.p + (row0 + g) * x.stride + d;
        elem_t<IN> now[8];
        const auto load = [&](int head) {
#pragma unroll
          for (int n = 0; n < 8; ++n)
            if (g + n >= from && g + n < to) now[n] = in[n * x.stride + head * x.head_stride];
        };
#pragma unroll
        for (int n = 0; n < 8; ++n) now[n] = (elem_t<IN>)0.0f;
        if (h < head_end) load(h);
        for (; h < head_end; h += beside) {
          v8 e;
#pragma unroll
          for (int n = 0; n < 8; ++n) e[n] = (T)(float)now[n];
          if (h + beside < head_end) load(h + beside);
          T* const p = (T*)(pools.v + tile0 + h * tile_step) + value_at(in_tile + g, d);
          if (g >= from && g + 8 <= to) {
            *(v8*)p = e;
          } else {
#pragma unroll
            for (int n = 0; n < 8; ++n)
              if (g + n >= from && g + n < to) p[n] = e[n];
          }
        }
      }
    } else if (kind == 1 && !whole_blocks) {
      for (int head = head0; head < head_end; ++head) {
        __syncthreads();  // the head before is out of the stage
        if (threadIdx.x < places) {
          float a[8], b[8];
          now.load(x.p, in + head * x.head_stride, at);
          now.get(a, b);
          if (at.pair >= 0) rotate(r, turns + t * half + at.pair, a, b);
          store8<QMM_F32>(stage, t * (dim + 4) + at.a, a);
          store8<QMM_F32>(stage, t * (dim + 4) + at.b, b);
        }
        __syncthreads();
        uint8_t* const out = pools.k + tile0 + head * tile_step;
        // four lanes quantize a block of 32 channels, eight each
        for (int i = threadIdx.x; i < count * (dim >> 3); i += kThreads) {
          const int d = 8 * (i % (dim >> 3)), token = from + i / (dim >> 3);
          float x8[8];
          load8<QMM_F32>(stage, token * (dim + 4) + d, x8);
          store_codes(out, dim, in_tile + token, d, (i & 3) == 0, quant_part<8>(x8));
        }
      }
    } else if (kind == 1) {
      // a block's values are in four lanes (the halves' runs) or two (16 in a row): nothing
      // passes through LDS
      if (mine) {
        const bool in_halves = at.b != at.a + 8;
        for (; h < head_end; h += side) {
          float a[8], b[8];
          now.get(a, b);
          if (h + side < head_end) now.load(x.p, in + (h + side) * x.head_stride, at);
          if (at.pair >= 0) rotate(r, turns + t * half + at.pair, a, b);
          uint8_t* const out = pools.k + tile0 + h * tile_step;
          if (in_halves) {
            store_codes(out, dim, in_tile + t, at.a, (at.a & 31) == 0, quant_part<8>(a));
            store_codes(out, dim, in_tile + t, at.b, (at.b & 31) == 0, quant_part<8>(b));
          } else {
            const Q8Part<16> q = quant_sixteen(a, b);
            store_codes(out, dim, in_tile + t, at.a, (at.a & 31) == 0, Q8Part<8>{{q.codes[0], q.codes[1]}, q.pair});
            store_codes(out, dim, in_tile + t, at.b, false, Q8Part<8>{{q.codes[2], q.codes[3]}, q.pair});
          }
        }
      }
    } else {
      // values: blocks quantized where they are loaded, their codes turned in LDS, `side` heads at a time
      for (int head = head0; head < head_end; head += side, h += side) {
        const int heads = min(side, head_end - head), pitch = kSlots * (dim + 4);
        __syncthreads();  // the heads before are out of LDS
        if (mine && h < head_end) {
          float a[8], b[8];
          now.get(a, b);
          if (h + side < head_end) now.load(x.p, in + (h + side) * x.head_stride, at);
          const Q8Part<16> q = quant_sixteen(a, b);
          uint32_t* const to_lds = (uint32_t*)(codes + (h - head) * pitch + t * (dim + 4) + at.a);
#pragma unroll
          for (int i = 0; i < 4; ++i) to_lds[i] = q.codes[i] ^ 0x80808080u;
          if ((at.a & 31) == 0)
            *(uint16_t*)(pools.v + tile0 + h * tile_step + scale_at(dim, in_tile + t, at.a >> 5)) = (uint16_t)q.pair;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < heads * 2 * dim; i += kThreads) {
          const int d = i % dim, j = i / dim, g = 8 * (j & 1);
          if (g + 8 <= from || g >= to) continue;
          const uint8_t* const c = codes + (j >> 1) * pitch + g * (dim + 4) + d;
          uint8_t* const p = pools.v + tile0 + (head + (j >> 1)) * tile_step + value_code_at(in_tile + g, d);
          if (g >= from && g + 8 <= to) {
            uint32_t w[2] = {0, 0};
#pragma unroll
            for (int n = 0; n < 8; ++n) w[n >> 2] |= (uint32_t)c[n * (dim + 4)] << (8 * (n & 3));
            *(uint2*)p = make_uint2(w[0], w[1]);
          } else {
            for (int n = 0; n < 8; ++n)
              if (g + n >= from && g + n < to) p[n] = c[n * (dim + 4)];
          }
        }
      }
    }
    __syncthreads();  // the next 16 slots' turns
  }
}

// The cache read back, 16 slots of some heads at a time: of keys a thread takes eight
// channels of a slot, of values eight slots of a channel, as they lie in the tiles.  Of few
// tokens a work-group's path bounds it: 1674 of 8 heads of 128 from q8 7.3 us (10 MB).
template <int CACHE, int OUT>
__global__ __launch_bounds__(kThreads) void read_kernel(Pools pools, Batch batch, int heads_per_job, void* k, void* v) {
  typedef elem_t<OUT> T;
  const int s = blockIdx.z, dim = pools.dim, runs = dim >> 3;
  const Sequence seq = sequence(batch, pools.page_shift, s);
  if (seq.count == 0) return;
  const int slot0 = seq.length - seq.count, head0 = blockIdx.y * heads_per_job;
  const int heads = min(heads_per_job, pools.heads - head0);
  const int64_t tile_step = (int64_t)tile_bytes(CACHE, dim) << (pools.page_shift - 5);
  for (int block = blockIdx.x;; block += gridDim.x) {
    const int base = ((slot0 >> 4) + block) * kSlots;
    if (base >= seq.length) break;
    const int from = max(0, slot0 - base), to = min(kSlots, seq.length - base), count = to - from;
    const int row0 = seq.first + base - slot0, in_tile = base & 31;
    const int64_t tile0 = base < 0 ? -1 : tile_offset<true>(batch, pools, s, 0, base >> 5);
    for (int i = threadIdx.x; k != nullptr && i < count * heads * runs; i += kThreads) {
      const int d = 8 * (i % runs), j = i / runs, t = from + j % count, h = head0 + j / count, r = in_tile + t;
      float x[8] = {};
      if (tile0 >= 0) {
        const uint8_t* const tile = pools.k + tile0 + h * tile_step;
        if constexpr (CACHE == QMM_Q8) {
          const float scale = (float)*(const _Float16*)(tile + scale_at(dim, r, d >> 5));
          const uint2 c = *(const uint2*)(tile + key_code_at(r, d));
#pragma unroll
          for (int n = 0; n < 8; ++n) x[n] = (float)((int)(((n < 4 ? c.x : c.y) >> (8 * (n & 3))) & 255) - 128) * scale;
        } else {
          load8<CACHE>(tile, key_at(r, d), x);
        }
      }
      store8<OUT>(k, ((int64_t)(row0 + t) * pools.heads + h) * dim + d, x);
    }
    for (int i = threadIdx.x; v != nullptr && i < 2 * heads * dim; i += kThreads) {
      const int d = i % dim, j = i / dim, g = 8 * (j & 1), h = head0 + (j >> 1), r = in_tile + g;
      if (g + 8 <= from || g >= to) continue;
      float x[8] = {};
      if (tile0 >= 0) {
        const uint8_t* const tile = pools.v + tile0 + h * tile_step;
        if constexpr (CACHE == QMM_Q8) {
          typedef _Float16 v8 __attribute__((ext_vector_type(8)));
          const v8 scale = *(const v8*)(tile + scale_at(dim, r, d >> 5));
          const uint2 c = *(const uint2*)(tile + value_code_at(r, d));
#pragma unroll
          for (int n = 0; n < 8; ++n)
            x[n] = (float)((int)(((n < 4 ? c.x : c.y) >> (8 * (n & 3))) & 255) - 128) * (float)scale[n];
        } else {
          load8<CACHE>(tile, value_at(r, d), x);
        }
      }
#pragma unroll
      for (int n = 0; n < 8; ++n)
        if (g + n >= from && g + n < to) ((T*)v)[((int64_t)(row0 + g + n) * pools.heads + h) * dim + d] = (T)x[n];
    }
  }
}

template <int IN>
void launch_in(const RopeArgs& r, const Pools& p, const Batch& b, dim3 grid, size_t lds, hipStream_t s) {
  if (p.type == QMM_Q8) rope_kernel<IN, QMM_Q8><<<grid, kThreads, lds, s>>>(r, p, b);
  else if (p.type == QMM_F16) rope_kernel<IN, QMM_F16><<<grid, kThreads, lds, s>>>(r, p, b);
  else rope_kernel<IN, QMM_BF16><<<grid, kThreads, lds, s>>>(r, p, b);
}

template <int CACHE>
void launch_out(const Pools& p, const Batch& b, int type, int heads, void* k, void* v, dim3 grid, hipStream_t s) {
  if (type == QMM_F32) read_kernel<CACHE, QMM_F32><<<grid, kThreads, 0, s>>>(p, b, heads, k, v);
  else if (type == QMM_F16) read_kernel<CACHE, QMM_F16><<<grid, kThreads, 0, s>>>(p, b, heads, k, v);
  else read_kernel<CACHE, QMM_BF16><<<grid, kThreads, 0, s>>>(p, b, heads, k, v);
}

// Groups of 16 slots of a sequence.  Thousands of sequences with max_new unknown would have
// millions of them, most without a token: a work-group takes several then.
int64_t slot_groups(int64_t max_new, int64_t n_seq) {
  const int64_t most = std::max<int64_t>((1 << 18) / n_seq, 4);
  return std::min<int64_t>((std::max<int64_t>(max_new, 1) + 2 * kSlots - 2) / kSlots, std::min<int64_t>(most, 1 << 16));
}

}  // namespace

hipError_t launch_rope(RopeArgs r, const Pools& p, const Batch& b, int64_t max_new, hipStream_t s) {
  const int64_t blocks = slot_groups(max_new, b.n_seq);
  // As many heads for a work-group as leave a few work-groups of 16-bit values, or twice that
  // many of f32 ones, for every compute unit: of fewer, larger ones too few bytes are on
  // their way, of more the turns and starts cost.  3314 tokens of 32+32 heads of 128: from f32
  // 51.5 us with 9 heads, 56.7 with 19; q alone from f16 15.0 with 6, 17.3 with 3, 31 with 1.
  const int heads = r.q_heads + (r.k.p != nullptr ? p.heads : 0) + (r.v.p != nullptr ? p.heads : 0);
  r.q_heads_per_job = (int)std::clamp<int64_t>(blocks * b.n_seq * heads / (r.type == QMM_F32 ? 2048 : 1024), 2, 32);
  r.heads_per_job = p.type == QMM_Q8 ? std::min(r.q_heads_per_job, 8) : r.q_heads_per_job;  // codes' LDS
  const auto jobs = [](const void* x, int n, int per) { return x == nullptr ? 0 : (n + per - 1) / per; };
  r.q_jobs = jobs(r.q.p, r.q_heads, r.q_heads_per_job);
  r.k_jobs = jobs(r.k.p, p.heads, r.heads_per_job);
  const dim3 grid((unsigned)blocks, (unsigned)(r.q_jobs + r.k_jobs + jobs(r.v.p, p.heads, r.heads_per_job)), (unsigned)b.n_seq);
  size_t lds = kSlots * (size_t)r.n_rot * 4;
  if (p.type == QMM_Q8) {  // a key's values beside the turns, or the codes of a job's values
    lds = std::max(lds + kSlots * (size_t)(p.dim + 4) * 4, (size_t)r.heads_per_job * kSlots * (p.dim + 4));
  }
  (r.type == QMM_F32 ? launch_in<QMM_F32> : r.type == QMM_F16 ? launch_in<QMM_F16> : launch_in<QMM_BF16>)(r, p, b, grid,
                                                                                                         lds, s);
  return hipGetLastError();
}

hipError_t launch_cache_read(const Pools& p, const Batch& b, int64_t max_new, int type, void* k, void* v, hipStream_t s) {
  const int64_t blocks = slot_groups(max_new, b.n_seq);
  const int heads = (int)std::clamp<int64_t>(blocks * b.n_seq * p.heads / 1024, 1, 8);
  const dim3 grid((unsigned)blocks, (unsigned)((p.heads + heads - 1) / heads), (unsigned)b.n_seq);
  (p.type == QMM_Q8 ? launch_out<QMM_Q8> : p.type == QMM_F16 ? launch_out<QMM_F16> : launch_out<QMM_BF16>)(
      p, b, type, heads, k, v, grid, s);
  return hipGetLastError();
}

}  // namespace qmm
