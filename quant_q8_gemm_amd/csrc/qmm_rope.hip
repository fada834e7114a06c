// qmm_rope.hip -- rotary positions of the new tokens' queries and keys, and keys and
// values kept in the paged cache; and the cache read back.
//
//   (a, b) at position p -> m*(a cos t - b sin t, a sin t + b cos t),  t = p*f
//
// t in turns is formed and reduced to half a turn in 64 bits: at position 10^6 the
// product in 32 bits would be off by up to 0.03 radians.  Sine and cosine of what is left
// (f32, within an ulp or two) are formed once for a work-group's tokens and used
// for all of its heads.
//
// Memory bounds it: q, k and v are read once, q and the cache written once.  A
// work-group takes 16 slots that lie in one tile of the cache, so that keys leave as runs of
// 256 bytes (a lane's eight channels are one piece of the tile) and values as
// runs of 512 (a lane gathers eight tokens of a channel, so that only the first
// and last slots of a chunk are written one by one).
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

// IN: type of q, k and v; CACHE: of the cache.  blockIdx: x the 16 slots (in steps of
// the grid, where the sequence has more), y the job (heads_per_job heads of q, k or v),
// z the sequence.
template <int IN, int CACHE>
__global__ __launch_bounds__(kThreads) void rope_kernel(RopeArgs r, Pools pools, Batch batch) {
  extern __shared__ float lds[];
  const int s = blockIdx.z, job = blockIdx.y;
  const Sequence seq = sequence(batch, pools.page_shift, s);
  if (seq.count == 0) return;
  // which tensor, and which of its heads
  const int kind = job < r.q_jobs ? 0 : job < r.q_jobs + r.k_jobs ? 1 : 2;
  const int head0 = (job - (kind == 0 ? 0 : kind == 1 ? r.q_jobs : r.q_jobs + r.k_jobs)) * r.heads_per_job;
  const int heads = min(r.heads_per_job, (kind == 0 ? r.q_heads : pools.heads) - head0);
  const int dim = pools.dim, units = dim >> 4, half = r.n_rot >> 1;
  const int slot0 = seq.length - seq.count;  // of the first new token; below 0: tokens without a slot
  float2* const turns = (float2*)lds;                               // [16][half]
  float* const stage = lds + (kind == 2 ? 0 : 2 * kSlots * half);   // q8: [16][dim + 4] values of a head
  uint8_t* const codes = (uint8_t*)(stage + kSlots * (dim + 4));    // q8: [16][dim + 4] codes

  for (int block = blockIdx.x;; block += gridDim.x) {
    const int base = ((slot0 >> 4) + block) * kSlots;
    if (base >= seq.length) break;
    const int from = max(0, slot0 - base), to = min(kSlots, seq.length - base), count = to - from;
    const int row0 = seq.first + base - slot0;  // row of slot `base`
    if (kind < 2) {
      for (int i = threadIdx.x; i < count * half; i += kThreads) {
        const int t = from + i / half, pair = i % half;
        const int p = r.positions != nullptr ? r.positions[row0 + t] : base + t;
        const double turn = (double)p * r.frequencies[pair] * 0.15915494309189533577;  // 1/(2 pi)
        float sine, cosine;
        sincospif(2.0f * (float)(turn - __builtin_rint(turn)), &sine, &cosine);
        turns[t * half + pair] = make_float2(cosine * r.magnitude, sine * r.magnitude);
      }
      __syncthreads();
    }
    if (kind == 0) {
      for (int i = threadIdx.x; i < count * heads * units; i += kThreads) {
        const int u = i % units, j = i / units, t = from + j % count, h = head0 + j / count;
        const Unit at = unit(r, u);
        const int64_t in = (row0 + t) * r.q.stride + h * r.q.head_stride;
        const int64_t out = (row0 + t) * r.q_out.stride + h * r.q_out.head_stride;
        float a[8], b[8];
        load8<IN>(r.q.p, in + at.a, a);
        load8<IN>(r.q.p, in + at.b, b);
        if (at.pair >= 0) rotate(r, turns + t * half + at.pair, a, b);
        store8_any(r.out_type, (void*)r.q_out.p, out + at.a, a);
        store8_any(r.out_type, (void*)r.q_out.p, out + at.b, b);
      }
    } else if (base >= 0) {  // keys and values; slots below 0 are none
      const Rows& x = kind == 1 ? r.k : r.v;
      const int tile = base >> 5, in_tile = base & 31;
      if constexpr (CACHE != QMM_Q8) {
        if (kind == 1) {
          for (int i = threadIdx.x; i < count * heads * units; i += kThreads) {
            const int u = i % units, j = i / units, t = from + j % count, h = head0 + j / count;
            const Unit at = unit(r, u);
            const int64_t in = (row0 + t) * x.stride + h * x.head_stride;
            float a[8], b[8];
            load8<IN>(x.p, in + at.a, a);
            load8<IN>(x.p, in + at.b, b);
            if (at.pair >= 0) rotate(r, turns + t * half + at.pair, a, b);
            const int64_t to_tile = tile_offset(batch, pools, s, h, tile);
            if (to_tile < 0) continue;
            store8<CACHE>(pools.k + to_tile, key_at(in_tile + t, at.a), a);
            store8<CACHE>(pools.k + to_tile, key_at(in_tile + t, at.b), b);
          }
        } else {
          typedef elem_t<CACHE> T;
          typedef T v8 __attribute__((ext_vector_type(8)));
          for (int i = threadIdx.x; i < 2 * heads * dim; i += kThreads) {  // eight slots of a channel
            const int d = i % dim, j = i / dim, g = 8 * (j & 1), h = head0 + (j >> 1);
            if (g + 8 <= from || g >= to) continue;
            const int64_t to_tile = tile_offset(batch, pools, s, h, tile);
            if (to_tile < 0) continue;
            v8 e;
#pragma unroll
            for (int n = 0; n < 8; ++n) {
              const bool is = g + n >= from && g + n < to;
              e[n] = is ? (T)(float)((const elem_t<IN>*)x.p)[(row0 + g + n) * x.stride + h * x.head_stride + d] : (T)0.0f;
            }
            T* const p = (T*)(pools.v + to_tile) + value_at(in_tile + g, d);
            if (g >= from && g + 8 <= to) {
              *(v8*)p = e;
            } else {
#pragma unroll
              for (int n = 0; n < 8; ++n)
                if (g + n >= from && g + n < to) p[n] = e[n];
            }
          }
        }
      } else {
        for (int h = head0; h < head0 + heads; ++h) {
          __syncthreads();  // the head before is out of the stage
          for (int i = threadIdx.x; i < count * units; i += kThreads) {
            const int u = i % units, t = from + i / units;
            const Unit at = kind == 1 ? unit(r, u) : Unit{16 * u, 16 * u + 8, -1};
            const int64_t in = (row0 + t) * x.stride + h * x.head_stride;
            float a[8], b[8];
            load8<IN>(x.p, in + at.a, a);
            load8<IN>(x.p, in + at.b, b);
            if (at.pair >= 0) rotate(r, turns + t * half + at.pair, a, b);
            store8<QMM_F32>(stage, t * (dim + 4) + at.a, a);
            store8<QMM_F32>(stage, t * (dim + 4) + at.b, b);
          }
          __syncthreads();
          const int64_t to_tile = tile_offset(batch, pools, s, h, tile);  // the same in every thread
          if (to_tile < 0) continue;
          uint8_t* const out = (kind == 1 ? pools.k : pools.v) + to_tile;
          // four lanes quantize a block of 32 channels, eight each; dim/32 blocks times 4 lanes
          // times the tokens, in whole groups of four lanes
          for (int i = threadIdx.x; i < count * (dim >> 3); i += kThreads) {
            const int d = 8 * (i % (dim >> 3)), t = from + i / (dim >> 3);
            float x8[8];
            load8<QMM_F32>(stage, t * (dim + 4) + d, x8);
            const Q8Part<8> q = quant_part<8>(x8);
            const uint2 c = make_uint2(q.codes[0] ^ 0x80808080u, q.codes[1] ^ 0x80808080u);
            if (kind == 1) {
              *(uint2*)(out + key_code_at(in_tile + t, d)) = c;
            } else {
              *(uint32_t*)(codes + t * (dim + 4) + d) = c.x;
              *(uint32_t*)(codes + t * (dim + 4) + d + 4) = c.y;
            }
            if ((i & 3) == 0) *(uint16_t*)(out + scale_at(dim, in_tile + t, d >> 5)) = (uint16_t)q.pair;
          }
          if (kind == 2) {
            __syncthreads();
            for (int i = threadIdx.x; i < 2 * dim; i += kThreads) {
              const int d = i % dim, g = 8 * (i / dim);
              if (g + 8 <= from || g >= to) continue;
              uint8_t* const p = out + value_code_at(in_tile + g, d);
              if (g >= from && g + 8 <= to) {
                uint32_t w[2] = {0, 0};
#pragma unroll
                for (int n = 0; n < 8; ++n) w[n >> 2] |= (uint32_t)codes[(g + n) * (dim + 4) + d] << (8 * (n & 3));
                *(uint2*)p = make_uint2(w[0], w[1]);
              } else {
                for (int n = 0; n < 8; ++n)
                  if (g + n >= from && g + n < to) p[n] = codes[(g + n) * (dim + 4) + d];
              }
            }
          }
        }
      }
    }
    __syncthreads();  // the next 16 slots' turns
  }
}

template <int TYPE>
__device__ __forceinline__ void put8(void* p, int64_t i, const float (&x)[8]) {
  if (p != nullptr) store8<TYPE>(p, i, x);
}

// A thread reads eight channels of a token's head from both pools.
template <int CACHE, int OUT>
__global__ __launch_bounds__(kThreads) void read_kernel(Pools pools, Batch batch, void* k, void* v) {
  const int s = blockIdx.z, runs = pools.dim >> 3;
  const Sequence seq = sequence(batch, pools.page_shift, s);
  const int slot0 = seq.length - seq.count;
  const int64_t all = (int64_t)seq.count * pools.heads * runs;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < all; i += (int64_t)gridDim.x * kThreads) {
    const int d = 8 * (int)(i % runs), h = (int)(i / runs % pools.heads), t = (int)(i / runs / pools.heads);
    const int slot = slot0 + t, r = slot & 31;
    const int64_t tile = slot < 0 ? -1 : tile_offset(batch, pools, s, h, slot >> 5);
    float a[8] = {}, b[8] = {};
    if (tile >= 0) {
      const uint8_t *tk = pools.k + tile, *tv = pools.v + tile;
      if constexpr (CACHE == QMM_Q8) {
        const float sk = (float)*(const _Float16*)(tk + scale_at(pools.dim, r, d >> 5));
        const float sv = (float)*(const _Float16*)(tv + scale_at(pools.dim, r, d >> 5));
        const uint2 c = *(const uint2*)(tk + key_code_at(r, d));
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          a[n] = (float)((int)(((n < 4 ? c.x : c.y) >> (8 * (n & 3))) & 255) - 128) * sk;
          b[n] = (float)((int)tv[value_code_at(r, d + n)] - 128) * sv;
        }
      } else {
        load8<CACHE>(tk, key_at(r, d), a);
#pragma unroll
        for (int n = 0; n < 8; ++n) b[n] = (float)((const elem_t<CACHE>*)tv)[value_at(r, d + n)];
      }
    }
    const int64_t out = ((int64_t)(seq.first + t) * pools.heads + h) * pools.dim + d;
    put8<OUT>(k, out, a);
    put8<OUT>(v, out, b);
  }
}

template <int IN>
void launch_in(const RopeArgs& r, const Pools& p, const Batch& b, dim3 grid, size_t lds, hipStream_t s) {
  if (p.type == QMM_Q8) rope_kernel<IN, QMM_Q8><<<grid, kThreads, lds, s>>>(r, p, b);
  else if (p.type == QMM_F16) rope_kernel<IN, QMM_F16><<<grid, kThreads, lds, s>>>(r, p, b);
  else rope_kernel<IN, QMM_BF16><<<grid, kThreads, lds, s>>>(r, p, b);
}

template <int CACHE>
void launch_out(const Pools& p, const Batch& b, int type, void* k, void* v, dim3 grid, hipStream_t s) {
  if (type == QMM_F32) read_kernel<CACHE, QMM_F32><<<grid, kThreads, 0, s>>>(p, b, k, v);
  else if (type == QMM_F16) read_kernel<CACHE, QMM_F16><<<grid, kThreads, 0, s>>>(p, b, k, v);
  else read_kernel<CACHE, QMM_BF16><<<grid, kThreads, 0, s>>>(p, b, k, v);
}

}  // namespace

hipError_t launch_rope(RopeArgs r, const Pools& p, const Batch& b, int64_t max_new, hipStream_t s) {
  const int64_t blocks = std::min<int64_t>((std::max<int64_t>(max_new, 1) + 2 * kSlots - 2) / kSlots, 1 << 16);
  // Turns cost about as much as four heads' rotation, so a work-group takes as many
  // heads as leave some work-groups for every compute unit.
  const int heads = r.q_heads + (r.k.p != nullptr ? p.heads : 0) + (r.v.p != nullptr ? p.heads : 0);
  r.heads_per_job = (int)std::clamp<int64_t>(blocks * b.n_seq * heads / 1024, 2, 32);
  const auto jobs = [&](const void* x, int n) { return x == nullptr ? 0 : (n + r.heads_per_job - 1) / r.heads_per_job; };
  r.q_jobs = jobs(r.q.p, r.q_heads);
  r.k_jobs = jobs(r.k.p, p.heads);
  const dim3 grid((unsigned)blocks, (unsigned)(r.q_jobs + r.k_jobs + jobs(r.v.p, p.heads)), (unsigned)b.n_seq);
  const size_t lds = kSlots * ((size_t)r.n_rot * 4 + (p.type == QMM_Q8 ? (size_t)(p.dim + 4) * 5 : 0));
  (r.type == QMM_F32 ? launch_in<QMM_F32> : r.type == QMM_F16 ? launch_in<QMM_F16> : launch_in<QMM_BF16>)(r, p, b, grid,
                                                                                                         lds, s);
  return hipGetLastError();
}

hipError_t launch_cache_read(const Pools& p, const Batch& b, int64_t max_new, int type, void* k, void* v, hipStream_t s) {
  const int64_t work = std::max<int64_t>(max_new, 1) * p.heads * (p.dim / 8);
  const dim3 grid((unsigned)std::min<int64_t>((work + kThreads - 1) / kThreads, 1 << 16), 1, (unsigned)b.n_seq);
  (p.type == QMM_Q8 ? launch_out<QMM_Q8> : p.type == QMM_F16 ? launch_out<QMM_F16> : launch_out<QMM_BF16>)(p, b, type, k,
                                                                                                         v, grid, s);
  return hipGetLastError();
}

}  // namespace qmm
