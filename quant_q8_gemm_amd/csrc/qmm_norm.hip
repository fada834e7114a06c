// qmm_norm.hip -- what stands between two blocks of a layer: the norm after a
// block, its gate, the scaled residual sum, and the norm before the next block
// with its quantization into the q8 blocks the MMQ reads.
//
//   u = gate * norm(y);  s = rs*h + bs*u;  n = norm(s);  q8 blocks of n
//
// Every element is read once and written once; a row's statistics need the
// whole row, so a work-group owns a row and keeps it in registers between the
// passes.  The mean square (RMS) or the mean and then the mean of the squared
// deviations (layer) are summed in f32: per thread, over the wave, over the
// waves, always in the same order.
//
// Its bytes bound it, of one row the launch.  In a graph, without a post-norm: 3314 x
// 4096 f32 to the sum and q8 blocks, 178 MB, 28.8 us (35.9 at a copy's 4.96 TB/s from
// memory; part of it comes from the cache); 509 x 11008 f16 layer norm to the sum and
// numbers, 45 MB, 9.3 to 10.1; one row of 4096 2.9 to 3.3 (an empty launch: 2.1).  A row's
// own path bounds the few-row launches: 512 x 5120 bf16 with a post-norm and a gate
// takes 7.2 for 3.8 of bytes.
//
// The statistics are f32 throughout; 1/sqrt is the hardware's, an ulp off, of a mean
// formed with a rounded 1/id: about an ulp that a whole row shares.
#include "qmm_internal.h"
#include "qmm_common.h"
#include "qmm_quant.h"

#include <algorithm>

namespace qmm {

namespace {

constexpr int kMaxThreads = 1024;
constexpr int kMaxWaves = kMaxThreads / 64;

// Sum over the wave's 64 lanes, in every lane: four DPP steps give each row of
// 16 its sum, the four rows are added in order.
__device__ __forceinline__ float dpp_add(float v, int moved) { return v + __builtin_bit_cast(float, moved); }
__device__ __forceinline__ float wave_sum(float v) {
  v = dpp_add(v, dpp<kDppQuadXor1>(__builtin_bit_cast(int, v)));
  v = dpp_add(v, dpp<kDppQuadXor2>(__builtin_bit_cast(int, v)));
  v = dpp_add(v, dpp<kDppHalfMirror>(__builtin_bit_cast(int, v)));
  v = dpp_add(v, dpp<kDppMirror>(__builtin_bit_cast(int, v)));
  const int b = __builtin_bit_cast(int, v);
  const float r0 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 0));
  const float r1 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 16));
  const float r2 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 32));
  const float r3 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 48));
  return (r0 + r1) + (r2 + r3);
}

// Sum over the work-group; `red` is used by this one sum only.
__device__ __forceinline__ float group_sum(float v, float* red) {
  v = wave_sum(v);
  const int waves = blockDim.x >> 6;
  if (waves == 1) return v;
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = red[0];
  for (int w = 1; w < waves; ++w) s += red[w];
  return s;
}

struct Stats {
  float mean, rstd;
};

// 1/sqrt of a mean square.  NaN where the squares did not add up in f32: the 0 that
// 1/sqrt of infinity is would make clean zeros of such a row.
__device__ __forceinline__ float inverse_root(float square) {
  return square < __builtin_inff() ? rsqrtf(square) : __builtin_nanf("");
}

// Eight consecutive elements of a row in one thread.
struct Oct {
  float4 a, b;
};
template <class F>
__device__ __forceinline__ Oct each(const Oct& x, F&& f) {
  return {make_float4(f(x.a.x), f(x.a.y), f(x.a.z), f(x.a.w)), make_float4(f(x.b.x), f(x.b.y), f(x.b.z), f(x.b.w))};
}
template <class F>
__device__ __forceinline__ Oct each(const Oct& x, const Oct& y, F&& f) {
  return {make_float4(f(x.a.x, y.a.x), f(x.a.y, y.a.y), f(x.a.z, y.a.z), f(x.a.w, y.a.w)),
          make_float4(f(x.b.x, y.b.x), f(x.b.y, y.b.y), f(x.b.z, y.b.z), f(x.b.w, y.b.w))};
}
__device__ __forceinline__ Oct operator*(const Oct& x, const Oct& y) {
  return each(x, y, [](float p, float q) { return p * q; });
}
__device__ __forceinline__ Oct operator+(const Oct& x, const Oct& y) {
  return each(x, y, [](float p, float q) { return p + q; });
}
__device__ __forceinline__ float sum8(const Oct& x) {
  return ((x.a.x + x.a.y) + (x.a.z + x.a.w)) + ((x.b.x + x.b.y) + (x.b.z + x.b.w));
}

template <int TYPE>
__device__ __forceinline__ Oct load8(const void* p, int64_t i) {
  return {load4<TYPE>(p, i), load4<TYPE>(p, i + 4)};
}
template <int TYPE>
__device__ __forceinline__ void store8(void* p, int64_t i, const Oct& x) {
  store4<TYPE>(p, i, x.a);
  store4<TYPE>(p, i + 4, x.b);
}

// (x - mean)*rstd*weight + bias
__device__ __forceinline__ Oct apply(const Oct& x, const Stats& st, const Oct& weight) {
  return each(x, [&](float v) { return (v - st.mean) * st.rstd; }) * weight;
}
__device__ __forceinline__ Oct apply(const Oct& x, const Stats& st, const float* __restrict__ weight,
                                     const float* __restrict__ bias, int64_t e) {
  const Oct n = apply(x, st, load8<QMM_F32>(weight, e));
  return bias == nullptr ? n : n + load8<QMM_F32>(bias, e);
}

__device__ __forceinline__ float squares(const Oct& x, float mean) {
  return sum8(each(x, [&](float v) { return (v - mean) * (v - mean); }));
}

// What the type holds of x.
template <int TYPE>
__device__ __forceinline__ Oct rounded(const Oct& x) {
  return each(x, [](float v) { return (float)(elem_t<TYPE>)v; });
}

// Elements e .. e + 7 of token t: four lanes hold a q8 block.
__device__ __forceinline__ void store_q8(uint8_t* qact, int64_t t_pad, int id, int64_t t, int e, const Oct& n) {
  const float v[8] = {n.a.x, n.a.y, n.a.z, n.a.w, n.b.x, n.b.y, n.b.z, n.b.w};
  const Q8Part<8> r = quant_part(v);
  const int sub = threadIdx.x & 3, tt = (int)(t & 31);
  const int64_t frag = (t >> 5) * (id >> 5) + (e >> 5);
  *(uint2*)(qact + frag * 1024 + (sub >> 1) * 512 + tt * 16 + (sub & 1) * 8) = make_uint2(r.codes[0], r.codes[1]);
  if (sub == 0) *(uint32_t*)(qact + t_pad * id + frag * 128 + tt * 4) = r.pair;
}

// rs*p + bs*q, in the same two roundings wherever it is formed
__device__ __forceinline__ float sum(const qmm_norm& a, float p, float q) {
  return fmaf(a.residual_scale, p, a.block_scale * q);
}

// A padding token's zeros.
__device__ __forceinline__ void zero_q8(uint8_t* qact, int64_t t_pad, int id, int64_t t) {
  const int tt = (int)(t & 31);
  for (int c = threadIdx.x; c < id / 32; c += blockDim.x) {
    const int64_t frag = (t >> 5) * (id >> 5) + c;
    *(uint4*)(qact + frag * 1024 + tt * 16) = make_uint4(0, 0, 0, 0);
    *(uint4*)(qact + frag * 1024 + 512 + tt * 16) = make_uint4(0, 0, 0, 0);
    *(uint32_t*)(qact + t_pad * id + frag * 128 + tt * 4) = 0;
  }
}

// Work-group -> token.  A token's codes go out as 16-byte pieces, eight tokens
// to a 128-byte line.  Work-groups are dealt round-robin to the 8 XCDs, each
// with its own L2, so groups of 64 work-groups give each XCD eight consecutive
// tokens: a line's pieces meet in one L2.
__device__ __forceinline__ int64_t token_of(int b, int n) {
  const int r = b & 63;
  return (b | 63) < n ? (int64_t)(b - r) + (r & 7) * 8 + (r >> 3) : (int64_t)b;
}

struct Reduce {
  float sums[4][kMaxWaves];  // one row per sum over the work-group
};

// The row in registers: V times eight elements per thread, element
// 8*(v*threads + thread); id is a multiple of 256, so the four lanes of a q8 block
// are inside the row or outside it together.  What every row reads is loaded before the
// first reduction, at V = 1 the weights and the gate too, so that these do not wait
// behind a barrier (at V = 2 their registers would halve the rows in flight); biases
// are loaded where they are added.
template <int TYPE, int V>
__global__ void __launch_bounds__(kMaxThreads)
norm_kernel(qmm_norm a, int64_t t_pad, int n_tok, int id) {
  __shared__ Reduce red;
  const int64_t t = token_of((int)blockIdx.x, (int)gridDim.x);
  uint8_t* const qact = (uint8_t*)a.qact;
  if (t >= n_tok) {
    zero_q8(qact, t_pad, id, t);
    return;
  }
  constexpr bool kAhead = V == 1;
  const bool layer = a.kind == QMM_NORM_LAYER, out = a.normed != nullptr || qact != nullptr;
  const float inv_id = 1.0f / (float)id;
  const int e0 = 8 * threadIdx.x, step = 8 * blockDim.x;
  auto stats = [&](const Oct(&x)[V], int at) __attribute__((always_inline)) {
    Stats st{0.0f, 0.0f};
    if (layer) {
      float s = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (e0 + v * step < id) s += sum8(x[v]);
      st.mean = group_sum(s, red.sums[at]) * inv_id;
    }
    float s = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (e0 + v * step < id) s += squares(x[v], st.mean);
    st.rstd = inverse_root(group_sum(s, red.sums[at + 1]) * inv_id + a.eps);
    return st;
  };

  Oct s[V], u[V], w[V], pw[V], gt[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = e0 + v * step;
    if (e < id) {
      s[v] = load8<TYPE>(a.h, t * a.h_stride + e);
      if (a.y != nullptr) u[v] = load8<TYPE>(a.y, t * a.y_stride + e);
      if (kAhead) {
        if (a.post_weight != nullptr) pw[v] = load8<QMM_F32>(a.post_weight, e);
        if (a.gate != nullptr) gt[v] = load8<TYPE>(a.gate, t * a.gate_stride + e);
        if (out) w[v] = load8<QMM_F32>(a.weight, e);
      }
    }
  }
  if (a.y != nullptr) {
    if (a.post_weight != nullptr) {
      const Stats st = stats(u, 0);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int e = e0 + v * step;
        if (e < id) {
          u[v] = apply(u[v], st, kAhead ? pw[v] : load8<QMM_F32>(a.post_weight, e));
          if (a.post_bias != nullptr) u[v] = u[v] + load8<QMM_F32>(a.post_bias, e);
        }
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = e0 + v * step;
      if (e < id) {
        if (a.gate != nullptr) u[v] = u[v] * (kAhead ? gt[v] : load8<TYPE>(a.gate, t * a.gate_stride + e));
        s[v] = rounded<TYPE>(each(s[v], u[v], [&](float p, float q) { return sum(a, p, q); }));
      }
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) s[v] = rounded<TYPE>(each(s[v], [&](float p) { return p * a.residual_scale; }));
  }
  if (a.h_out != nullptr) {
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (e0 + v * step < id) store8<TYPE>(a.h_out, t * a.h_out_stride + e0 + v * step, s[v]);
  }
  if (!out) return;
  const Stats st = stats(s, 2);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = e0 + v * step;
    if (e < id) {
      Oct n = apply(s[v], st, kAhead ? w[v] : load8<QMM_F32>(a.weight, e));
      if (a.bias != nullptr) n = n + load8<QMM_F32>(a.bias, e);
      if (a.normed != nullptr) store8<TYPE>(a.normed, t * a.normed_stride + e, n);
      if (qact != nullptr) store_q8(qact, t_pad, id, t, e, n);
    }
  }
}

// Rows too long for the registers: every pass reads its operands again.  The sum
// is read back from h_out where it is stored (a thread reads only what it wrote)
// and formed again from h and y where it is not.
template <int TYPE>
__global__ void __launch_bounds__(kMaxThreads)
norm_long_kernel(qmm_norm a, int64_t t_pad, int n_tok, int id) {
  __shared__ Reduce red;
  const int64_t t = token_of((int)blockIdx.x, (int)gridDim.x);
  uint8_t* const qact = (uint8_t*)a.qact;
  if (t >= n_tok) {
    zero_q8(qact, t_pad, id, t);
    return;
  }
  const bool layer = a.kind == QMM_NORM_LAYER;
  const float inv_id = 1.0f / (float)id;
  const int e0 = 8 * threadIdx.x, step = 8 * blockDim.x;
  auto stats = [&](auto&& get, int at) __attribute__((always_inline)) {
    Stats st{0.0f, 0.0f};
    if (layer) {
      float s = 0.0f;
      for (int e = e0; e < id; e += step) s += sum8(get(e));
      st.mean = group_sum(s, red.sums[at]) * inv_id;
    }
    float s = 0.0f;
    for (int e = e0; e < id; e += step) s += squares(get(e), st.mean);
    st.rstd = inverse_root(group_sum(s, red.sums[at + 1]) * inv_id + a.eps);
    return st;
  };
  Stats post{0.0f, 0.0f};
  if (a.y != nullptr && a.post_weight != nullptr)
    post = stats([&](int e) { return load8<TYPE>(a.y, t * a.y_stride + e); }, 0);
  auto form = [&](int e) __attribute__((always_inline)) {
    Oct s = load8<TYPE>(a.h, t * a.h_stride + e);
    if (a.y == nullptr) return rounded<TYPE>(each(s, [&](float p) { return p * a.residual_scale; }));
    Oct u = load8<TYPE>(a.y, t * a.y_stride + e);
    if (a.post_weight != nullptr) u = apply(u, post, a.post_weight, a.post_bias, e);
    if (a.gate != nullptr) u = u * load8<TYPE>(a.gate, t * a.gate_stride + e);
    return rounded<TYPE>(each(s, u, [&](float p, float q) { return sum(a, p, q); }));
  };
  if (a.h_out != nullptr)
    for (int e = e0; e < id; e += step) store8<TYPE>(a.h_out, t * a.h_out_stride + e, form(e));
  if (a.normed == nullptr && qact == nullptr) return;
  auto kept = [&](int e) __attribute__((always_inline)) {
    return a.h_out != nullptr ? load8<TYPE>(a.h_out, t * a.h_out_stride + e) : form(e);
  };
  const Stats st = stats(kept, 2);
  for (int e = e0; e < id; e += step) {
    const Oct n = apply(kept(e), st, a.weight, a.bias, e);
    if (a.normed != nullptr) store8<TYPE>(a.normed, t * a.normed_stride + e, n);
    if (qact != nullptr) store_q8(qact, t_pad, id, t, e, n);
  }
}

template <int TYPE>
hipError_t launch_typed(const qmm_norm& a, int64_t n_tok, int64_t t_pad, int64_t id, hipStream_t s) {
  const dim3 grid((unsigned)std::max(n_tok, t_pad));
  // threads for V groups of eight per thread, in whole waves
  const auto threads = [&](int v) { return dim3((unsigned)((id / 8 + v * 64 - 1) / (v * 64) * 64)); };
  if (id > 4 * 8 * kMaxThreads)
    norm_long_kernel<TYPE><<<grid, dim3(kMaxThreads), 0, s>>>(a, t_pad, (int)n_tok, (int)id);
  else if (id > 2 * 8 * kMaxThreads)
    norm_kernel<TYPE, 4><<<grid, threads(4), 0, s>>>(a, t_pad, (int)n_tok, (int)id);
  else if (id > 8 * kMaxThreads)
    norm_kernel<TYPE, 2><<<grid, threads(2), 0, s>>>(a, t_pad, (int)n_tok, (int)id);
  else
    norm_kernel<TYPE, 1><<<grid, threads(1), 0, s>>>(a, t_pad, (int)n_tok, (int)id);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_norm(const qmm_norm& a, int64_t n_tok, int64_t t_pad, int64_t id, hipStream_t s) {
  return a.type == QMM_F32   ? launch_typed<QMM_F32>(a, n_tok, t_pad, id, s)
         : a.type == QMM_F16 ? launch_typed<QMM_F16>(a, n_tok, t_pad, id, s)
                             : launch_typed<QMM_BF16>(a, n_tok, t_pad, id, s);
}

}  // namespace qmm
