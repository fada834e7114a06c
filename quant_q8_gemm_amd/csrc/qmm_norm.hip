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

__device__ __forceinline__ float4 operator+(float4 a, float4 b) {
  return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}
__device__ __forceinline__ float4 operator*(float4 a, float4 b) {
  return make_float4(a.x * b.x, a.y * b.y, a.z * b.z, a.w * b.w);
}
__device__ __forceinline__ float4 operator*(float4 a, float b) {
  return make_float4(a.x * b, a.y * b, a.z * b, a.w * b);
}
__device__ __forceinline__ float4 operator-(float4 a, float b) {
  return make_float4(a.x - b, a.y - b, a.z - b, a.w - b);
}
__device__ __forceinline__ float sum4(float4 a) { return (a.x + a.y) + (a.z + a.w); }

// (x - mean)*rstd*weight + bias of elements e .. e + 3
__device__ __forceinline__ float4 apply(float4 x, const Stats& st, const float* __restrict__ weight,
                                        const float* __restrict__ bias, int64_t e) {
  float4 n = (x - st.mean) * st.rstd * *(const float4*)(weight + e);
  if (bias != nullptr) n = n + *(const float4*)(bias + e);
  return n;
}

// What the type holds of x.
template <int TYPE>
__device__ __forceinline__ float4 rounded(float4 x) {
  typedef elem_t<TYPE> T;
  return make_float4((float)(T)x.x, (float)(T)x.y, (float)(T)x.z, (float)(T)x.w);
}

__device__ __forceinline__ void store_q8(uint8_t* qact, int64_t t_pad, int id, int64_t t, int e, float4 n) {
  const Q8Quad r = quant_quad(n);
  const int sub = threadIdx.x & 7, tt = (int)(t & 31);
  const int64_t frag = (t >> 5) * (id >> 5) + (e >> 5);
  *(uint32_t*)(qact + frag * 1024 + (sub >> 2) * 512 + tt * 16 + (sub & 3) * 4) = r.codes;
  if (sub == 0) *(uint32_t*)(qact + t_pad * id + frag * 128 + tt * 4) = r.pair;
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

// The row in registers: V times four elements per thread, element
// 4*(v*threads + thread).  A wave's four-element groups cover 256 elements, and
// id is a multiple of 256, so a wave is inside the row or outside it whole.
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
  const bool layer = a.kind == QMM_NORM_LAYER;
  const float inv_id = 1.0f / (float)id;
  const int e0 = 4 * threadIdx.x, step = 4 * blockDim.x;
  auto stats = [&](const float4(&x)[V], int at) __attribute__((always_inline)) {
    Stats st{0.0f, 0.0f};
    if (layer) {
      float s = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (e0 + v * step < id) s += sum4(x[v]);
      st.mean = group_sum(s, red.sums[at]) * inv_id;
    }
    float s = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (e0 + v * step < id) s += sum4((x[v] - st.mean) * (x[v] - st.mean));
    st.rstd = rsqrtf(group_sum(s, red.sums[at + 1]) * inv_id + a.eps);
    return st;
  };

  float4 s[V], u[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = e0 + v * step;
    if (e < id) {
      s[v] = load4<TYPE>(a.h, t * a.h_stride + e);
      if (a.y != nullptr) u[v] = load4<TYPE>(a.y, t * a.y_stride + e);
    }
  }
  if (a.y != nullptr) {
    if (a.post_weight != nullptr) {
      const Stats st = stats(u, 0);
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (e0 + v * step < id) u[v] = apply(u[v], st, a.post_weight, a.post_bias, e0 + v * step);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = e0 + v * step;
      if (e < id) {
        if (a.gate != nullptr) u[v] = u[v] * load4<TYPE>(a.gate, t * a.gate_stride + e);
        s[v] = rounded<TYPE>(s[v] * a.residual_scale + u[v] * a.block_scale);
      }
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) s[v] = rounded<TYPE>(s[v] * a.residual_scale);
  }
  if (a.h_out != nullptr) {
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (e0 + v * step < id) store4<TYPE>(a.h_out, t * a.h_out_stride + e0 + v * step, s[v]);
  }
  if (a.normed == nullptr && qact == nullptr) return;
  const Stats st = stats(s, 2);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = e0 + v * step;
    if (e < id) {
      const float4 n = apply(s[v], st, a.weight, a.bias, e);
      if (a.normed != nullptr) store4<TYPE>(a.normed, t * a.normed_stride + e, n);
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
  const int e0 = 4 * threadIdx.x, step = 4 * blockDim.x;
  auto stats = [&](auto&& get, int at) __attribute__((always_inline)) {
    Stats st{0.0f, 0.0f};
    if (layer) {
      float s = 0.0f;
      for (int e = e0; e < id; e += step) s += sum4(get(e));
      st.mean = group_sum(s, red.sums[at]) * inv_id;
    }
    float s = 0.0f;
    for (int e = e0; e < id; e += step) {
      const float4 d = get(e) - st.mean;
      s += sum4(d * d);
    }
    st.rstd = rsqrtf(group_sum(s, red.sums[at + 1]) * inv_id + a.eps);
    return st;
  };
  Stats post{0.0f, 0.0f};
  if (a.y != nullptr && a.post_weight != nullptr)
    post = stats([&](int e) { return load4<TYPE>(a.y, t * a.y_stride + e); }, 0);
  auto form = [&](int e) __attribute__((always_inline)) {
    float4 s = load4<TYPE>(a.h, t * a.h_stride + e) * a.residual_scale;
    if (a.y != nullptr) {
      float4 u = load4<TYPE>(a.y, t * a.y_stride + e);
      if (a.post_weight != nullptr) u = apply(u, post, a.post_weight, a.post_bias, e);
      if (a.gate != nullptr) u = u * load4<TYPE>(a.gate, t * a.gate_stride + e);
      s = s + u * a.block_scale;
    }
    return rounded<TYPE>(s);
  };
  if (a.h_out != nullptr)
    for (int e = e0; e < id; e += step) store4<TYPE>(a.h_out, t * a.h_out_stride + e, form(e));
  if (a.normed == nullptr && qact == nullptr) return;
  auto sum = [&](int e) __attribute__((always_inline)) {
    return a.h_out != nullptr ? load4<TYPE>(a.h_out, t * a.h_out_stride + e) : form(e);
  };
  const Stats st = stats(sum, 2);
  for (int e = e0; e < id; e += step) {
    const float4 n = apply(sum(e), st, a.weight, a.bias, e);
    if (a.normed != nullptr) store4<TYPE>(a.normed, t * a.normed_stride + e, n);
    if (qact != nullptr) store_q8(qact, t_pad, id, t, e, n);
  }
}

template <int TYPE>
hipError_t launch_typed(const qmm_norm& a, int64_t n_tok, int64_t t_pad, int64_t id, hipStream_t s) {
  const dim3 grid((unsigned)std::max(n_tok, t_pad));
  // threads for V groups of four per thread, in whole waves
  const auto threads = [&](int v) { return dim3((unsigned)((id / 4 + v * 64 - 1) / (v * 64) * 64)); };
  if (id > 8 * 4 * kMaxThreads)
    norm_long_kernel<TYPE><<<grid, dim3(kMaxThreads), 0, s>>>(a, t_pad, (int)n_tok, (int)id);
  else if (id > 4 * 4 * kMaxThreads)
    norm_kernel<TYPE, 8><<<grid, threads(8), 0, s>>>(a, t_pad, (int)n_tok, (int)id);
  else
    norm_kernel<TYPE, 4><<<grid, threads(4), 0, s>>>(a, t_pad, (int)n_tok, (int)id);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_norm(const qmm_norm& a, int64_t n_tok, int64_t t_pad, int64_t id, hipStream_t s) {
  return a.type == QMM_F32   ? launch_typed<QMM_F32>(a, n_tok, t_pad, id, s)
         : a.type == QMM_F16 ? launch_typed<QMM_F16>(a, n_tok, t_pad, id, s)
                             : launch_typed<QMM_BF16>(a, n_tok, t_pad, id, s);
}

}  // namespace qmm
