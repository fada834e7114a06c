// qmm_epilogue.h -- the epilogue of a product, shared by the MMQ and the
// few-token product: from the f32 sum v of output element (token t, row j),
//
//   scale * mul[t][j] * act(v + bias[j]) + residual_scale * residual[t][j]
//
// in f32, rounded once to the output's type (or quantized with its 32-block).
#pragma once

#include "qmm_common.h"
#include "qmm_quant.h"

#include "../../include/qmm.h"

#include <type_traits>

namespace qmm {

// A kernel without an epilogue: its outputs are the f32 sums themselves.
struct NoEpilogue {
  static constexpr bool kOn = false;
};

// The caller's epilogue and output, checked; strides in elements (up to 2^24).
struct Epilogue {
  static constexpr bool kOn = true;
  const float* bias;     // or nullptr
  const void* mul;       // or nullptr
  const void* residual;  // or nullptr
  void* out;
  int64_t t_pad;  // QMM_Q8: tokens of the output's qact buffer
  int mul_stride, residual_stride, out_stride;
  float scale, residual_scale;
  int act;
  int side_type;  // element type of mul and residual
  int out_type;   // element type of out, or QMM_Q8
};

// x * sigmoid(z).  No cancellation on either side: exp(-z) overflows to infinity for
// large negative z and its reciprocal is then 0.  The exponential's argument is rounded,
// so for negative z the relative error grows as about 2|z| units of 2^-24.
__device__ __forceinline__ float times_sigmoid(float x, float z) {
  return x * __builtin_amdgcn_rcpf(1.0f + __expf(-z));
}

// x * Phi(x), Phi the normal distribution function.  For a = |x|, Phi(-a) =
// exp(-a^2/2) * R(a) with a smooth R, fitted as t*P(t), t = 1/(1 + 0.3a), P of degree
// 7 with the least relative error over 0 <= a <= 14.5 (1.7e-7; beyond, the
// exponential is zero in f32).  In f32 the fit's roundings add some 10 units of 2^-24 and
// the exponential's argument about a^2: the negative tail is right to 7e-7 for a up to
// 3, 2e-6 up to 6 and 8e-6 up to 13, relative to itself.
// The library's erfc cost 9% of a product of 11008 x 4096 by 3314 tokens.
__device__ __forceinline__ float gelu(float x) {
  const float a = fabsf(x);
  const float t = __builtin_amdgcn_rcpf(fmaf(0.3f, a, 1.0f));
  float p = 3.542385948e-02f;
  p = fmaf(p, t, -1.561589360e-01f);
  p = fmaf(p, t, 2.045575700e-01f);
  p = fmaf(p, t, -5.203468462e-02f);
  p = fmaf(p, t, 1.276920947e-01f);
  p = fmaf(p, t, 1.001758594e-01f);
  p = fmaf(p, t, 1.207121488e-01f);
  p = fmaf(p, t, 1.196320065e-01f);
  const float tail = p * t * __expf(-0.5f * a * a);
  return x * (x < 0.0f ? tail : 1.0f - tail);
}

__device__ __forceinline__ float activate(float x, int act) {
  switch (act) {
    case QMM_ACT_RELU: return __builtin_elementwise_maximum(x, 0.0f);  // NaN stays NaN
    case QMM_ACT_SILU: return times_sigmoid(x, x);
    case QMM_ACT_GELU: return gelu(x);
    case QMM_ACT_GELU_TANH:  // 0.5*x*(1 + tanh(z)) = x*sigmoid(2z), z = sqrt(2/pi)*(x + 0.044715*x^3)
      return times_sigmoid(x, 1.5957691f * (x + 0.044715f * x * x * x));
    default: return x;
  }
}

// Rows j .. j + 3 of a token's row of mul, residual or out, at element offset i, of
// any alignment; n of them exist: one access where all four do, else one each.  As
// loaded, one element per word or, all four of 16 bits, two: a conversion would wait
// for the load where it stands.  Words without an element stay unset, as a zero would
// wait for loads in flight to the same register.
struct Side {
  uint32_t w[4];
};
template <int TYPE>
__device__ __forceinline__ Side load_typed(const void* p, int64_t i, int n) {
  typedef std::conditional_t<TYPE == QMM_F32, uint32_t, uint16_t> B;
  typedef B v4 __attribute__((ext_vector_type(4)));
  typedef v4 any __attribute__((aligned(sizeof(B))));
  const B* const q = (const B*)p + i;
  Side s;
  if (n == 4) {
    const v4 v = *(const any*)q;
    if constexpr (TYPE == QMM_F32) {
      s.w[0] = v.x;
      s.w[1] = v.y;
      s.w[2] = v.z;
      s.w[3] = v.w;
    } else {
      const uint2 u = __builtin_bit_cast(uint2, v);
      s.w[0] = u.x;
      s.w[1] = u.y;
    }
  } else {
#pragma unroll
    for (int k = 0; k < 3; ++k)
      if (k < n) s.w[k] = q[k];
  }
  return s;
}
__device__ __forceinline__ Side load_side(const void* p, int type, int64_t i, int n) {
  return type == QMM_F32 ? load_typed<QMM_F32>(p, i, n) : load_typed<QMM_F16>(p, i, n);  // bf16: the same bits
}
__device__ __forceinline__ float side_value(uint32_t w, int type, int half) {
  if (type == QMM_BF16) return __uint_as_float(half ? w & 0xFFFF0000u : w << 16);
  return f16_bits_to_float((half ? w >> 16 : w) & 0xFFFF);
}
__device__ __forceinline__ float4 side_values(const Side& s, int type, int n) {
  if (type == QMM_F32)
    return make_float4(__uint_as_float(s.w[0]), __uint_as_float(s.w[1]), __uint_as_float(s.w[2]), __uint_as_float(s.w[3]));
  const bool two = n == 4;
  return make_float4(side_value(s.w[0], type, 0), two ? side_value(s.w[0], type, 1) : side_value(s.w[1], type, 0),
                     side_value(two ? s.w[1] : s.w[2], type, 0), side_value(s.w[1], type, 1));
}

// What the epilogue of rows j .. j + 3 of one token reads, n of which exist; parts that
// the epilogue has not stay unset.
struct Sides {
  Side bias, mul, residual;
  int n;
};
__device__ __forceinline__ Sides load_sides(const Epilogue& ep, int t, int j, int n) {
  Sides s;
  s.n = n;
  if (ep.bias != nullptr) s.bias = load_typed<QMM_F32>(ep.bias, j, n);
  if (ep.mul != nullptr) s.mul = load_side(ep.mul, ep.side_type, (int64_t)t * ep.mul_stride + j, n);
  if (ep.residual != nullptr) s.residual = load_side(ep.residual, ep.side_type, (int64_t)t * ep.residual_stride + j, n);
  return s;
}

// The epilogue of those rows' sums.
__device__ __forceinline__ float4 finish(const Epilogue& ep, float4 v, const Sides& side) {
  if (ep.bias != nullptr) {
    const float4 b = side_values(side.bias, QMM_F32, side.n);
    v = make_float4(v.x + b.x, v.y + b.y, v.z + b.z, v.w + b.w);
  }
  if (ep.act != QMM_ACT_NONE)
    v = make_float4(activate(v.x, ep.act), activate(v.y, ep.act), activate(v.z, ep.act), activate(v.w, ep.act));
  v = make_float4(v.x * ep.scale, v.y * ep.scale, v.z * ep.scale, v.w * ep.scale);
  if (ep.mul != nullptr) {
    const float4 m = side_values(side.mul, ep.side_type, side.n);
    v = make_float4(v.x * m.x, v.y * m.y, v.z * m.z, v.w * m.w);
  }
  if (ep.residual != nullptr) {
    const float s = ep.residual_scale;
    const float4 r = side_values(side.residual, ep.side_type, side.n);
    v = make_float4(fmaf(s, r.x, v.x), fmaf(s, r.y, v.y), fmaf(s, r.z, v.z), fmaf(s, r.w, v.w));
  }
  return v;
}

template <int TYPE>
__device__ __forceinline__ void put_typed(void* p, const float4& v, int64_t i, int n) {
  if (n == 4) {
    store4_any<TYPE>(p, i, v);
  } else {
    const float f[3] = {v.x, v.y, v.z};
#pragma unroll
    for (int k = 0; k < 3; ++k)
      if (k < n) store1<TYPE>(p, i + k, f[k]);
  }
}
__device__ __forceinline__ void put(const Epilogue& ep, float4 v, int t, int j, int n) {
  const int64_t i = (int64_t)t * ep.out_stride + j;
  if (ep.out_type == QMM_F32) put_typed<QMM_F32>(ep.out, v, i, n);
  else if (ep.out_type == QMM_F16) put_typed<QMM_F16>(ep.out, v, i, n);
  else put_typed<QMM_BF16>(ep.out, v, i, n);
}

// Into the next product's qact (od/32 chunks): one lane's four codes of rows
// 32*block + 4*quad .. of token t, and from quad 0 the chunk's (dh, s) pair.
__device__ __forceinline__ void put_q8(const Epilogue& ep, const Q8Quad& r, int t, int block, int od, int quad) {
  const int64_t frag = (int64_t)(t >> 5) * (od >> 5) + block;
  *(uint32_t*)((uint8_t*)ep.out + frag * 1024 + (quad >> 2) * 512 + (t & 31) * 16 + (quad & 3) * 4) = r.codes;
  if (quad == 0) *(uint32_t*)((uint8_t*)ep.out + ep.t_pad * od + frag * 128 + (t & 31) * 4) = r.pair;
}

// The zeros of padding token t there: half of its codes, and with half 0 its pair.
__device__ __forceinline__ void zero_q8(const Epilogue& ep, int t, int block, int od, int half) {
  const int64_t frag = (int64_t)(t >> 5) * (od >> 5) + block;
  *(uint4*)((uint8_t*)ep.out + frag * 1024 + half * 512 + (t & 31) * 16) = make_uint4(0, 0, 0, 0);
  if (half == 0) *(uint32_t*)((uint8_t*)ep.out + ep.t_pad * od + frag * 128 + (t & 31) * 4) = 0;
}

}  // namespace qmm
