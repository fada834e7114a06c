// qmm_quant.h -- the arithmetic of one q8 block of 32 activations, shared by every
// kernel that writes such blocks: eight lanes hold a block, four consecutive
// values each (lanes 8i .. 8i + 7 of a wave).
#pragma once

#include "qmm_common.h"

namespace qmm {

// DPP controls: swap neighbours in a quad, swap pairs in a quad, and mirror
// each half-row of 8 lanes (lane i <-> 7 - i).  After the two quad steps every
// lane of a quad holds the quad's result, so the mirror step combines the two
// quads of an aligned group of 8 lanes.
constexpr int kDppQuadXor1 = 0xB1;     // quad_perm [1, 0, 3, 2]
constexpr int kDppQuadXor2 = 0x4E;     // quad_perm [2, 3, 0, 1]
constexpr int kDppHalfMirror = 0x141;  // row_half_mirror
constexpr int kDppMirror = 0x140;      // row_mirror: lane i <-> 15 - i of each row of 16

template <int CTRL>
__device__ __forceinline__ int dpp(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xf, 0xf, false);
}

// The larger of two magnitudes, NaN where one is (fmaxf would drop it, and a block that
// holds NaN would come out as numbers).
__device__ __forceinline__ float larger(float a, float b) { return __builtin_elementwise_maximum(fabsf(a), fabsf(b)); }

// Maximum of non-negative floats over the 8 lanes, on their bit patterns (ordered
// like the values, NaN last), so each step is one integer max.
__device__ __forceinline__ float max8(float v) {
  uint32_t u = __builtin_bit_cast(uint32_t, v);
  u = max(u, (uint32_t)dpp<kDppQuadXor1>((int)u));
  u = max(u, (uint32_t)dpp<kDppQuadXor2>((int)u));
  u = max(u, (uint32_t)dpp<kDppHalfMirror>((int)u));
  return __builtin_bit_cast(float, u);
}

__device__ __forceinline__ int sum8(int v) {
  v += dpp<kDppQuadXor1>(v);
  v += dpp<kDppQuadXor2>(v);
  return v + dpp<kDppHalfMirror>(v);
}

// q = clamp(rint(v / dh), -127, 127) where v / dh is the correctly rounded f32
// quotient (IEEE division) and rint rounds half to even.  The correctly rounded
// division costs about a dozen instructions, so the quotient is first formed as
// v * rcp(dh): with |v / dh| <= 127.1 (|v| <= amax, dh = f16(amax/127)) the
// reciprocal (1 ulp) and the product (0.5 ulp) put it within 2.3e-5 of the
// exact quotient, and the correctly rounded quotient is within 3.8e-6 of it.
// So unless the product lies within 1e-4 of a half-integer, both round to the
// same integer; when one of a lane's four products does, the lane divides all
// four exactly.  With dh == 0 the reciprocal is taken as 0, which gives q = 0.
__device__ __forceinline__ void quant4(const float4& v, float dhf, float inv, int q[4]) {
  const float r[4] = {v.x * inv, v.y * inv, v.z * inv, v.w * inv};
  float n[4], e[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    n[i] = __builtin_rintf(r[i]);
    e[i] = fabsf(r[i] - n[i]);
  }
  if (fmaxf(fmaxf(e[0], e[1]), fmaxf(e[2], e[3])) > 0.5f - 1e-4f) {
    n[0] = __builtin_rintf(v.x / dhf);
    n[1] = __builtin_rintf(v.y / dhf);
    n[2] = __builtin_rintf(v.z / dhf);
    n[3] = __builtin_rintf(v.w / dhf);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = (int)__builtin_amdgcn_fmed3f(n[i], -127.0f, 127.0f);
}

// The scale of a block whose largest magnitude is amax.
struct Q8Scale {
  _Float16 dh;
  float dhf, inv;
  __device__ __forceinline__ explicit Q8Scale(float amax) : Q8Scale((_Float16)(amax / 127.0f)) {}  // nearest even
  __device__ __forceinline__ explicit Q8Scale(_Float16 scale) {
    dh = scale;
    dhf = (float)dh;
    inv = dhf == 0.0f ? 0.0f : __builtin_amdgcn_rcpf(dhf);
  }
  // the (dh, s) word of the scale plane; S is the sum of the block's codes
  __device__ __forceinline__ uint32_t pair(int S) const {
    const _Float16 s = (_Float16)(dhf * (float)S);  // the product is exact in f32
    return (uint32_t)__builtin_bit_cast(uint16_t, dh) | ((uint32_t)__builtin_bit_cast(uint16_t, s) << 16);
  }
};

__device__ __forceinline__ uint32_t pack4(const int q[4]) {
  return (uint32_t)(q[0] & 255) | ((uint32_t)(q[1] & 255) << 8) | ((uint32_t)(q[2] & 255) << 16) |
         ((uint32_t)(q[3] & 255) << 24);
}

// One lane's part of a q8 block: its four codes, one per byte, and the block's
// (dh, s) word (the same in all eight lanes).
struct Q8Quad {
  uint32_t codes, pair;
};

__device__ __forceinline__ Q8Quad quant_quad(const float4& v) {
  const Q8Scale sc(max8(larger(larger(v.x, v.y), larger(v.z, v.w))));
  int q[4];
  quant4(v, sc.dhf, sc.inv, q);
  return {pack4(q), sc.pair(sum8(q[0] + q[1] + q[2] + q[3]))};
}

// The same block with N = 8 consecutive values per lane, four lanes (4i .. 4i + 3), or
// 16, two lanes: less shared work per value, and cheaper forms of the same numbers:
//  * amax/127 with one Newton step on the quotient's remainder, q + (a - 127q)/127
//    (Markstein): the correctly rounded quotient for every finite f32 whose
//    quotient is normal (checked for every significand; smaller ones round to a
//    scale of zero either way);
//  * v/dh with the same step from r = v * inv, which is 2.5 units of its last place
//    (ulp) off at most.  The remainder e = v - r*dh is exact: with dh's 11-bit
//    significand it is a few thousand times the product of the two last places.  So
//    r + e*inv is the quotient to 2^-20 ulp before its rounding, while a quotient of
//    24 by 11 bits is never a midpoint of two f32 and at least 2^-12 ulp away from
//    one: rounded once, it is the correctly rounded quotient.  (e underflows only
//    where |v| is far below dh/2 and the code is 0.)  Asking instead whether any
//    value is near a tie costs as much and sends most work-groups through a division;
//  * codes rounded by adding 1.5 * 2^23, whose sum holds the integer (half to
//    even) in its low bits;
//  * no clamp where dh is a normal f16: dh is then amax/127 to 2^-11, so that no
//    quotient exceeds 127.07 and rounds above 127.
template <int N>
struct Q8Part {
  uint32_t codes[N / 4], pair;
};

template <int N>
__device__ __forceinline__ Q8Part<N> quant_part(const float (&v)[N]) {
  static_assert(N == 8 || N == 16, "four or two lanes");
  constexpr float kRound = 12582912.0f;      // 1.5 * 2^23
  constexpr float kHalfMin = 6.103515625e-5f;  // the smallest normal f16
  float top = fabsf(v[0]);
#pragma unroll
  for (int i = 1; i < N; ++i) top = larger(top, v[i]);
  uint32_t u = __builtin_bit_cast(uint32_t, top);
  u = max(u, (uint32_t)dpp<kDppQuadXor1>((int)u));
  if (N == 8) u = max(u, (uint32_t)dpp<kDppQuadXor2>((int)u));
  const float amax = __builtin_bit_cast(float, u);
  const float q0 = amax * (1.0f / 127.0f);
  const Q8Scale sc((_Float16)fmaf(fmaf(-127.0f, q0, amax), 1.0f / 127.0f, q0));
  float n[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float r = v[i] * sc.inv;
    n[i] = fmaf(fmaf(-r, sc.dhf, v[i]), sc.inv, r);
  }
  if (sc.dhf < kHalfMin) {
#pragma unroll
    for (int i = 0; i < N; ++i) n[i] = __builtin_amdgcn_fmed3f(n[i], -127.0f, 127.0f);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) n[i] += kRound;
  Q8Part<N> r;
  int S = 0;
#pragma unroll
  for (int k = 0; k < N / 4; ++k) {
    const uint32_t a = __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, n[4 * k + 1]),
                                             __builtin_bit_cast(uint32_t, n[4 * k]), 0x0C0C0400u);
    const uint32_t b = __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, n[4 * k + 3]),
                                             __builtin_bit_cast(uint32_t, n[4 * k + 2]), 0x04000C0Cu);
    r.codes[k] = a | b;
    S = __builtin_amdgcn_sdot4((int)r.codes[k], 0x01010101, S, false);
  }
  S += dpp<kDppQuadXor1>(S);
  if (N == 8) S += dpp<kDppQuadXor2>(S);
  r.pair = sc.pair(S);
  return r;
}

}  // namespace qmm
