// qmm_common.h -- small device helpers shared by the library's HIP kernels.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace qmm {

typedef int v2i __attribute__((ext_vector_type(2)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v16i __attribute__((ext_vector_type(16)));
typedef float v16f __attribute__((ext_vector_type(16)));

// Empty asm that claims to modify v: the value must be produced before this
// point and cannot be recomputed after it.  Emits no instruction; used to keep
// software-pipeline stages where they are written.
template <class T>
__device__ __forceinline__ void pin(T& v) {
  asm volatile("" : "+v"(v));
}

// A pointer every lane of the wave holds, moved to scalar registers.
__device__ __forceinline__ const void* uniform_ptr(const void* p) {
  const uint64_t v = (uint64_t)p;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return (const void*)(((uint64_t)hi << 32) | lo);
}

__device__ __forceinline__ float f16_bits_to_float(uint32_t bits) {
  return (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
}

// Activations of the element types QMM_F32, QMM_F16 and QMM_BF16 (0, 1, 2),
// always computed on as f32: a conversion to f32 is exact, one back rounds to
// nearest even, once, where the value is stored.
template <int TYPE>
struct Elem;
template <>
struct Elem<0> { typedef float type; };
template <>
struct Elem<1> { typedef _Float16 type; };
template <>
struct Elem<2> { typedef __bf16 type; };
template <int TYPE>
using elem_t = typename Elem<TYPE>::type;

template <int TYPE>
__device__ __forceinline__ void store1(void* p, int64_t i, float f) {
  ((elem_t<TYPE>*)p)[i] = (elem_t<TYPE>)f;
}
// Four consecutive elements at p[i] .. p[i + 3] as one access; p + i is aligned to
// four of them (load4, store4) or only to one (store4_any: the hardware takes such
// addresses, and the compiler keeps the access whole).
template <int TYPE>
__device__ __forceinline__ float4 load4(const void* p, int64_t i) {
  typedef elem_t<TYPE> v4 __attribute__((ext_vector_type(4)));
  const v4 v = *(const v4*)((const elem_t<TYPE>*)p + i);
  return make_float4((float)v.x, (float)v.y, (float)v.z, (float)v.w);
}
template <int TYPE>
__device__ __forceinline__ void store4(void* p, int64_t i, const float4& f) {
  typedef elem_t<TYPE> T;
  typedef T v4 __attribute__((ext_vector_type(4)));
  *(v4*)((T*)p + i) = v4{(T)f.x, (T)f.y, (T)f.z, (T)f.w};
}

template <int TYPE>
__device__ __forceinline__ void store4_any(void* p, int64_t i, const float4& f) {
  typedef elem_t<TYPE> T;
  typedef T v4 __attribute__((ext_vector_type(4)));
  typedef v4 any __attribute__((aligned(sizeof(T))));
  *(any*)((T*)p + i) = v4{(T)f.x, (T)f.y, (T)f.z, (T)f.w};
}

}  // namespace qmm
