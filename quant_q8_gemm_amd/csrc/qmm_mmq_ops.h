// qmm_mmq_ops.h -- what the MMQ kernels share: the weight operands of a chunk, the
// matrix-core products and scales of a block dot, and the epilogue's layout.
#pragma once

#include "qmm_common.h"
#include "qmm_epilogue.h"
#include "qmm_internal.h"

namespace qmm {

// Weight fragment bytes per (32-row block, chunk): q6_K hi and lo planes of
// 1 KiB each; q4_K codes (16 bytes per lane).
template <int TYPE>
constexpr int kFragA = TYPE == QMM_Q6_K ? 2048 : TYPE == QMM_Q4_K_PACKED ? kQ4PackedFrag : kQ4CodeFrag;

// q4_K's stage record of one 32-row block (the wsm plane's 1 KiB record): the
// stage's 4 scales and the super-block's 8 mins as f16 integers, d*2^25 and
// -dmin in f32.
struct Q4Rec {
  uint16_t sc[32][4];     // [row][chunk of the stage]
  uint16_t mn[2][32][4];  // [chunk/4][row][chunk%4] of the super-block
  float d[2][32];         // [d*2^25, -dmin][row]
};
static_assert(sizeof(Q4Rec) == kQ4RecBytes && __builtin_offsetof(Q4Rec, mn) == kQ4RecMnOff &&
                  __builtin_offsetof(Q4Rec, d) == kQ4RecDOff,
              "the record as the repack writes it");

// The weight side of one chunk: the MFMA operand(s) read from a stage, the
// MFMA(s) against the activation fragment, and the scale-carrying block dot J
// of output element i.
template <int TYPE>
struct WeightOps;

template <>
struct WeightOps<QMM_Q6_K> {
  struct A { v4i hi, lo; };
  struct D { v16i hi, lo; };
  static constexpr int kMfma = 2;
  __device__ static A load(const int8_t* frag, int lane) {
    return {*(const v4i*)(frag + lane * 16), *(const v4i*)(frag + 1024 + lane * 16)};
  }
  __device__ static D mma(const A& a, v4i bq) {
    const v16i zero = {};
    return {__builtin_amdgcn_mfma_i32_32x32x32_i8(a.hi, bq, zero, 0, 0, 0),
            __builtin_amdgcn_mfma_i32_32x32x32_i8(a.lo, bq, zero, 0, 0, 0)};
  }
  __device__ static void keep(D& d) { pin(d.hi); pin(d.lo); }
  // the scale-folded block dot J of output element i, as an f32 (exact: |J| < 2^24)
  __device__ static float val(const D& d, int i) { return (float)((d.hi[i] << 6) + d.lo[i]); }
};

// q4_K block dots come out of the matrix core biased: the accumulator input is
// the bit pattern of the f32 value kQ4Bias (1/(2 pi), encoded as an inline
// constant of the instruction, so it costs no register), and since the code dot
// |D| <= 32*15*127 = 60960 is far inside the 2291075 steps below and 6097533
// above it that its binade [1/8, 1/4) holds, the f32 value of the result's bits
// is kQ4Bias + D*2^-26 exactly.  Subtracting kQ4Bias is exact (both within a
// factor of two), so val() = D*2^-26 with one full-rate subtraction, written
// as -(kQ4Bias - x): the subtraction then takes kQ4Bias as an inline constant
// (x - kQ4Bias would need -1/(2 pi), a 32-bit literal in every instruction),
// and the negation folds into the scale FMA's operand (it cannot be folded back
// into x - kQ4Bias: the two differ in the sign of a zero result).
// The compiler encodes the splat as the inline constant only for an MFMA whose
// accumulator input is used by no other instruction of its basic block; an
// empty asm goto after each such MFMA ends its block without emitting an
// instruction (an always-taken uniform branch did the same for two scalar
// instructions per MFMA).  Shared, the splat is materialized in 16 registers,
// which the kernel does not have.
constexpr uint32_t kQ4BiasBits = 0x3E22F983u;

template <>
struct WeightOps<QMM_Q4_K> {
  struct A { v4i c; };
  struct D { v16i c; };
  static constexpr int kMfma = 1;
  __device__ static A load(const int8_t* frag, int lane) { return {*(const v4i*)(frag + lane * 16)}; }
  __device__ static D mma(const A& a, v4i bq) {
    const v16i bias = (v16i)(int)kQ4BiasBits;
    D r;
    r.c = __builtin_amdgcn_mfma_i32_32x32x32_i8(a.c, bq, bias, 0, 0, 0);
    asm goto("" :::: block_end);
  block_end:
    return r;
  }
  __device__ static void keep(D& d) { pin(d.c); }
  // D*2^-26 of output element i; the 6-bit scale is not in it but in the scale
  // product that multiplies it (scale_outer below)
  // (the whole vector is reinterpreted: hipcc's __builtin_bit_cast of one
  // element of an ext-vector reads element 0 whatever the index)
  __device__ static float val(const D& d, int i) {
    const v16f f = __builtin_bit_cast(v16f, d.c);
    return -(__builtin_bit_cast(float, kQ4BiasBits) - f[i]);
  }
};

// q4_K with the codes kept two per byte: a lane's 8 bytes hold its 16 codes,
// code i in the low nibble of byte i and code i+8 in the high one (i < 8); two
// masks and two shifts unpack them into the 16 code bytes the MFMA takes.
// Everything after the load is q4_K's.
template <>
struct WeightOps<QMM_Q4_K_PACKED> : WeightOps<QMM_Q4_K> {
  __device__ static A load(const int8_t* frag, int lane) {
    const uint2 p = *(const uint2*)(frag + lane * 8);
    const v4i c = {(int)(p.x & 0x0F0F0F0Fu), (int)(p.y & 0x0F0F0F0Fu), (int)((p.x >> 4) & 0x0F0F0F0Fu),
                   (int)((p.y >> 4) & 0x0F0F0F0Fu)};
    return {c};
  }
};

// q4_K: the scale of output element (row j, token t) of chunk c is
// d(j)*sc(j, c) * dh(t, c); d is applied once per super-block, and the outer
// product sc(j, c)*dh(t, c) of a row vector and a token vector -- both exact f16
// values, a 6-bit integer and the f16 activation scale -- comes from one f16
// MFMA (32x32x8) in the same output layout as the int8 MFMA's block dots.  A
// holds the stage's 4 scales of the lane's row (the same 4 on both lane halves,
// k = 4*half + chunk), B the chunk's dh in slot cc of both halves and zeros
// elsewhere, so each product is formed twice and added: 2*sc*dh, exact.  That
// 2 and the block dot's 2^-26 are undone by the plane's d*2^25.
// cc is the chunk's index in the stage (a constant once the loops are unrolled).
//   a_sc      the lane's 4 f16 scales (row lane & 31, the stage's chunks)
//   dh_bits   the chunk's (dh, s) pair of the lane's token (lane & 31)
__device__ __forceinline__ v16f scale_outer(v2i a_sc, uint32_t dh_bits, int cc) {
  typedef _Float16 v4h __attribute__((ext_vector_type(4)));
  // dh into the low (cc even) or high (cc odd) half of the word, zero elsewhere
  const uint32_t y = __builtin_amdgcn_perm(0u, dh_bits, cc % 2 == 0 ? 0x0C0C0100u : 0x01000C0Cu);
  const v2i b = {cc < 2 ? (int)y : 0, cc < 2 ? 0 : (int)y};
  const v16f zero = {};
  return __builtin_amdgcn_mfma_f32_32x32x8f16(__builtin_bit_cast(v4h, a_sc), __builtin_bit_cast(v4h, b), zero,
                                              0, 0, 0);
}

// The epilogue's region of LDS: a wave's 32 x 32 sums as [token][row], token rows 36
// floats apart (both sides access 16 bytes per lane without bank conflicts).
constexpr int kEpRow = 36;
constexpr int kEpWave = 32 * kEpRow;  // floats per wave

// Zeros of a chunk of 32 padding tokens that no tile covers.
__device__ __forceinline__ void zero_block(const Epilogue& ep, int rblock, int tblock, int lane, int od) {
  const int64_t frag = (int64_t)tblock * (od >> 5) + rblock;
  *(uint4*)((uint8_t*)ep.out + frag * 1024 + lane * 16) = make_uint4(0, 0, 0, 0);
  if (lane < 32) *(uint32_t*)((uint8_t*)ep.out + ep.t_pad * od + frag * 128 + lane * 4) = 0;
}

}  // namespace qmm
