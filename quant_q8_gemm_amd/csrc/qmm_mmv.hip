// qmm_mmv.hip -- the product for one to sixteen tokens (decode steps, speculative
// tokens, small batches), straight from the activations:
//
//   out[t][j] = epilogue( sum over 32-blocks of weight block j x q8 block of x[t] )
//
// with the arithmetic of the prepass and the MMQ: x is quantized to the same q8
// blocks, block dots are exact integers, scales are applied and summed in f32.
//
// With so few tokens the weights' bytes bound the product, so they are kept as
// small as the k-quant blocks are (the rows form: 0.5625 bytes per q4_K weight,
// 0.8203 per q6_K weight, where the MMQ's planes have 1.25 and 2.02) and every
// byte is read once, straight into registers, 16 code bytes per lane.
//
// The dots run on the matrix core although few of its 16 token rows are filled: on
// the vector ALU the 4-element dots of 8 tokens alone cost 64 cycles per 16 rows
// and 32 weights, four times the memory's pace (32000 x 4096 q6_K, 8 tokens: 58 us,
// 57% of them issuing vector instructions).  The spare token rows do a second job.
// A scale applies to 16 (q6_K) or 32 (q4_K) weights, while one MFMA sums 64; so the
// activations are laid out block-diagonally: token rows 0.. see one scale group's
// activations and zeros elsewhere, the next token rows the next group's.  One
// 16x16x64 MFMA of 16 weight rows then gives the separate dots of four groups for
// up to four tokens, of two for up to eight, of one for up to sixteen.
//
// What bounds it: a large matrix its bytes (32000 x 4096 q6_K, 108 MB: 20.4 us with
// one token, 23.0 with five, a copy's rate is 4.96 TB/s); one that the CUs hold in a
// round the path of a wave, since with sixteen of them on a CU each vector
// instruction takes 7 ns (4096 x 4096 q4_K, 9.4 MB: 4.7 us, of which the launch 2.1
// and the bytes 1.9; 11008 x 4096: 6.7, with five tokens 8.3).  From numbers, every
// work-group quantizes the activations anew, 0.2 us (16 bits) or 0.3 (f32) per 4096
// values: with many tokens and long rows q8 blocks as the input are faster (16 x 4096
// values, 4096 rows: 9.3 or 10.7 and 6.1 us, 5 x 4096: 5.8 or 6.3 and 5.2; the blocks
// themselves take a launch of 2.5).
#include "qmm_internal.h"
#include "qmm_common.h"
#include "qmm_epilogue.h"
#include "qmm_quant.h"

#include <algorithm>

namespace qmm {

// ---------------------------------------------------------------------------
// The rows form of a weight matrix: tiles of kTile rows (padding rows all zero)
// by nsb super-blocks, planes in this order, each starting at a multiple of 256
// bytes.  Byte group g (0..3) of half h (0, 1) of a block is bytes 64h + 16g ..
// + 15 of its 128 code bytes: 16 codes in the low nibbles and 16 in the high
// ones.  n is the row in its tile.
//   q4_K  codes  [tiles][nsb][h][g][n][16]
//         heads  [tiles][nsb][n][4 words]: word i holds the six-bit scale and min
//                of 32-block 2i and scale and min of 2i + 1 from its lowest bit,
//                and in its top byte one byte of f16 d (i = 0, 1) or dmin (2, 3),
//                the lower one first
//   q6_K  low    [tiles][nsb][h][g][n][16]: the block's low code bits
//         high   [tiles][nsb][g][n][h][8]: the high bits of the byte group's 32
//                codes: byte b of the first (second) four bytes holds in bits 2j,
//                2j + 1 those of the low (high) nibble's code 4j + b, the upper of
//                the two inverted
//         scales [tiles][nsb][n][16]: the int8 scales plus 128
//         d      [tiles][nsb][n] f16
// A wave's loads are whole contiguous runs: 1 KiB of codes, 1 KiB of high bits.
// ---------------------------------------------------------------------------
namespace {

constexpr int kTile = 16;

constexpr size_t round256(size_t v) { return (v + 255) / 256 * 256; }

__device__ __forceinline__ uint4 load16(const uint8_t* p) {  // 16 bytes at an even address
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = (uint32_t)*(const uint16_t*)(p + 4 * i) | ((uint32_t)*(const uint16_t*)(p + 4 * i + 2) << 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ uint4 q4k_head(const uint8_t* B) {
  const uint8_t* P = B + 4;
  uint32_t word[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t six[4];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int c = 2 * i + k;
      six[2 * k] = c < 4 ? P[c] & 63 : (P[c + 4] & 15) | ((P[c - 4] >> 6) << 4);
      six[2 * k + 1] = c < 4 ? P[c + 4] & 63 : (P[c + 4] >> 4) | ((P[c] >> 6) << 4);
    }
    word[i] = six[0] | (six[1] << 6) | (six[2] << 12) | (six[3] << 18) | ((uint32_t)B[i] << 24);
  }
  return make_uint4(word[0], word[1], word[2], word[3]);
}

// One thread per (tile, super-block, half, byte group, row), striding over a
// capped grid.
__global__ void __launch_bounds__(256)
repack_rows_kernel(const uint8_t* __restrict__ raw, int q6, int od, int nsb, int64_t total, RowPlanes r) {
  const int64_t stride = (int64_t)gridDim.x * blockDim.x;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += stride) {
    const int n = (int)(i & 15), g = (int)(i >> 4) & 3, h = (int)(i >> 6) & 1;
    const int64_t ts = i >> 7;  // tile * nsb + super-block
    const int64_t row = ts / nsb * kTile + n;
    const bool real = row < od;
    const int64_t b = (real ? row : 0) * nsb + ts % nsb;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    if (q6) {
      const uint8_t* B = raw + b * 210;
      *(uint4*)(r.codes + i * 16) = real ? load16(B + 64 * h + 16 * g) : zero;
      const uint8_t* qh = B + 128 + 32 * h + 16 * (g & 1);
      uint32_t high[2] = {0, 0};
#pragma unroll
      for (int k = 0; k < 16; ++k)
#pragma unroll
        for (int m = 0; m < 2; ++m)
          high[m] |= (uint32_t)(((qh[k] >> (2 * (g >> 1) + 4 * m)) & 3) ^ 2) << (8 * (k & 3) + 2 * (k >> 2));
      *(uint2*)(r.heads + ((ts * 4 + g) * kTile + n) * 16 + 8 * h) = real ? make_uint2(high[0], high[1]) : make_uint2(0, 0);
      if (h == 0 && g == 0) {
        uint8_t* const s = r.scales + (ts * kTile + n) * 16;
        for (int k = 0; k < 16; ++k) s[k] = real ? (uint8_t)(B[192 + k] + 128) : 0;
        r.d[ts * kTile + n] = real ? (uint16_t)(B[208] | (B[209] << 8)) : 0;
      }
    } else {
      const uint8_t* B = raw + b * 144;
      *(uint4*)(r.codes + i * 16) = real ? *(const uint4*)(B + 16 + 64 * h + 16 * g) : zero;
      if (h == 0 && g == 0) *(uint4*)(r.heads + (ts * kTile + n) * 16) = real ? q4k_head(B) : zero;
    }
  }
}

}  // namespace

int64_t row_pad(int64_t od) { return (od + kTile - 1) / kTile * kTile; }

RowOffsets row_offsets(int type, int64_t od, int64_t id) {
  const size_t nb = (size_t)row_pad(od) * (size_t)(id / 256);
  const bool q6 = type == QMM_Q6_K_ROWS;
  RowOffsets r;
  r.heads = round256(nb * 128);
  r.scales = r.heads + round256(nb * (q6 ? 64 : 16));
  r.d = r.scales + (q6 ? round256(nb * 16) : 0);
  r.bytes = r.d + (q6 ? round256(nb * 2) : 0);
  return r;
}

hipError_t launch_repack_rows(const uint8_t* raw, int type, int64_t od, int64_t id, const RowPlanes& r, hipStream_t s) {
  const int64_t total = row_pad(od) * (id / 256) * 8;
  const int64_t blocks = std::min<int64_t>((total + 255) / 256, 1 << 14);
  repack_rows_kernel<<<dim3((unsigned)blocks), dim3(256), 0, s>>>(raw, type == QMM_Q6_K_ROWS, (int)od, (int)(id / 256),
                                                                 total, r);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// The product.  A work-group of up to kWaves waves first quantizes the activations into
// LDS, the whole inner dimension where it fits; then it walks row tiles: kg of its
// waves share a tile, each over its share of the super-blocks, and the tile's
// partial sums meet in LDS, are added in wave order and go through the epilogue.
//
// The MFMA's A operand are the activations (row m: lane & 15, k group: lane >> 4,
// 16 bytes), B the weights (row n of the tile: lane & 15, the same k groups: the
// four byte groups of a half block).  Lane (n, G) of the result holds token rows
// m = 4G .. 4G + 3 of weight row n:
//   TOK = 1, 2, 4 (up to as many tokens): m = 4*group + token: lane group G has the
//     tokens of byte group G, again in its other rows;
//   TOK = 8: m = 8*half + token.  q4_K: the halves are the two 32-blocks of the half
//     block (byte groups 0, 1 and 2, 3); q6_K: two byte groups, and a second MFMA
//     with the other two;
//   TOK = 16: m = token, an MFMA per 32-block (q4_K) or byte group (q6_K).
// A lane's scales are those of its own row n.
// ---------------------------------------------------------------------------
namespace {

constexpr int kWaves = 16;

// LDS per super-block: codes [h][nibble][g][token][16]; then for q6_K f32 dh
// [32-block][token], for q4_K the prepass's pairs, f16 (dh, s) [token][32-block].  TOK
// tokens, so that a lane's addresses differ by constants; codes of n_tok tokens with
// TOK = 16, where the room is wanted.
template <int TOK>
__device__ __host__ __forceinline__ int code_slots(int n_tok) {
  return TOK == 16 ? n_tok : TOK;
}
// Tokens whose sums a lane holds.
template <int TOK>
constexpr int kAcc = TOK < 4 ? TOK : 4;
template <int TOK>
constexpr int kScaleBytes = 32 * TOK;
// MFMAs per 64 weights of a row.
template <bool Q6, int TOK>
constexpr int kPasses = Q6 ? (TOK == 16 ? 4 : TOK == 8 ? 2 : 1) : (TOK == 16 ? 2 : 1);

struct MvArgs {
  RowPlanes w;
  const void* x;
  int x_stride;  // elements; of a qact buffer: bytes of its code plane (128 tokens)
  int x_type, n_tok, od, nsb;
  int tile_sb;  // super-blocks quantized at a time
  int kg_bits;  // 2^kg_bits waves share a row tile,
  int groups;   // groups of them in a work-group
  uint32_t over_n_tok, over_per_unit;  // see over()
  int db;  // threads / 2 / n_tok
  int steps;    // sets of so many row tiles
};

// n / d for n < 1024 and d >= 1, from over(d) = ceil(2^20 / d): the product's excess
// over n / d, n / 2^20, is below 1/d, d up to 1024, and with larger d the quotient 0
// stays below 1.
inline uint32_t over(int64_t d) { return (uint32_t)(((1 << 20) + d - 1) / d); }
__device__ __forceinline__ int divide(int n, uint32_t over_d) { return (int)(__umul24(n, over_d) >> 20); }

__device__ __host__ __forceinline__ int threads_of(const MvArgs& a) { return (64 << a.kg_bits) * a.groups; }

// A lane's weights of one super-block as loaded, and the f32 factors of its dots.
template <bool Q6>
struct Raw;
template <>
struct Raw<false> {
  uint4 code[2], head;
  // ts: tile*nsb + super-block (uniform)
  __device__ __forceinline__ void load(const RowPlanes& w, int64_t ts, uint32_t lane) {
    code[0] = *(const uint4*)(w.codes + ts * 2048 + lane * 16);
    code[1] = *(const uint4*)(w.codes + ts * 2048 + 1024 + lane * 16);
    head = *(const uint4*)(w.heads + ts * 256 + (lane & 15) * 16);
  }
};
template <>
struct Raw<true> {
  uint4 code[2], high, scales;
  uint32_t d;
  __device__ __forceinline__ void load(const RowPlanes& w, int64_t ts, uint32_t lane) {
    code[0] = *(const uint4*)(w.codes + ts * 2048 + lane * 16);
    code[1] = *(const uint4*)(w.codes + ts * 2048 + 1024 + lane * 16);
    high = *(const uint4*)(w.heads + ts * 1024 + lane * 16);
    scales = *(const uint4*)(w.scales + ts * 256 + (lane & 15) * 16);
    d = *(w.d + ts * 16 + (lane & 15));
  }
};

template <int N>
using Vec = float __attribute__((ext_vector_type(N)));

// LDS by its address, so that addresses can be pinned (computed where they stand).
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const uint8_t*)p;
}
template <class T>
__device__ __forceinline__ const __attribute__((address_space(3))) T* lds_at(uint32_t address) {
  return (const __attribute__((address_space(3))) T*)(uintptr_t)address;
}

__device__ __forceinline__ v4i mfma(v4i a, v4i b) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, v4i{0, 0, 0, 0}, 0, 0, 0);
}

// acc[i] += f * (dh[i] * dot[i]): one scale group's dots of the lane's tokens
template <int N>
__device__ __forceinline__ void add_dots(float (&acc)[N], const v4i& dot, float f, uint32_t dh) {
  const Vec<N> v = *lds_at<Vec<N>>(dh);
#pragma unroll
  for (int i = 0; i < N; ++i) acc[i] = fmaf((float)dot[i] * v[i], f, acc[i]);
}
// One super-block of q4_K.  codes(h, nibble, pass): the A operand of the dots; pairs:
// the address of the lane's (dh, s) pairs of token m and 32-blocks 2G and 2G + 1, or of
// zeros where row m does not see these (m >> 3 the pair of 32-blocks a row sees, but
// with TOK = 16 all).
//
// A dot's factor scale * dh is an outer product over rows and tokens, and the min terms
// are a product over the eight 32-blocks: an MFMA each, with k = 4G + (dh, s, dh, s), B
// the scales (zeros but for the dot's 32-blocks) or the mins of a lane's two 32-blocks.
// Their six bits stand for themselves as f16 subnormals, code * 2^-24; the products are
// exact.  The vector ALU is left with two instructions per dot and token.
template <int TOK, class Codes>
__device__ __forceinline__ void add_block(const Raw<false>& w, float (&acc)[kAcc<TOK>], int G, Codes&& codes,
                                          uint32_t pairs) {
  typedef _Float16 v4h __attribute__((ext_vector_type(4)));
  typedef float v4f __attribute__((ext_vector_type(4)));
  constexpr int kN = kAcc<TOK>;
  const v4h a = *lds_at<v4h>(pairs);
  auto outer = [&](uint32_t b0, uint32_t b1) __attribute__((always_inline)) {
    return __builtin_amdgcn_mfma_f32_16x16x16f16(a, __builtin_bit_cast(v4h, make_uint2(b0, b1)),
                                                 v4f{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
  };
  // scales and mins of 32-blocks 2G and 2G + 1, see q4k_head
  const uint32_t h0 = w.head.x, h1 = w.head.y, h2 = w.head.z, h3 = w.head.w;
  const uint32_t word = G & 2 ? (G & 1 ? h3 : h2) : (G & 1 ? h1 : h0);
  const uint32_t sc0 = word & 63, sc1 = (word >> 12) & 63;
  const v4f mins = outer((word << 10) & 0x3F0000u, (word >> 2) & 0x3F0000u);
  const float d = 16777216.0f * f16_bits_to_float(__builtin_amdgcn_perm(w.head.y, w.head.x, 0x0C0C0703u));
  // up to four tokens two lane groups see the same pair
  const float m = (TOK <= 4 ? -8388608.0f : -16777216.0f) *
                  f16_bits_to_float(__builtin_amdgcn_perm(w.head.w, w.head.z, 0x0C0C0703u));
  float inner[kN] = {};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t c[4] = {w.code[h].x, w.code[h].y, w.code[h].z, w.code[h].w};
    v4i lo, hi;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lo[i] = (int)(c[i] & 0x0F0F0F0Fu);
      hi[i] = (int)((c[i] >> 4) & 0x0F0F0F0Fu);
    }
#pragma unroll
    for (int k = 0; k < kPasses<false, TOK>; ++k) {
      const bool mine = TOK == 16 ? G == 2 * h + k : G >> 1 == h;
      const v4f f0 = outer(mine ? sc0 : 0, 0), f1 = outer(0, mine ? sc1 : 0);
      const v4i d0 = mfma(codes(h, 0, k), lo), d1 = mfma(codes(h, 1, k), hi);
#pragma unroll
      for (int i = 0; i < kN; ++i) inner[i] = fmaf((float)d1[i], f1[i], fmaf((float)d0[i], f0[i], inner[i]));
      if (TOK == 16) __builtin_amdgcn_sched_barrier(0);  // a pass at a time: else registers spill
    }
  }
#pragma unroll
  for (int i = 0; i < kN; ++i) acc[i] = fmaf(mins[i], m, fmaf(inner[i], d, acc[i]));
}

// One super-block of q6_K.  A code as four times (code - 32): its six bits, the top
// one inverted, in a byte's upper bits are that as an int8; the 4 is taken off d.
template <int TOK, class Codes>
__device__ __forceinline__ void add_block(const Raw<true>& w, float (&acc)[kAcc<TOK>], int G, Codes&& codes,
                                          uint32_t dh) {
  const float d = 0.25f * f16_bits_to_float(w.d), d128 = -128.0f * d;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t c[4] = {w.code[h].x, w.code[h].y, w.code[h].z, w.code[h].w};
    const uint32_t top[2] = {h ? w.high.z : w.high.x, h ? w.high.w : w.high.y};
    v4i b[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      b[0][i] = (int)(((c[i] << 2) & 0x3C3C3C3Cu) | ((top[0] << (6 - 2 * i)) & 0xC0C0C0C0u));
      b[1][i] = (int)(((c[i] >> 2) & 0x3C3C3C3Cu) | ((top[1] << (6 - 2 * i)) & 0xC0C0C0C0u));
    }
    const uint32_t sc[2] = {h ? w.scales.z : w.scales.x, h ? w.scales.w : w.scales.y};
#pragma unroll
    for (int nib = 0; nib < 2; ++nib) {
#pragma unroll
      for (int k = 0; k < kPasses<true, TOK>; ++k) {
        // byte group g: 16-group 8h + 4*nib + g, in 32-block 4h + 2*nib + g/2
        const int g = TOK == 16 ? k : TOK == 8 ? 2 * k + (G >> 1) : G;
        const uint32_t u = (sc[nib] >> (8 * g)) & 255;
        add_dots(acc, mfma(codes(h, nib, k), b[nib]), fmaf(d, (float)u, d128),
                 dh + 4 * TOK * (4 * h + 2 * nib + (g >> 1)));
      }
    }
  }
}

// Where eight codes of a token go: k counts eights from the first of the part.
template <bool Q6>
__device__ __forceinline__ uint8_t* place(uint8_t* lds, int sb_bytes, int slots, int t, int k) {
  const int c = (k >> 2) & 7, half16 = (k >> 1) & 1;  // 32-block, its 16 codes
  const int h = c >> 2, nib = Q6 ? (c >> 1) & 1 : c & 1, g = 2 * (Q6 ? c & 1 : (c >> 1) & 1) + half16;
  return lds + (k >> 5) * sb_bytes + (((2 * h + nib) * 4 + g) * slots + t) * 16 + (k & 1) * 8;
}
template <bool Q6, int TOK>
__device__ __forceinline__ void place_scales(uint8_t* lds, int sb_bytes, int slots, int t, int k, uint32_t pair) {
  uint8_t* const s = lds + (k >> 5) * sb_bytes + 256 * slots;
  const int c = (k >> 2) & 7;
  if (Q6)
    ((float*)s)[TOK * c + t] = f16_bits_to_float(pair & 0xFFFF);
  else
    ((uint32_t*)s)[8 * t + c] = pair;
}

// The activations of super-blocks [sb0, sb0 + n) of every token into LDS.  From
// numbers: sixteen per thread, two threads per 32-block, the tokens of a block next to
// each other, as LDS has them; the next sixteen are loaded while these are quantized;
// begin() loads the first ones, so that the caller can put other loads behind them.
// Eight per thread repeat more of the shared work (4096 x 11008 q4_K, 16 tokens of bf16:
// 26.1 instead of 20.7 us, 5 of f32: 11.7 and 11.1; one token of 2048: 3.7 and 3.8).  With
// f32 the sixteen beside two super-blocks of q4_K weights are more than the registers
// hold: 2 or 3 spill from two tokens on, 14 with more than eight (6 to q8 blocks; 4096 x
// 4096, 16 tokens: 10.7 us, of bf16 9.3); from 16 bits, q8 blocks and for q6_K none do.
template <bool Q6, int TOK, int XT>
struct Quantizer {
  static constexpr int kPer = 16;
  typedef elem_t<XT> Part __attribute__((ext_vector_type(kPer)));
  Part v;                    // as loaded: a conversion would wait here
  int t, b, blocks, dt, db;  // a thread's token and 32-block of the part
  __device__ __forceinline__ void fetch(const MvArgs& a, int sb0) {
    if (b < blocks) {
      const int64_t at = (int64_t)t * a.x_stride + (sb0 * 256 + 32 * b + kPer * (int)(threadIdx.x & 1));
      typedef Part Rows __attribute__((aligned(4 * sizeof(elem_t<XT>))));  // rows start at fours
      v = *(const Rows*)((const elem_t<XT>*)a.x + at);
    }
  }
  __device__ __forceinline__ void begin(const MvArgs& a, int sb0, int n) {
    blocks = n * 8;
    b = divide(threadIdx.x >> 1, a.over_n_tok);
    t = (threadIdx.x >> 1) - __umul24(b, a.n_tok);
    db = a.db;  // the threads' stride in blocks and tokens
    dt = threads_of(a) / 2 - db * a.n_tok;
    fetch(a, sb0);
  }
  __device__ __forceinline__ void run(const MvArgs& a, uint8_t* lds, int sb_bytes, int sb0) {
    while (b < blocks) {
      float c[kPer];
#pragma unroll
      for (int i = 0; i < kPer; ++i) c[i] = (float)v[i];
      const int tok = t, at = 4 * b + 2 * (threadIdx.x & 1);
      b += db;
      t += dt;
      if (t >= a.n_tok) {
        t -= a.n_tok;
        ++b;
      }
      fetch(a, sb0);
      const Q8Part<kPer> r = quant_part(c);
      const int slots = code_slots<TOK>(a.n_tok);
      *(uint4*)place<Q6>(lds, sb_bytes, slots, tok, at) = make_uint4(r.codes[0], r.codes[1], r.codes[2], r.codes[3]);
      if ((at & 2) == 0) place_scales<Q6, TOK>(lds, sb_bytes, slots, tok, at, r.pair);
    }
  }
};

// From a qact buffer (one block of 32 tokens): 16 codes, half a 32-block, per thread,
// in a slot per token (1, 2, 4, 8 or 16 of them).
template <bool Q6, int TOK>
struct Quantizer<Q6, TOK, QMM_Q8> {
  uint4 codes;
  uint32_t pair;
  int t, half, halves, bits;
  __device__ __forceinline__ void fetch(const MvArgs& a, int sb0) {
    if (half < halves && t < a.n_tok) {
      const uint8_t* const q = (const uint8_t*)a.x;
      const uint32_t c = (uint32_t)(sb0 * 8 + (half >> 1));
      codes = *(const uint4*)(q + (size_t)c * 1024 + (half & 1) * 512 + t * 16);
      if ((half & 1) == 0) pair = *(const uint32_t*)(q + a.x_stride + (size_t)c * 128 + t * 4);
    }
  }
  __device__ __forceinline__ void begin(const MvArgs& a, int sb0, int n) {
    bits = a.n_tok > 8 ? 4 : a.n_tok > 4 ? 3 : a.n_tok > 2 ? 2 : a.n_tok > 1 ? 1 : 0;
    t = threadIdx.x & ((1 << bits) - 1);
    half = threadIdx.x >> bits;
    halves = n * 16;
    fetch(a, sb0);
  }
  __device__ __forceinline__ void run(const MvArgs& a, uint8_t* lds, int sb_bytes, int sb0) {
    while (half < halves) {
      const uint4 c = codes;
      const uint32_t pr = pair;
      const int at = 2 * half;
      half += threads_of(a) >> bits;
      fetch(a, sb0);
      if (t < a.n_tok) {
        const int n = code_slots<TOK>(a.n_tok);
        *(uint4*)place<Q6>(lds, sb_bytes, n, t, at) = c;
        if ((at & 2) == 0) place_scales<Q6, TOK>(lds, sb_bytes, n, t, at, pr);
      }
    }
  }
};

// The sum over both halves of the wave of a in the lower half, of b in the upper.
__device__ __forceinline__ float halves_sum(float a, float b) {
  const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b),
                                                  false, false);
  return __builtin_bit_cast(float, (uint32_t)r[0]) + __builtin_bit_cast(float, (uint32_t)r[1]);
}

// Of each half of the wave: the sum over its two rows of 16 lanes.
__device__ __forceinline__ float quarters_sum(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, x),
                                                  false, false);
  return __builtin_bit_cast(float, (uint32_t)r[0]) + __builtin_bit_cast(float, (uint32_t)r[1]);
}

// OUT8: the output is kept as q8 blocks (its code beside the other outputs' cost
// every call 0.9 us).
template <bool Q6, int TOK, int XT, bool OUT8>
__global__ void __launch_bounds__(64 * kWaves)
mmv_kernel(MvArgs a, Epilogue ep) {
  extern __shared__ uint4 lds_raw[];
  uint8_t* const lds = (uint8_t*)lds_raw;
  const int slots = code_slots<TOK>(a.n_tok);
  const int sb_bytes = 256 * slots + kScaleBytes<TOK>;
  // the partial sums [2][wave][token][kTile], and the codes of a super-block as zeros
  float* const red = (float*)(lds + (size_t)a.tile_sb * sb_bytes);
  uint4* const zeros = (uint4*)(red + 2 * kWaves * TOK * kTile);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kgs = 1 << a.kg_bits, rg = wave >> a.kg_bits, kg = wave & (kgs - 1), groups = a.groups;
  const int tiles = (a.od + kTile - 1) / kTile;
  const bool one_tile = a.tile_sb == a.nsb;
  const int m = lane & 15, G = lane >> 4;

  // Loads return in order, so the activations' go first.
  Quantizer<Q6, TOK, XT> quant;
  quant.begin(a, 0, a.tile_sb);
  // The wave's weights, kAhead super-blocks ahead: super-blocks kg, kg + kgs, ... of
  // its tile of this step, then of the next step's (past the last step: the last
  // step's again, unused).
  constexpr int kAhead = Q6 ? 1 : 2;
  Raw<Q6> ahead[kAhead];
  int f_step = blockIdx.x, f_sb = kg;
  auto fetch = [&](Raw<Q6>& to) __attribute__((always_inline)) {
    to.load(a.w, (int64_t)min(f_step * groups + rg, tiles - 1) * a.nsb + f_sb, (uint32_t)lane);
    f_sb += kgs;
    if (f_sb >= a.nsb) {
      f_sb = kg;
      f_step = min(f_step + (int)gridDim.x, a.steps - 1);
    }
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) fetch(ahead[i]);
  // The lane's A operand: its token's codes of its byte group G, or zeros where G is
  // not what its row sees in the pass.
  const int tok = m & (TOK - 1);
  const bool own = tok < a.n_tok && (TOK == 16 || (TOK == 8 ? (m >> 3) == (Q6 ? G & 1 : G >> 1) : (m >> 2) == G));
  const int pass = Q6 && TOK == 16 ? G : G >> 1;  // the lane's, of several
  constexpr int kPass = kPasses<Q6, TOK>;
  uint32_t first[kPass];  // LDS address, of the wave's first super-block
  int step_sb[kPass];     // to its next one
#pragma unroll
  for (int k = 0; k < kPass; ++k) {
    const bool live = own && (kPass == 1 || pass == k);
    first[k] = live ? lds_address(lds) + kg * sb_bytes + (G * slots + tok) * 16 : lds_address(zeros);
    step_sb[k] = live ? kgs * sb_bytes : 0;
    pin(first[k]);
    pin(step_sb[k]);
  }
  // Its scales: q6_K of the tokens whose sums it holds, q4_K see add_block.
  uint32_t scales = lds_address(lds) + kg * sb_bytes + 256 * slots;
  int scale_step = kgs * sb_bytes;
  if constexpr (Q6) {
    scales += 4 * (TOK == 16 ? 4 * G : TOK == 8 ? 4 * (G & 1) : 0);
  } else {
    const bool live = tok < a.n_tok && (TOK == 16 || m >> 3 == (G & 1));
    scales = live ? scales + tok * 32 + G * 8 : lds_address(zeros);
    scale_step = live ? scale_step : 0;
    pin(scale_step);
  }
  pin(scales);
  // The thread that finishes four rows of a token: of which unit, a row tile or, for
  // a q8 output, a pair of them (a 32-block: eight threads).
  constexpr int kUnit = OUT8 ? 2 : 1, kQuads = 4 * kUnit;
  const int units = groups / kUnit, per_unit = kQuads * a.n_tok;
  const int e_unit = divide(threadIdx.x, a.over_per_unit);
  const uint32_t e_at = threadIdx.x - __umul24(e_unit, per_unit);
  const int e_tok = e_at / kQuads, e_quad = e_at % kQuads;

  // Its sides, early: a step ahead, in front of the first with no quantizing to come,
  // whose registers they would take.
  auto row_of = [&](int step) __attribute__((always_inline)) { return (step * groups + e_unit * kUnit) * kTile + 4 * e_quad; };
  auto left_of = [&](int row) __attribute__((always_inline)) { return e_unit < units ? min(a.od - row, 4) : 0; };
  int row = row_of(blockIdx.x), left = left_of(row);
  Sides side;

  for (int i = threadIdx.x; i < 16 * slots; i += threads_of(a)) zeros[i] = make_uint4(0, 0, 0, 0);
  if (one_tile) quant.run(a, lds, sb_bytes, 0);
  if (!OUT8 && left > 0) side = load_sides(ep, e_tok, row, left);
  __syncthreads();

  int buf = 0;
  for (int step = blockIdx.x; step < a.steps; step += gridDim.x, buf ^= 1) {
    float acc[kAcc<TOK>] = {};
    for (int sb0 = 0; sb0 < a.nsb; sb0 += a.tile_sb) {
      const int n = min(a.tile_sb, a.nsb - sb0);
      if (!one_tile) {
        if (sb0 > 0 || step != (int)blockIdx.x) quant.begin(a, sb0, n);
        __syncthreads();  // the last part's readers are done
        quant.run(a, lds, sb_bytes, sb0);
        __syncthreads();
      }
      uint32_t at[kPass];
#pragma unroll
      for (int k = 0; k < kPass; ++k) at[k] = first[k];
      uint32_t scales_at = scales;
      for (int sb = kg; sb < n; sb += kgs) {
        const Raw<Q6> w = ahead[0];
#pragma unroll
        for (int i = 0; i + 1 < kAhead; ++i) ahead[i] = ahead[i + 1];
        fetch(ahead[kAhead - 1]);
        auto codes = [&](int h, int nib, int k) __attribute__((always_inline)) {
          return *lds_at<v4i>(at[k] + (2 * h + nib) * 64 * slots);
        };
        add_block<TOK>(w, acc, G, codes, scales_at);
#pragma unroll
        for (int k = 0; k < kPass; ++k) at[k] += step_sb[k];
        scales_at += scale_step;
      }
    }
    // the sums of the lane groups that share tokens, into [token][row]
    float* const out = red + ((size_t)buf * kWaves + wave) * (TOK * kTile) + m;
    if constexpr (TOK == 16) {
#pragma unroll
      for (int i = 0; i < 4; ++i) out[(4 * G + i) * kTile] = acc[i];
    } else if constexpr (TOK <= 2) {
      const float x = quarters_sum(halves_sum(acc[0], acc[TOK - 1]));  // upper half of the wave: the second token
      if ((G & 1) == 0) out[TOK == 2 ? (G >> 1) * kTile : 0] = x;
    } else {
      const float x = halves_sum(acc[0], acc[1]), y = halves_sum(acc[2], acc[3]);
      if constexpr (TOK == 8) {  // lower half of the wave: tokens 4*(G&1) and + 2, upper: + 1 and + 3
        const int t0 = 4 * (G & 1) + (G >> 1);
        out[t0 * kTile] = x;
        out[(t0 + 2) * kTile] = y;
      } else {  // the odd rows of 16 lanes of x and the even ones of y change places
        const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, x),
                                                        __builtin_bit_cast(uint32_t, y), false, false);
        out[((G >> 1) + 2 * (G & 1)) * kTile] =
            __builtin_bit_cast(float, (uint32_t)r[0]) + __builtin_bit_cast(float, (uint32_t)r[1]);
      }
    }
    __syncthreads();
    // two buffers: the next step's sums do not overwrite these, the one after has
    // passed the next barrier
    if (left > 0) {
      const int tile = e_unit * kUnit + (e_quad >> 2);  // of the set
      const float* p = red + ((size_t)buf * kWaves + (tile << a.kg_bits)) * (TOK * kTile) + e_tok * kTile + 4 * (e_quad & 3);
      float4 f = *(const float4*)p;
      for (int k = 1; k < kgs; ++k) {
        const float4 e = *(const float4*)(p + (size_t)k * (TOK * kTile));
        f = make_float4(f.x + e.x, f.y + e.y, f.z + e.z, f.w + e.w);
      }
      f = finish(ep, f, OUT8 ? load_sides(ep, e_tok, row, 4) : side);
      if constexpr (OUT8)
        put_q8(ep, quant_quad(f), e_tok, row >> 5, a.od, e_quad);
      else
        put(ep, f, e_tok, row, left);
    }
    if constexpr (OUT8)
      for (int i = threadIdx.x; i < units * 2 * (int)ep.t_pad; i += threads_of(a)) {  // the padding tokens' zeros
        const int t = (i >> 1) & ((int)ep.t_pad - 1), block = step * groups / 2 + i / (2 * (int)ep.t_pad);
        if (t >= a.n_tok && block < a.od >> 5) zero_q8(ep, t, block, a.od, i & 1);
      }
    row = row_of(step + gridDim.x);
    left = left_of(row);
    if (!OUT8 && left > 0) side = load_sides(ep, e_tok, row, left);
  }
}

template <bool Q6, int TOK, int XT, bool OUT8>
hipError_t launch_kernel(const MvArgs& in, const Epilogue& ep, int num_cus, hipStream_t s) {
  MvArgs a = in;
  // LDS: the whole inner dimension where it fits the CU's 160 KB, else parts of it,
  // quantized again for every set of row tiles
  constexpr size_t kMost = 160 * 1024;
  constexpr size_t kRed = (size_t)2 * kWaves * TOK * kTile * sizeof(float) + 256 * TOK;
  const size_t per_sb = (size_t)256 * code_slots<TOK>(a.n_tok) + kScaleBytes<TOK>;
  a.tile_sb = (int)std::min<size_t>(a.nsb, (kMost - kRed) / per_sb);
  if (a.tile_sb < a.nsb) a.tile_sb = a.tile_sb / kWaves * kWaves;  // a wave's super-blocks go on across parts
  const size_t lds = a.tile_sb * per_sb + kRed;
  // One work-group per CU.  Waves per row tile: as few as fill the GPU's CUs with
  // row tiles of their own, and the fewest rounds of them, counted in the
  // super-blocks that each wave walks (and half of one for the sums).
  const int64_t tiles = (a.od + kTile - 1) / kTile;
  const int most = OUT8 ? kWaves / 2 : kWaves;  // q8: row tiles in pairs
  double best = 0;
  for (int bits = 0, kg = 1; kg <= most && (kg == 1 || kg <= a.nsb); kg = 1 << ++bits) {
    const int64_t steps = (tiles + kWaves / kg - 1) / (kWaves / kg);
    const double cost = (double)((steps + num_cus - 1) / num_cus) * ((a.nsb + kg - 1) / kg + 0.5);
    if (kg == 1 || cost < best) {
      best = cost;
      a.kg_bits = bits;
    }
  }
  // Row tiles per work-group: as few as leave no more work-groups than CUs.
  const int64_t share = (tiles + num_cus - 1) / num_cus;
  a.groups = (int)std::min<int64_t>(kWaves >> a.kg_bits, OUT8 ? (share + 1) / 2 * 2 : share);
  a.steps = (int)((tiles + a.groups - 1) / a.groups);
  a.over_n_tok = over(a.n_tok);
  a.db = threads_of(a) / 2 / a.n_tok;
  a.over_per_unit = over((OUT8 ? 8 : 4) * a.n_tok);
  const int grid = (int)std::min<int64_t>(a.steps, num_cus);
  if (lds > 64 * 1024) {
    hipError_t e = hipFuncSetAttribute((const void*)mmv_kernel<Q6, TOK, XT, OUT8>, hipFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)lds);
    if (e != hipSuccess) return e;
  }
  mmv_kernel<Q6, TOK, XT, OUT8><<<dim3((unsigned)grid), dim3((unsigned)threads_of(a)), lds, s>>>(a, ep);
  return hipGetLastError();
}

template <bool Q6, int TOK, int XT>
hipError_t launch_out(const MvArgs& a, const Epilogue& ep, int num_cus, hipStream_t s) {
  return ep.out_type == QMM_Q8 ? launch_kernel<Q6, TOK, XT, true>(a, ep, num_cus, s)
                               : launch_kernel<Q6, TOK, XT, false>(a, ep, num_cus, s);
}

template <bool Q6, int TOK>
hipError_t launch_typed(const MvArgs& a, const Epilogue& ep, int num_cus, hipStream_t s) {
  return a.x_type == QMM_F32    ? launch_out<Q6, TOK, QMM_F32>(a, ep, num_cus, s)
         : a.x_type == QMM_F16  ? launch_out<Q6, TOK, QMM_F16>(a, ep, num_cus, s)
         : a.x_type == QMM_BF16 ? launch_out<Q6, TOK, QMM_BF16>(a, ep, num_cus, s)
                                : launch_out<Q6, TOK, QMM_Q8>(a, ep, num_cus, s);
}

template <bool Q6>
hipError_t launch_tokens(const MvArgs& a, const Epilogue& ep, int num_cus, hipStream_t s) {
  return a.n_tok > 8   ? launch_typed<Q6, 16>(a, ep, num_cus, s)
         : a.n_tok > 4 ? launch_typed<Q6, 8>(a, ep, num_cus, s)
         : a.n_tok > 2 ? launch_typed<Q6, 4>(a, ep, num_cus, s)
         : a.n_tok > 1 ? launch_typed<Q6, 2>(a, ep, num_cus, s)
                       : launch_typed<Q6, 1>(a, ep, num_cus, s);
}

}  // namespace

hipError_t launch_mmv(const Planes& p, const void* x, int x_type, int64_t x_stride, int n_tok, const Epilogue& ep,
                      int num_cus, hipStream_t s) {
  MvArgs a{};
  a.w = p.rows;
  a.x = x;
  a.x_stride = (int)x_stride;
  a.x_type = x_type;
  a.n_tok = n_tok;
  a.od = (int)p.od;
  a.nsb = (int)p.nsb;
  return p.type == QMM_Q6_K_ROWS ? launch_tokens<true>(a, ep, num_cus, s) : launch_tokens<false>(a, ep, num_cus, s);
}

}  // namespace qmm
