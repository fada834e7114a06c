// qmm_mmv.hip -- the product for one to eight tokens (decode steps, speculative
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
// byte is read once, in rows, 16 code bytes per lane: eight lanes hold a
// super-block, a wave eight consecutive ones.  Dots are 4-element integer dot
// products on the vector ALU: the matrix core's tiles of 16 or 32 tokens would
// be mostly empty.
//
// A work-group first quantizes the tokens' activations into LDS (the whole inner
// dimension, where it fits), then walks row groups: each of its waves takes kRows
// rows, so that an activation read from LDS serves kRows rows, over its share of
// the super-blocks; a row group's shares are added through LDS in a fixed order
// and go through the epilogue.
#include "qmm_internal.h"
#include "qmm_common.h"
#include "qmm_epilogue.h"
#include "qmm_quant.h"

#include <algorithm>

namespace qmm {

// ---------------------------------------------------------------------------
// The rows form of a weight matrix of od rows and nsb super-blocks per row,
// planes in this order, each starting at a multiple of 256 bytes:
//   q4_K  codes  [od][nsb][128]: the block's 128 code bytes
//         heads  [od][nsb][16]: for each pair i of 32-blocks (2i, 2i + 1) three
//                bytes, 24 bits from the lowest: scale and min of block 2i, scale
//                and min of block 2i + 1, six bits each; then f16 d, f16 dmin
//   q6_K  low    [od][nsb][128]: the block's 128 bytes of low code bits
//         high   [od][nsb][8][8]: for byte group p (the 16 low bytes 16p ..) the
//                high bits of its 32 codes: byte b of the first (second) four
//                bytes holds in bits 2j, 2j + 1 those of the low (high) nibble's
//                code 4j + b, the upper of the two inverted
//         scales [od][nsb][8][2]: the int8 scales of byte group p's low nibbles
//                and of its high nibbles
//         d      [od][nsb] f16
// ---------------------------------------------------------------------------
namespace {

constexpr size_t round256(size_t v) { return (v + 255) / 256 * 256; }

__device__ __forceinline__ uint4 load16(const uint8_t* p) {  // 16 bytes at an even address
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = (uint32_t)*(const uint16_t*)(p + 4 * i) | ((uint32_t)*(const uint16_t*)(p + 4 * i + 2) << 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ uint4 q4k_head(const uint8_t* B) {
  uint32_t pair[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t six[4];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int c = 2 * i + k;
      const uint8_t* P = B + 4;
      six[2 * k] = c < 4 ? P[c] & 63 : (P[c + 4] & 15) | ((P[c - 4] >> 6) << 4);
      six[2 * k + 1] = c < 4 ? P[c + 4] & 63 : (P[c + 4] >> 4) | ((P[c] >> 6) << 4);
    }
    pair[i] = six[0] | (six[1] << 6) | (six[2] << 12) | (six[3] << 18);
  }
  return make_uint4(pair[0] | (pair[1] << 24), (pair[1] >> 8) | (pair[2] << 16), (pair[2] >> 16) | (pair[3] << 8),
                    (uint32_t)B[0] | ((uint32_t)B[1] << 8) | ((uint32_t)B[2] << 16) | ((uint32_t)B[3] << 24));
}

// One thread per (super-block, byte group p), striding over a capped grid.
__global__ void __launch_bounds__(256)
repack_rows_kernel(const uint8_t* __restrict__ raw, int q6, int64_t total, RowPlanes r) {
  const int64_t stride = (int64_t)gridDim.x * blockDim.x;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += stride) {
    const int64_t b = i >> 3;
    const int p = (int)(i & 7);
    if (q6) {
      const uint8_t* B = raw + b * 210;
      *(uint4*)(r.codes + b * 128 + 16 * p) = load16(B + 16 * p);
      const int shift = 2 * ((p >> 1) & 1);
      const uint8_t* qh = B + 128 + 32 * (p >> 2) + 16 * (p & 1);
      uint32_t high[2] = {0, 0};
      for (int k = 0; k < 16; ++k)
        for (int n = 0; n < 2; ++n)
          high[n] |= (uint32_t)(((qh[k] >> (shift + 4 * n)) & 3) ^ 2) << (8 * (k & 3) + 2 * (k >> 2));
      *(uint2*)(r.heads + b * 64 + 8 * p) = make_uint2(high[0], high[1]);
      const int g = p + 4 * (p >> 2);  // the 16-weight group of the low nibbles; the high ones' is 4 further
      r.scales[b * 16 + 2 * p] = B[192 + g];
      r.scales[b * 16 + 2 * p + 1] = B[192 + g + 4];
      if (p == 0) r.d[b] = (uint16_t)(B[208] | (B[209] << 8));
    } else {
      const uint8_t* B = raw + b * 144;
      *(uint4*)(r.codes + b * 128 + 16 * p) = *(const uint4*)(B + 16 + 16 * p);
      if (p == 0) *(uint4*)(r.heads + b * 16) = q4k_head(B);
    }
  }
}

}  // namespace

RowPlanes row_planes(int type, int64_t od, int64_t id, void* base, size_t* bytes) {
  const size_t nb = (size_t)od * (size_t)(id / 256);
  const bool q6 = type == QMM_Q6_K_ROWS;
  RowPlanes r{};
  r.heads_offset = round256(nb * 128);
  r.scales_offset = r.heads_offset + round256(nb * (q6 ? 64 : 16));
  r.d_offset = r.scales_offset + (q6 ? round256(nb * 16) : 0);
  *bytes = r.d_offset + (q6 ? round256(nb * 2) : 0);
  r.codes = (uint8_t*)base;
  r.heads = r.codes + r.heads_offset;
  r.scales = r.codes + r.scales_offset;
  r.d = (uint16_t*)(r.codes + r.d_offset);
  return r;
}

hipError_t launch_repack_rows(const uint8_t* raw, int type, int64_t od, int64_t id, const RowPlanes& r, hipStream_t s) {
  const int64_t total = od * (id / 256) * 8;
  const int64_t blocks = std::min<int64_t>((total + 255) / 256, 1 << 14);
  repack_rows_kernel<<<dim3((unsigned)blocks), dim3(256), 0, s>>>(raw, type == QMM_Q6_K_ROWS, total, r);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// The product.
// ---------------------------------------------------------------------------
namespace {

constexpr int kWaves = 8;
constexpr int kRows = 4;  // rows a wave takes at once
constexpr int kItem = 8;  // super-blocks a wave reads at once

// Activations in LDS, per token and super-block: 256 code bytes as [low, high][8
// byte groups][16], the codes that meet the low and the high nibbles of weight
// byte group p; and per pair of 32-blocks the f32 scales: q4_K (dh, s) of the
// low nibbles' block and of the high ones', q6_K both dh.
template <bool Q6>
constexpr int kScaleBytes = Q6 ? 32 : 64;
template <bool Q6>
constexpr int kSbBytes = 256 + kScaleBytes<Q6>;

struct MvArgs {
  RowPlanes w;
  const void* x;
  int64_t x_stride;
  int x_type, n_tok, od, nsb;
  int tile_sb;  // super-blocks quantized at a time
  int kg;       // waves that share a row group, each over its share of the super-blocks
  int steps;    // row-group sets: ceil(od / (kWaves / kg * kRows))
};

// A lane's weights of one row: 32 codes and what scales them.
struct Q4Lane {
  uint4 code, head;
};
struct Q6Lane {
  uint4 low;
  uint2 high;
  uint32_t scales, d;  // two int8; f16
};

__device__ __forceinline__ int dot16(const uint32_t (&a)[4], const v4i& b) {
  int s = __builtin_amdgcn_sdot4((int)a[0], b[0], 0, false);
  s = __builtin_amdgcn_sdot4((int)a[1], b[1], s, false);
  s = __builtin_amdgcn_sdot4((int)a[2], b[2], s, false);
  return __builtin_amdgcn_sdot4((int)a[3], b[3], s, false);
}

template <int NT>
__device__ __forceinline__ void add_row(const Q4Lane& w, const v4i (&qa)[NT], const v4i (&qb)[NT],
                                        const float4 (&sc)[NT], int pair, float (&acc)[NT]) {
  uint32_t lo[4], hi[4];
  const uint32_t c[4] = {w.code.x, w.code.y, w.code.z, w.code.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    lo[i] = c[i] & 0x0F0F0F0Fu;
    hi[i] = (c[i] >> 4) & 0x0F0F0F0Fu;
  }
  // the pair's 24 bits: bytes 3*pair .. of the head's first twelve
  const uint32_t h0 = w.head.x, h1 = w.head.y, h2 = w.head.z;
  const uint32_t low = pair < 2 ? h0 : pair == 2 ? h1 : h2, up = pair < 2 ? h1 : h2;
  const uint32_t f = __builtin_amdgcn_alignbit(up, low, (24u * (uint32_t)pair) & 31u);
  const int sa = (int)(f & 63), sb = (int)((f >> 12) & 63);
  const float ma = (float)((f >> 6) & 63), mb = (float)((f >> 18) & 63);
  const float d = f16_bits_to_float(w.head.w & 0xFFFF);
  const float m = -0.5f * f16_bits_to_float(w.head.w >> 16);  // both lanes of a pair add the min term
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const float da = (float)__mul24(sa, dot16(lo, qa[t])), db = (float)__mul24(sb, dot16(hi, qb[t]));
    acc[t] = fmaf(d, fmaf(da, sc[t].x, db * sc[t].z), acc[t]);
    acc[t] = fmaf(m, fmaf(ma, sc[t].y, mb * sc[t].w), acc[t]);
  }
}

// q6_K codes as four times (code - 32): the six bits, the top one inverted, in a
// byte's upper bits are that as an int8; the 4 is taken off d.
template <int NT>
__device__ __forceinline__ void add_row(const Q6Lane& w, const v4i (&qa)[NT], const v4i (&qb)[NT],
                                        const float2 (&sc)[NT], int, float (&acc)[NT]) {
  uint32_t lo[4], hi[4];
  const uint32_t c[4] = {w.low.x, w.low.y, w.low.z, w.low.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    lo[i] = ((c[i] << 2) & 0x3C3C3C3Cu) | ((w.high.x << (6 - 2 * i)) & 0xC0C0C0C0u);
    hi[i] = ((c[i] >> 2) & 0x3C3C3C3Cu) | ((w.high.y << (6 - 2 * i)) & 0xC0C0C0C0u);
  }
  const int sa = (int)(int8_t)w.scales, sb = (int)(int8_t)(w.scales >> 8);
  const float d = 0.25f * f16_bits_to_float(w.d);
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const float da = (float)__mul24(sa, dot16(lo, qa[t])), db = (float)__mul24(sb, dot16(hi, qb[t]));
    acc[t] = fmaf(d, fmaf(da, sc[t].x, db * sc[t].y), acc[t]);
  }
}

// Sums over the wave of N values per lane.  Two values share a register after
// the halves are swapped and added, four after the rows of 16 are, so the last
// four steps run on N/4 registers.  Row r of register k ends with the sum of value
// 4k + {0, 2, 1, 3}[r], in all of its lanes.
template <int N>
__device__ __forceinline__ void wave_sums(float (&v)[N], float (&w)[(N + 3) / 4]) {
  float h[(N + 3) / 4 * 2];
#pragma unroll
  for (int i = 0; i < (N + 3) / 4 * 2; ++i) {
    const uint32_t a = 2 * i < N ? __builtin_bit_cast(uint32_t, v[2 * i < N ? 2 * i : 0]) : 0;
    const uint32_t b = 2 * i + 1 < N ? __builtin_bit_cast(uint32_t, v[2 * i + 1 < N ? 2 * i + 1 : 0]) : 0;
    const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    h[i] = __builtin_bit_cast(float, (uint32_t)r[0]) + __builtin_bit_cast(float, (uint32_t)r[1]);
  }
#pragma unroll
  for (int k = 0; k < (N + 3) / 4; ++k) {
    const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, h[2 * k]),
                                                    __builtin_bit_cast(uint32_t, h[2 * k + 1]), false, false);
    float s = __builtin_bit_cast(float, (uint32_t)r[0]) + __builtin_bit_cast(float, (uint32_t)r[1]);
    s += __builtin_bit_cast(float, dpp<kDppQuadXor1>(__builtin_bit_cast(int, s)));
    s += __builtin_bit_cast(float, dpp<kDppQuadXor2>(__builtin_bit_cast(int, s)));
    s += __builtin_bit_cast(float, dpp<kDppHalfMirror>(__builtin_bit_cast(int, s)));
    w[k] = s + __builtin_bit_cast(float, dpp<kDppMirror>(__builtin_bit_cast(int, s)));
  }
}

// Quantizes super-blocks [sb0, sb0 + n) of every token into LDS: a thread per
// four activations, eight lanes per 32-block, as the prepass.
template <bool Q6, int NT>
__device__ __forceinline__ void quantize_tile(const MvArgs& a, uint8_t* lds, int sb0, int n) {
  const int per_tok = n * 64;  // quads of a token: whole waves
  for (int i = threadIdx.x; i < NT * per_tok; i += 64 * kWaves) {
    const int t = i / per_tok, k = i % per_tok;  // t is uniform over the wave
    const int64_t at = t * a.x_stride + (int64_t)sb0 * 256 + 4 * k;
    const float4 v = a.x_type == QMM_F32   ? load4<QMM_F32>(a.x, at)
                     : a.x_type == QMM_F16 ? load4<QMM_F16>(a.x, at)
                                           : load4<QMM_BF16>(a.x, at);
    const Q8Quad r = quant_quad(v);
    const int sb = k >> 6, g = (k >> 2) & 15;  // 16-code group of the super-block
    // its place: which nibbles it meets, and of which byte group
    const int hi = Q6 ? (g >> 2) & 1 : (g >> 1) & 1;
    const int p = Q6 ? 4 * (g >> 3) + (g & 3) : 2 * (g >> 2) + (g & 1);
    uint8_t* const q = lds + (t * a.tile_sb + sb) * kSbBytes<Q6>;
    *(uint32_t*)(q + hi * 128 + p * 16 + (k & 3) * 4) = r.codes;
    if ((k & 7) == 0) {
      const int c = (k >> 3) & 7;  // 32-block of the super-block
      float* const s = (float*)(q + 256);
      if (Q6) {  // pair 2*(c/4) + c%2, nibble (c/2)%2
        s[2 * (2 * (c >> 2) + (c & 1)) + ((c >> 1) & 1)] = f16_bits_to_float(r.pair & 0xFFFF);
      } else {
        *(float2*)(s + 2 * c) = make_float2(f16_bits_to_float(r.pair & 0xFFFF), f16_bits_to_float(r.pair >> 16));
      }
    }
  }
}

template <bool Q6, int NT>
__global__ void __launch_bounds__(64 * kWaves)
mmv_kernel(MvArgs a, Epilogue ep) {
  extern __shared__ uint4 lds_raw[];
  uint8_t* const lds = (uint8_t*)lds_raw;
  float* const red = (float*)(lds + (size_t)NT * a.tile_sb * kSbBytes<Q6>);  // [2][wave][NT][kRows]
  constexpr int kVals = NT * kRows;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rg = wave / a.kg, kg = wave % a.kg, groups = kWaves / a.kg;
  const int p = lane & 7, sbl = lane >> 3;
  const bool one_tile = a.tile_sb == a.nsb;
  if (one_tile) quantize_tile<Q6, NT>(a, lds, 0, a.nsb);
  if (one_tile) __syncthreads();
  int buf = 0;
  for (int step = blockIdx.x; step < a.steps; step += gridDim.x, buf ^= 1) {
    const int r0 = (step * groups + rg) * kRows;
    float acc[kRows][NT];
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
      for (int t = 0; t < NT; ++t) acc[r][t] = 0.0f;
    for (int sb0 = 0; sb0 < a.nsb; sb0 += a.tile_sb) {
      const int n = min(a.tile_sb, a.nsb - sb0);
      if (!one_tile) {
        __syncthreads();  // the last tile's readers are done
        quantize_tile<Q6, NT>(a, lds, sb0, n);
        __syncthreads();
      }
      if (r0 < a.od)
        for (int it = kg * kItem; it < n; it += a.kg * kItem) {
          const int sb = it + sbl;
          if (sb < n) {
            typedef typename std::conditional<Q6, Q6Lane, Q4Lane>::type Lane;
            typedef typename std::conditional<Q6, float2, float4>::type Scale;
            Lane w[kRows];
#pragma unroll
            for (int r = 0; r < kRows; ++r) {  // rows past the end read the last one
              const int64_t b = (int64_t)min(r0 + r, a.od - 1) * a.nsb + sb0 + sb;
              if constexpr (Q6) {
                w[r].low = *(const uint4*)(a.w.codes + b * 128 + 16 * p);
                w[r].high = *(const uint2*)(a.w.heads + b * 64 + 8 * p);
                w[r].scales = *(const uint16_t*)(a.w.scales + b * 16 + 2 * p);
                w[r].d = a.w.d[b];
              } else {
                w[r].code = *(const uint4*)(a.w.codes + b * 128 + 16 * p);
                w[r].head = *(const uint4*)(a.w.heads + b * 16);
              }
            }
            v4i qa[NT], qb[NT];
            Scale sc[NT];
            const int pair = Q6 ? 2 * (p >> 2) + ((p >> 1) & 1) : p >> 1;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              const uint8_t* const q = lds + (t * a.tile_sb + sb) * kSbBytes<Q6>;
              qa[t] = *(const v4i*)(q + 16 * p);
              qb[t] = *(const v4i*)(q + 128 + 16 * p);
              sc[t] = *(const Scale*)(q + 256 + sizeof(Scale) * pair);
            }
#pragma unroll
            for (int r = 0; r < kRows; ++r) add_row<NT>(w[r], qa, qb, sc, pair, acc[r]);
          }
        }
    }
    // the wave's sums, then the row group's over its waves in order
    float v[kVals], s[(kVals + 3) / 4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int r = 0; r < kRows; ++r) v[t * kRows + r] = acc[r][t];
    wave_sums<kVals>(v, s);
    float* const out = red + ((size_t)buf * kWaves + wave) * kVals;
    if ((lane & 15) == 0) {
      const int row = lane >> 4, order = row == 1 ? 2 : row == 2 ? 1 : row;
#pragma unroll
      for (int k = 0; k < kVals / 4; ++k) out[4 * k + order] = s[k];
    }
    __syncthreads();
    // two buffers: the next step's sums do not overwrite these, the one after has
    // passed the next barrier
    if (kg == 0 && lane < a.n_tok && r0 < a.od) {
      float4 f = *(const float4*)(out + lane * kRows);
      for (int k = 1; k < a.kg; ++k) {
        const float4 g = *(const float4*)(out + k * kVals + lane * kRows);
        f = make_float4(f.x + g.x, f.y + g.y, f.z + g.z, f.w + g.w);
      }
      const int n = min(a.od - r0, kRows);
      put(ep, finish(ep, f, lane, r0, n), lane, r0, n);
    }
  }
}

template <bool Q6, int NT>
hipError_t launch_mmv_tokens(const MvArgs& in, const Epilogue& ep, int num_cus, hipStream_t s) {
  MvArgs a = in;
  // LDS: the whole inner dimension where it fits 150 of the CU's 160 KB, else
  // tiles of it, quantized again for every row-group set
  constexpr size_t kRed = 2 * kWaves * NT * kRows * sizeof(float);
  constexpr size_t kMost = 150 * 1024;
  const size_t per_sb = (size_t)NT * kSbBytes<Q6>;
  a.tile_sb = (int)std::min<size_t>(a.nsb, (kMost - kRed) / per_sb);
  const size_t lds = a.tile_sb * per_sb + kRed;
  // Waves per row group: enough to fill the GPU with 16 waves per CU, each with a
  // whole item of its own.
  const int64_t row_groups = (a.od + kRows - 1) / kRows;
  a.kg = 1;
  while (a.kg < kWaves && row_groups * a.kg < 16 * (int64_t)num_cus && a.nsb >= 2 * a.kg * kItem) a.kg *= 2;
  const int groups = kWaves / a.kg;
  a.steps = (int)((row_groups + groups - 1) / groups);
  const int per_cu = (int)std::max<size_t>(1, std::min<size_t>(2, (160 * 1024) / lds));
  const int grid = std::min(a.steps, num_cus * per_cu);
  if (lds > 64 * 1024) {
    hipError_t e = hipFuncSetAttribute((const void*)mmv_kernel<Q6, NT>, hipFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)lds);
    if (e != hipSuccess) return e;
  }
  mmv_kernel<Q6, NT><<<dim3((unsigned)grid), dim3(64 * kWaves), lds, s>>>(a, ep);
  return hipGetLastError();
}

template <bool Q6>
hipError_t launch_mmv_type(const MvArgs& a, const Epilogue& ep, int num_cus, hipStream_t s) {
  switch (a.n_tok) {
    case 1: return launch_mmv_tokens<Q6, 1>(a, ep, num_cus, s);
    case 2: return launch_mmv_tokens<Q6, 2>(a, ep, num_cus, s);
    case 3: return launch_mmv_tokens<Q6, 3>(a, ep, num_cus, s);
    case 4: return launch_mmv_tokens<Q6, 4>(a, ep, num_cus, s);
    case 5: return launch_mmv_tokens<Q6, 5>(a, ep, num_cus, s);
    case 6: return launch_mmv_tokens<Q6, 6>(a, ep, num_cus, s);
    case 7: return launch_mmv_tokens<Q6, 7>(a, ep, num_cus, s);
    default: return launch_mmv_tokens<Q6, 8>(a, ep, num_cus, s);
  }
}

}  // namespace

hipError_t launch_mmv(const Planes& p, const void* x, int x_type, int64_t x_stride, int n_tok, const Epilogue& ep,
                      int num_cus, hipStream_t s) {
  MvArgs a{};
  a.w = p.rows;
  a.x = x;
  a.x_stride = x_stride;
  a.x_type = x_type;
  a.n_tok = n_tok;
  a.od = (int)p.od;
  a.nsb = (int)p.nsb;
  return p.type == QMM_Q6_K_ROWS ? launch_mmv_type<true>(a, ep, num_cus, s) : launch_mmv_type<false>(a, ep, num_cus, s);
}

}  // namespace qmm
