// qmm_attention_parts.h -- what the attention kernels share: operands from the
// cache's tiles, the columns of a work-group, the running softmax, and the stores.
//
// A column is a (token, head of the group) pair of one sequence and cache head:
// all of them want the same keys and values, so the heads that share a cache head
// share its loads, and one token of many heads fills a matrix operand as many
// tokens of one head do.
//
//   S^T = K Q^T     32 slots x 32 columns, K the left operand: a lane holds one
//                   column (lane % 32) and 16 of the slots, so that a column's
//                   maximum and sum are a lane's own, but for one exchange with the
//                   lane of the other half
//   O^T = V^T P^T   32 channels x 32 columns; P^T as the lane already holds it: with the key
//                   rows in the cache's order, accumulators 8s .. 8s + 7 are the slots
//                   16s + 8*(lane / 32) + (0 .. 7) of the right operand's step s
#pragma once

#include "qmm_attention.h"
#include "qmm_common.h"
#include "qmm_quant.h"

namespace qmm {

typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float v4f __attribute__((ext_vector_type(4)));

constexpr float kNone = -__builtin_inff();

// What is multiplied: f16, also for a q8 cache, or bf16.
template <int TYPE>
struct Math {
  typedef f16x8 v8;
  typedef _Float16 e;
  static constexpr uint16_t kExponent = 0x7c00;
  // Probabilities are 2^kRaise times what they stand for, and so is their sum.  f16's are whole numbers of
  // 2^-24: with the largest, 2^kSlack, raised to 2^15, weights of 2^-22 of the largest one have all of
  // their bits, and smaller ones are off by 2^-33 of it at most, 2^20 of them by 2^-13, a quarter of
  // the result's own half step.  (At 2^0 weights below 2^-25 are lost: of 131072 keys 0.4%.)
  static constexpr float kRaise = 8.0f;
  static __device__ __forceinline__ v16f mma(const v8& a, const v8& b, const v16f& c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
  }
};
template <>
struct Math<QMM_BF16> {
  typedef bf16x8 v8;
  typedef __bf16 e;
  static constexpr uint16_t kExponent = 0x7f80;
  static constexpr float kRaise = 0.0f;  // f32's exponents
  static __device__ __forceinline__ v16f mma(const v8& a, const v8& b, const v16f& c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
};

// Four q8 codes (plus 128, one per byte) as f16: 1024 + code + 128 by putting the
// byte under the exponent of 1024, minus 1152 (exact), times the scales (rounded once: an
// 11-bit product of 7 and 11 bits, an eighth of what the codes' own rounding is off).
__device__ __forceinline__ void codes4(uint32_t w, const f16x2& s0, const f16x2& s1, f16x2& a, f16x2& b) {
  const f16x2 off = {(_Float16)1152.0f, (_Float16)1152.0f};
  a = (__builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, w, 0x04010400u)) - off) * s0;
  b = (__builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, w, 0x04030402u)) - off) * s1;
}
__device__ __forceinline__ f16x8 codes8(uint32_t w0, uint32_t w1, const f16x8& s) {
  f16x2 r[4];
  codes4(w0, f16x2{s[0], s[1]}, f16x2{s[2], s[3]}, r[0], r[1]);
  codes4(w1, f16x2{s[4], s[5]}, f16x2{s[6], s[7]}, r[2], r[3]);
  return f16x8{r[0].x, r[0].y, r[1].x, r[1].y, r[2].x, r[2].y, r[3].x, r[3].y};
}
__device__ __forceinline__ f16x8 splat8(_Float16 s) { return f16x8{s, s, s, s, s, s, s, s}; }

// The columns of a work-group's tile: flat = token * group + head of the group, from
// `first` on; a lane's own is first + column. Where there is none (past the sequence's
// last), it stands for the last one and is not stored.
struct Column {
  bool real;
  int row, head;   // of q and out
  int low, high;   // slots it sees: [low, high)
};

__device__ __forceinline__ Column column(const AttnArgs& a, const Sequence& seq, int kv_head, int flat) {
  const int last = seq.count * a.group - 1;
  const bool real = flat <= last;
  flat = min(flat, last);
  const int token = a.by_group.of(flat);
  Column c = {real, seq.first + token, kv_head * a.group + flat - token * a.group, 0, seq.length};
  if (a.causal) {
    const int end = seq.length - seq.count + token + 1;
    c.high = max(0, end);
    if (a.window > 0 && a.window < end) c.low = end - (int)a.window;
  }
  return c;
}

// The slots that any of the tokens from `first` to `last` sees.
__device__ __forceinline__ void seen(const AttnArgs& a, const Sequence& seq, int first, int last, int& low, int& high) {
  low = 0;
  high = seq.length;
  if (a.causal) {
    const int begin = seq.length - seq.count + first + 1;
    high = max(0, seq.length - seq.count + last + 1);
    if (a.window > 0 && a.window < begin) low = begin - (int)a.window;
  }
}

// Columns' queries as right operands: lane (column, half) has channels 16*step + 8*half ..
template <int TYPE, int DB>
__device__ __forceinline__ void load_queries(const AttnArgs& a, const Column& c, int lane, typename Math<TYPE>::v8 (&q)[2 * DB]) {
  typedef typename Math<TYPE>::v8 v8;
  const uint16_t* p = (const uint16_t*)a.q + c.row * a.q_stride + c.head * a.q_head_stride + 8 * (lane >> 5);
#pragma unroll
  for (int i = 0; i < 2 * DB; ++i) q[i] = *(const v8*)(p + 16 * i);
}

// A value of this lane's column from both halves' lanes, without a trip through LDS:
// v_permlane32_swap_b32 exchanges one register's upper lanes with another's lower.
struct Halves {
  float a, b;
};
__device__ __forceinline__ Halves halves(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return {__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1])};
}
__device__ __forceinline__ float both_sum(float x) {
  const Halves h = halves(x);
  return h.a + h.b;
}

// A running softmax's state of a lane's column: what its scores are taken relative to (the
// same in both halves' lanes) and this lane's part of the sum.
struct Running {
  float top = kNone, sum = 0.0f;
};

// Scores (16 a lane and block of 32 slots) -> right operands of the second product.
// exp(scale*(s - top)) is 2^(s*scale2 - top*scale2), one fma and one v_exp_f32.  `top` only
// follows the maximum once that is kSlack powers of two above it in some column, so that
// the accumulators are scaled a few times a sequence and not with most tiles: a probability
// may then be up to 2^kSlack (times 2^kRaise), which f16 and bf16 hold as exactly as one below 1 (and an
// f32 sum of 2^31 of them too), and what is small is no smaller than relative to the maximum itself.
// A column without a score above -infinity stays at sum 0; NaN scores stay NaN, as a sum
// that is not a number shows.
constexpr float kSlack = 7.0f;
template <int TYPE, int DB, int KB>
__device__ __forceinline__ void soften(v16f (&s)[KB], float scale2, Running& run, v16f (&o)[DB],
                                       typename Math<TYPE>::v8 (&p)[2 * KB]) {
  typedef typename Math<TYPE>::e e;
  float top = s[0][0];
#pragma unroll
  for (int k = 0; k < KB; ++k)
#pragma unroll
    for (int i = 0; i < 16; ++i) top = fmaxf(top, s[k][i]);
  const Halves t = halves(top);
  top = fmaxf(t.a, t.b);
  const bool far = (top - run.top) * scale2 > kSlack;  // -infinity minus itself is not
  if (__any(far)) {
    top = far ? top : run.top;  // a column's numbers do not go by its neighbours'
    const float by = run.top == kNone ? 0.0f : __builtin_amdgcn_exp2f((run.top - top) * scale2);
    run.top = top;
    run.sum *= by;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[d][i] *= by;
  }
  const float off = run.top == kNone ? 0.0f : Math<TYPE>::kRaise - run.top * scale2;
  float sum = 0.0f;
#pragma unroll
  for (int k = 0; k < KB; ++k)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float x = __builtin_amdgcn_exp2f(fmaf(s[k][i], scale2, off));
      sum += x;
      p[2 * k + (i >> 3)][i & 7] = (e)x;
    }
  run.sum += sum;
}

// Scores of slots that a column does not see: -infinity.  slot0: of the block of 32.
__device__ __forceinline__ void hide(v16f& s, int slot0, int half, int low, int high) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int slot = slot0 + 16 * (i >> 3) + 8 * half + (i & 7);
    if (slot < low || slot >= high) s[i] = kNone;
  }
}

// The operand with zeros for what is no finite number.
template <int TYPE, class V>
__device__ __forceinline__ V finite(const V& v) {
  u16x8 u = __builtin_bit_cast(u16x8, v);
#pragma unroll
  for (int j = 0; j < 8; ++j) u[j] = (u[j] & Math<TYPE>::kExponent) == Math<TYPE>::kExponent ? 0 : u[j];
  return __builtin_bit_cast(V, u);
}

// Value of slot r and channel d of a tile of values, as the product takes it.
template <int TYPE>
__device__ __forceinline__ float value_of(const uint8_t* tile, int dim, int r, int d) {
  if constexpr (TYPE == QMM_Q8)
    return (float)((_Float16)(float)((int)tile[value_code_at(r, d)] - 128) * *(const _Float16*)(tile + scale_at(dim, r, d >> 5)));
  else
    return (float)((const elem_t<TYPE>*)tile)[value_at(r, d)];
}

// The slots that only some columns of a work-group see, or none: a value there that is
// no finite number must not reach the others, and on the matrix core their 0 times it
// would be NaN.  A result that is no finite number may be such a one: the work-group then
// does its tile again with zeros for those values in the product (`finite`), and they are
// added here to the columns that see them, channel by channel.  Both go by the same 32 slots: in a
// tile that every column sees nothing is taken out and nothing added.
struct Edges {
  int from, end;  // tiles of the split
  int low, high;  // slots that every column sees
};
template <int TYPE>
__device__ __forceinline__ void add_edges(const Pools& pools, const Batch& batch, int s, int h, const Edges& e, const Column& c,
                                          int d, float4& x) {
#pragma unroll 1
  for (int t = e.from; t < e.end; ++t) {
    // where every column sees the tile its values were left as they are
    if ((32 * t >= e.low && 32 * t + 32 <= e.high) || 32 * t >= c.high || 32 * t + 32 <= c.low) continue;
    const int64_t at = tile_offset(batch, pools, s, h, t);
    if (at < 0) continue;
#pragma unroll 1
    for (int slot = max(32 * t, c.low); slot < min(32 * t + 32, c.high); ++slot) {
      float v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = value_of<TYPE>(pools.v + at, pools.dim, slot & 31, d + i);
        if (fabsf(v[i]) < __builtin_inff()) v[i] = 0.0f;
      }
      x.x += v[0], x.y += v[1], x.z += v[2], x.w += v[3];
    }
  }
}

// Four channels of one output, d a multiple of 4; eight lanes that hold a block of 32
// channels call it together where the output is q8 blocks.
template <int TYPE>
__device__ __forceinline__ void store_four(const AttnArgs& a, int dim, int row, int head, int d, const float4& x) {
  if (!a.q8_out) {
    constexpr int T = TYPE == QMM_BF16 ? QMM_BF16 : QMM_F16;
    store4<T>(a.out, row * a.out_stride + (int64_t)head * dim + d, x);
    return;
  }
  const int k = head * dim + d;
  const int64_t id = (int64_t)a.heads * dim, block = (int64_t)(row >> 5) * (id >> 5) + (k >> 5);
  const Q8Quad q = quant_quad(x);
  uint8_t* const out = (uint8_t*)a.out;
  *(uint32_t*)(out + block * 1024 + ((k & 31) >> 4) * 512 + (row & 31) * 16 + (k & 15)) = q.codes;
  if ((k & 31) == 0) *(uint32_t*)(out + a.t_pad * id + block * 128 + (row & 31) * 4) = q.pair;
}

// Adds a part's sums, which are relative to `mine`, to sums relative to `top`.
__device__ __forceinline__ void add_part(float4& x, float& total, const float4& part, float mine, float sum, float top,
                                         float scale2) {
  const float by = mine == kNone ? 0.0f : __builtin_amdgcn_exp2f((mine - top) * scale2);
  total = fmaf(sum, by, total);
  x.x = fmaf(part.x, by, x.x), x.y = fmaf(part.y, by, x.y), x.z = fmaf(part.z, by, x.z), x.w = fmaf(part.w, by, x.w);
}

// Four channels' results from a column's sums.  Nothing seen, or no score above -infinity: zeros, and
// not 0 times a value that is no number.
__device__ __forceinline__ float4 divided(const float4& x, float total) {
  const float by = 1.0f / total;
  return total == 0.0f ? make_float4(0, 0, 0, 0) : make_float4(x.x * by, x.y * by, x.z * by, x.w * by);
}

// Four channels of a column's sums: to the split's partial results, or as the output.
template <int TYPE>
__device__ __forceinline__ void store_part(const AttnArgs& a, int dim, int n_tok, int split, const Column& c, int d,
                                           const float4& x, float top, float total) {
  if (a.splits > 1) {
    const int64_t row = (int64_t)c.row * a.heads + c.head + (int64_t)split * n_tok * a.heads;
    *(float4*)(a.part + row * dim + d) = x;
    if (d == 0) a.sums[row] = make_float2(top, total);
  } else {
    store_four<TYPE>(a, dim, c.row, c.head, d, divided(x, total));
  }
}

// The columns from `first` to `last` have no part in this split: a sum of 0, whose numbers the
// join does not read.
__device__ __forceinline__ void no_part(const AttnArgs& a, const Sequence& seq, int n_tok, int kv_head, int split, int first,
                                        int last) {
  for (int flat = first + (int)threadIdx.x; flat <= last; flat += (int)blockDim.x) {
    const Column c = column(a, seq, kv_head, flat);
    a.sums[(int64_t)c.row * a.heads + c.head + (int64_t)split * n_tok * a.heads] = make_float2(kNone, 0.0f);
  }
}

// Zeros in the padding tokens of a qact buffer, by `threads` threads together.
__device__ __forceinline__ void zero_padding(const AttnArgs& a, int dim, int n_tok, int64_t thread, int64_t threads) {
  const int64_t id = (int64_t)a.heads * dim, blocks = id >> 5, tokens = a.t_pad - n_tok;
  uint8_t* const out = (uint8_t*)a.out;
  for (int64_t i = thread; i < tokens * blocks; i += threads) {
    const int64_t row = n_tok + i % tokens, block = (row >> 5) * blocks + i / tokens;
    *(uint4*)(out + block * 1024 + (row & 31) * 16) = make_uint4(0, 0, 0, 0);
    *(uint4*)(out + block * 1024 + 512 + (row & 31) * 16) = make_uint4(0, 0, 0, 0);
    *(uint32_t*)(out + a.t_pad * id + block * 128 + (row & 31) * 4) = 0;
  }
}

}  // namespace qmm
