// qmm_mmq_few.hip -- the MMQ with an epilogue for few tokens (short prompts, batches
// too large for the few-token product on the rows form): one or two blocks of 32
// tokens per work-group, straight from the MMQ's planes.
//
// With so few tokens the planes' bytes bound the product (q4_K 1.25, packed 0.75,
// q6_K 2.02 bytes per weight), and a weight fragment meets no more token blocks than
// one wave has, so that staging it in LDS shares it with nobody.  A wave owns 32 rows
// and a share of the super-blocks and loads its operands straight into registers,
// kAhead chunks ahead; the waves of a row block add their sums in LDS, in order, where
// the tiled MMQ splits a launch this small along the inner dimension into partial
// tiles that a second kernel adds.  The block dots, scales and their order within a
// super-block are the tiled MMQ's.
//
// Measured in a graph, 32 tokens: 11008 x 4096 packed (34 MB) 10.2 us, q4_K (56 MB)
// 12.4, q6_K (91 MB) 20.5, a copy's rate being 4.96 TB/s; 4096 x 4096 q4_K 7.6, 256 x
// 512 q6_K 4.0.  4096 x 11008 q6_K, 91 MB as well, takes 24.3: its 128 row blocks leave
// half of the CUs idle.
#include "qmm_internal.h"
#include "qmm_common.h"
#include "qmm_epilogue.h"
#include "qmm_mmq_ops.h"

#include <algorithm>

namespace qmm {

// Measured against the tiled MMQ (in a graph, us, here / tiled).  One token block is
// always worth it (4096 x 4096 q4_K 7.7 / 15.7, 32000 x 4096 q6_K 42.6 / 63.4, 32
// tokens).  More of them, a wave each, read the weights once each, mostly from cache,
// and win while the work-groups fit one round of the CUs (4096 x 11008 q6_K, 64
// tokens: 18.3 / 27.3), with short rows two (4096 x 4096 q4_K, 128 tokens: 10.0 /
// 15.7).  Over two rounds the lead shrinks with the rows' length: 4096 rows, 128 tokens,
// at 8, 16, 24, 28, 32, 36 and 43 super-blocks q4_K 7.9 / 13.7, 11.5 / 16.9, 15.5 / 17.9,
// 18.8 / 19.5, 19.7 / 20.9, 22.5 / 22.4, 25.2 / 25.2, q6_K 8.8 / 14.8, 14.3 / 17.2, 19.1 /
// 21.1, 23.3 / 23.2, 24.3 / 25.1, 28.1 / 27.3, 31.6 / 30.8; hence 32.  Other shapes lie a
// few super-blocks to either side (2752 rows, 160 tokens, 32: q6_K 38.7 / 35.4, packed 19.9
// / 30.2).  Past one round two token blocks share a
// wave (11008 x 4096 q4_K, 64 tokens: 17.3 / 24.4, a wave each 22.9; 32000 x 4096
// q6_K: 48.7 / 66.4); within one, a wave each is better (4096 x 4096: 8.1, shared
// 10.2), and for more than two the tiled kernel is (11008 x 4096, 96 tokens: shared
// 30.2 / 24.7).
int mmq_few_blocks(const Planes& p, int64_t n_tok, int num_cus) {
  const int64_t tblocks = (n_tok + 31) / 32, blocks = (p.od + 31) / 32 * tblocks;
  if (tblocks == 1 || blocks <= num_cus) return 1;
  if (tblocks == 2) return 2;
  return p.nsb <= 32 && blocks <= 2 * (int64_t)num_cus ? 1 : 0;
}

namespace {

// Waves of a work-group: 128 registers each with one token block, 256 with two.
constexpr int waves_of(int WT) { return WT == 1 ? 16 : 8; }

struct FewArgs {
  const int8_t* wq;
  const float* wd;
  const uint8_t* wsm;
  const uint8_t* qq;
  const uint8_t* qs;
  int nchunk, nsb, od, n_tok;
  int kg_bits, groups;  // 2^kg_bits waves share a row block, groups of them in a work-group
};

// Chunks loaded ahead: what the registers hold beside the sums (32 to 64 KiB of
// weights per CU in flight; four chunks with one token block spill: 11008 x 4096
// q4_K, 32 tokens: 17.0 instead of 13.0 us).
template <int WT>
constexpr int kAhead = WT == 1 ? 2 : 4;

// A super-block's scales, mins and d (q6_K: d only).
template <int TYPE>
struct Small {
  v2i sc[2], mins;
  float d;
};

// WT: token blocks per wave.
template <int TYPE, int WT>
__global__ void __launch_bounds__(64 * waves_of(WT))
mmq_few_kernel(FewArgs a, Epilogue ep) {
  using W = WeightOps<TYPE>;
  constexpr bool kQ4 = is_q4k(TYPE);
  constexpr int kWaves = waves_of(WT), kN = kAhead<WT>;
  __shared__ float red[kWaves * WT * kEpWave];
  __shared__ float dd_all[kWaves][64];  // a super-block's d of 32 rows; q4_K: d*2^25, then -dmin
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kgs = 1 << a.kg_bits;
  const int group = wave >> a.kg_bits, kg = wave & (kgs - 1), groups = a.groups;
  const int rblocks = (a.od + 31) / 32;
  const int rb = min((int)blockIdx.x * groups + group, rblocks - 1);  // past the last: the last again, not stored
  const int row = lane & 31;
  const int tb0 = blockIdx.y * WT;
  const int sb0 = kg * a.nsb >> a.kg_bits, sb1 = (kg + 1) * a.nsb >> a.kg_bits;
  float* const dd = dd_all[wave];

  const int8_t* const pa = a.wq + (int64_t)rb * a.nchunk * kFragA<TYPE>;
  const uint8_t* pb[WT];
  const uint8_t* ps[WT];
#pragma unroll
  for (int w = 0; w < WT; ++w) {
    const int64_t at = (int64_t)(tb0 + w) * a.nchunk;
    pb[w] = a.qq + at * 1024;
    ps[w] = a.qs + at * 128;
  }
  const uint8_t* const pr = a.wsm + (int64_t)rb * (a.nchunk / 4) * kQ4RecBytes;  // q4_K
  const float* const pd = a.wd + (int64_t)rb * a.nsb * 32;                        // q6_K

  typename W::A qa[kN];
  v4i qb[kN][WT];
  uint32_t pair[kN][WT];
  const int last = sb1 * 8 - 1;  // the last chunk of the wave's share
  auto load = [&](int slot, int c) __attribute__((always_inline)) {
    c = min(c, last);
    qa[slot] = W::load(pa + (int64_t)c * kFragA<TYPE>, lane);
#pragma unroll
    for (int w = 0; w < WT; ++w) {
      qb[slot][w] = *(const v4i*)(pb[w] + (int64_t)c * 1024 + lane * 16);
      pair[slot][w] = *(const uint32_t*)(ps[w] + (int64_t)c * 128 + (lane & 31) * 4);
    }
  };
  auto small = [&](int sb) __attribute__((always_inline)) {
    Small<TYPE> r{};
    if constexpr (kQ4) {
      const uint8_t* const rec = pr + (int64_t)sb * 2 * kQ4RecBytes;
      r.sc[0] = *(const v2i*)(rec + kQ4RecScOff + row * 8);
      r.sc[1] = *(const v2i*)(rec + kQ4RecBytes + kQ4RecScOff + row * 8);
      r.mins = *(const v2i*)(rec + kQ4RecMnOff + lane * 8);
      r.d = *(const float*)(rec + kQ4RecDOff + lane * 4);
    } else {
      r.d = pd[sb * 32 + (lane & 31)];
    }
    return r;
  };
  constexpr bool kSmallAhead = !kQ4 || WT == 2;  // where the registers hold the next super-block's
  Small<TYPE> next{};
  if (kSmallAhead) next = small(sb0);
#pragma unroll
  for (int i = 0; i < kN; ++i) load(i, sb0 * 8 + i);

  float acc[WT][16], inner[WT][16];
#pragma unroll
  for (int w = 0; w < WT; ++w)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[w][i] = 0.0f;
  const bool lane_hi = lane >= 32;
  for (int sb = sb0; sb < sb1; ++sb) {
    const Small<TYPE> now = kSmallAhead ? next : small(sb);
    if (kSmallAhead) next = small(min(sb + 1, sb1 - 1));
    v2i bs[WT] = {};
    uint32_t even[WT] = {};
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const int slot = c % kN;
      typename W::D dot[WT];
      uint32_t pr_c[WT];
#pragma unroll
      for (int w = 0; w < WT; ++w) {
        dot[w] = W::mma(qa[slot], qb[slot][w]);
        pr_c[w] = pair[slot][w];
      }
      load(slot, sb * 8 + c + kN);
#pragma unroll
      for (int w = 0; w < WT; ++w) {
        v16f sd;
        float dh = 0.0f;
        if constexpr (kQ4) {
          sd = scale_outer(now.sc[c >> 2], pr_c[w], c & 3);
          if (c & 1) {  // the scaled sums of chunks c - 1 and c
            const int two = (int)__builtin_amdgcn_perm(pr_c[w], even[w], 0x07060302u);
            if (lane_hi == (c >= 4)) bs[w][(c & 3) >> 1] = two;
          } else {
            even[w] = pr_c[w];
          }
        } else {
          dh = f16_bits_to_float(pr_c[w] & 0xFFFF);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float f = kQ4 ? sd[i] : dh;
          inner[w][i] = c == 0 ? W::val(dot[w], i) * f : fmaf(W::val(dot[w], i), f, inner[w][i]);
          pin(inner[w][i]);
        }
      }
      // a chunk at a time: the loads ahead need the other registers
      __builtin_amdgcn_sched_barrier(0);
    }
    dd[lane] = now.d;
#pragma unroll
    for (int w = 0; w < WT; ++w) {
      v16f mt;
      if constexpr (kQ4) {
        typedef _Float16 v4h __attribute__((ext_vector_type(4)));
        const v16f zero = {};
        mt = __builtin_amdgcn_mfma_f32_32x32x8f16(__builtin_bit_cast(v4h, now.mins), __builtin_bit_cast(v4h, bs[w]),
                                                  zero, 0, 0, 0);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float4 f = *(const float4*)(dd + 8 * q + 4 * (lane >> 5));
        acc[w][4 * q + 0] = fmaf(inner[w][4 * q + 0], f.x, acc[w][4 * q + 0]);
        acc[w][4 * q + 1] = fmaf(inner[w][4 * q + 1], f.y, acc[w][4 * q + 1]);
        acc[w][4 * q + 2] = fmaf(inner[w][4 * q + 2], f.z, acc[w][4 * q + 2]);
        acc[w][4 * q + 3] = fmaf(inner[w][4 * q + 3], f.w, acc[w][4 * q + 3]);
        if constexpr (kQ4) {
          const float4 m = *(const float4*)(dd + 32 + 8 * q + 4 * (lane >> 5));
          acc[w][4 * q + 0] = fmaf(mt[4 * q + 0], m.x, acc[w][4 * q + 0]);
          acc[w][4 * q + 1] = fmaf(mt[4 * q + 1], m.y, acc[w][4 * q + 1]);
          acc[w][4 * q + 2] = fmaf(mt[4 * q + 2], m.z, acc[w][4 * q + 2]);
          acc[w][4 * q + 3] = fmaf(mt[4 * q + 3], m.w, acc[w][4 * q + 3]);
        }
      }
    }
  }

#pragma unroll
  for (int w = 0; w < WT; ++w) {
    float* const mine = red + (wave * WT + w) * kEpWave;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      *(float4*)(mine + (lane & 31) * kEpRow + 8 * q + 4 * (lane >> 5)) =
          make_float4(acc[w][4 * q], acc[w][4 * q + 1], acc[w][4 * q + 2], acc[w][4 * q + 3]);
  }
  __syncthreads();
  // four rows of a token per thread: eight threads hold a token's 32 rows
  const bool q8 = ep.out_type == QMM_Q8;
#pragma unroll 1
  for (int i = threadIdx.x; i < groups * WT * 256; i += blockDim.x) {
    const int g = i / (WT * 256), w = (i >> 8) % WT, tl = (i >> 3) & 31, quad = i & 7;
    const int b = (int)blockIdx.x * groups + g, j = b * 32 + 4 * quad, t = (tb0 + w) * 32 + tl;
    const int n = min(a.od - j, 4);
    const bool live = t < a.n_tok && n > 0;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (live) {
      const Sides side = load_sides(ep, t, j, n);
      const float* p = red + ((g << a.kg_bits) * WT + w) * kEpWave + tl * kEpRow + 4 * quad;
      v = *(const float4*)p;
      for (int k = 1; k < kgs; ++k) {
        const float4 e = *(const float4*)(p + k * WT * kEpWave);
        v = make_float4(v.x + e.x, v.y + e.y, v.z + e.z, v.w + e.w);
      }
      v = finish(ep, v, side);
    }
    if (q8 && b < rblocks)  // od % 256 == 0: whole blocks; padding tokens are zeros
      put_q8(ep, quant_quad(v), t, b, a.od, quad);
    else if (live)
      put(ep, v, t, j, n);
  }
  if (q8 && blockIdx.y + 1 == gridDim.y && kg == 0 && (int)blockIdx.x * groups + group < rblocks)
    for (int b = tb0 + WT; b * 32 < ep.t_pad; ++b) zero_block(ep, rb, b, lane, a.od);
}

// Waves per row block: the fewest rounds of work-groups (one per CU), counted in the
// super-blocks that each wave walks (and half of one for the sums).  Row blocks per
// work-group: as few as leave no more work-groups than CUs.
template <int TYPE, int WT>
void launch_blocks(FewArgs a, int64_t tgroups, const Epilogue& ep, int num_cus, hipStream_t s) {
  constexpr int kWaves = waves_of(WT);
  const int64_t rblocks = (a.od + 31) / 32;
  double best = 0;
  for (int bits = 0, kg = 1; kg <= kWaves && (kg == 1 || kg <= a.nsb); kg = 1 << ++bits) {
    const int64_t wgs = (rblocks + kWaves / kg - 1) / (kWaves / kg) * tgroups;
    const double cost = (double)((wgs + num_cus - 1) / num_cus) * ((a.nsb + kg - 1) / kg + 0.5);
    if (kg == 1 || cost < best) {
      best = cost;
      a.kg_bits = bits;
    }
  }
  a.groups = (int)std::min<int64_t>(kWaves >> a.kg_bits, (rblocks * tgroups + num_cus - 1) / num_cus);
  mmq_few_kernel<TYPE, WT><<<dim3((unsigned)((rblocks + a.groups - 1) / a.groups), (unsigned)tgroups),
                             dim3((64 * a.groups) << a.kg_bits), 0, s>>>(a, ep);
}

template <int TYPE>
hipError_t launch_typed(const Planes& p, const uint8_t* qact, int64_t n_tok, int64_t t_pad, const Epilogue& ep,
                        int num_cus, hipStream_t s) {
  FewArgs a{p.wq, p.wd, p.wsm, qact, qact + (size_t)t_pad * (size_t)p.id, (int)p.nchunk, (int)p.nsb, (int)p.od,
            (int)n_tok, 0, 1};
  const int64_t tblocks = (n_tok + 31) / 32;
  if (mmq_few_blocks(p, n_tok, num_cus) == 2)
    launch_blocks<TYPE, 2>(a, 1, ep, num_cus, s);
  else
    launch_blocks<TYPE, 1>(a, tblocks, ep, num_cus, s);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mmq_few(const Planes& p, const uint8_t* qact, int64_t n_tok, int64_t t_pad, const Epilogue& ep,
                          int num_cus, hipStream_t s) {
  return p.type == QMM_Q6_K   ? launch_typed<QMM_Q6_K>(p, qact, n_tok, t_pad, ep, num_cus, s)
         : p.type == QMM_Q4_K ? launch_typed<QMM_Q4_K>(p, qact, n_tok, t_pad, ep, num_cus, s)
                              : launch_typed<QMM_Q4_K_PACKED>(p, qact, n_tok, t_pad, ep, num_cus, s);
}

}  // namespace qmm
