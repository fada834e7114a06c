// qmm_prepass.hip -- the quantize-transpose prepass (r45 page, section 1.1):
// f32 activations -> q8 blocks of 32 with a (dh, s) scale pair, written in the
// MFMA fragment order the MMQ reads.
#include "qmm_internal.h"
#include "qmm_common.h"
#include "qmm_quant.h"

#include "../../include/qmm.h"

namespace qmm {

// ---------------------------------------------------------------------------
// Quantize prepass.  Work-group = one 32-token block x kQuantChunks chunks;
// 8 lanes per (token, chunk), each lane holding 4 consecutive activations.
// A wave covers 8 consecutive tokens of one chunk, so its q bytes land as two
// contiguous 128-byte runs of the fragment and its scale pairs as 32 bytes.
// The kernel streams HBM: every lane issues all of its loads before the first
// wait, and the reductions over a (token, chunk)'s 8 lanes stay in registers
// (DPP moves).
// ---------------------------------------------------------------------------
constexpr int kQuantChunks = 2;

__global__ void __launch_bounds__(256)
quantize_kernel(const float* __restrict__ x, int n_tok, int id, int nchunk, int chunk_major,
                uint8_t* __restrict__ qq, uint8_t* __restrict__ qs) {
  const int tb = chunk_major ? blockIdx.y : blockIdx.x;
  const int c0 = (chunk_major ? blockIdx.x : blockIdx.y) * kQuantChunks;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int tt = wave * 8 + (lane >> 3);
  const int sub = lane & 7;
  const int64_t t = (int64_t)tb * 32 + tt;
  const bool live = t < n_tok;
  const bool block_full = (int64_t)(tb + 1) * 32 <= n_tok;  // uniform: no lane past the end
  // Lanes past the last token read the last token's row (and chunks past the
  // end read the last chunk), so that every load is in bounds and issued
  // unconditionally; their values are replaced by zeros below.
  const float* xr = x + (live ? t : (int64_t)n_tok - 1) * id + 4 * sub;

  float4 v[kQuantChunks];
#pragma unroll
  for (int i = 0; i < kQuantChunks; ++i)
    v[i] = *(const float4*)(xr + 32 * min(c0 + i, nchunk - 1));
#pragma unroll
  for (int i = 0; i < kQuantChunks; ++i) {
    const int c = c0 + i;
    if (c >= nchunk) break;
    if (!block_full && !live) v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    const Q8Quad r = quant_quad(v[i]);
    const int64_t frag = (int64_t)tb * nchunk + c;
    *(uint32_t*)(qq + frag * 1024 + (sub >> 2) * 512 + tt * 16 + (sub & 3) * 4) = r.codes;
    if (sub == 0) *(uint32_t*)(qs + frag * 128 + tt * 4) = r.pair;
  }
}

hipError_t launch_quantize(const float* x, int64_t n_tok, int64_t t_pad, int64_t id,
                           uint8_t* qact, hipStream_t s) {
  const int64_t nchunk = id / 32;
  const unsigned n_tb = (unsigned)(t_pad / 32), n_cg = (unsigned)((nchunk + kQuantChunks - 1) / kQuantChunks);
  // Work-group order.  Many tokens: chunk groups fastest, so consecutive
  // work-groups read consecutive stretches of the same 32 rows (3314 x 4096:
  // 22% faster; with token blocks fastest the rows' power-of-two stride
  // concentrates the reads).  Few tokens: token blocks fastest (4-8% faster at
  // 512 and 2048 tokens).
  const int chunk_major = n_tb > 96;
  const dim3 grid = chunk_major ? dim3(n_cg, n_tb) : dim3(n_tb, n_cg);
  quantize_kernel<<<grid, dim3(256), 0, s>>>(x, (int)n_tok, (int)id, (int)nchunk, chunk_major, qact,
                                             qact + (size_t)t_pad * (size_t)id);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Reading a qact buffer back: a thread per four codes of one token and chunk, in
// the prepass's mapping (its fragment words back into rows of numbers).
// ---------------------------------------------------------------------------
template <int TYPE>
__global__ void __launch_bounds__(256)
dequantize_kernel(const uint8_t* __restrict__ qq, const uint8_t* __restrict__ qs, int n_tok, int nchunk,
                  void* __restrict__ out, int64_t out_stride) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int tt = wave * 8 + (lane >> 3), sub = lane & 7;
  const int64_t t = (int64_t)blockIdx.y * 32 + tt;
  if (t >= n_tok) return;
#pragma unroll
  for (int i = 0; i < kQuantChunks; ++i) {
    const int c = blockIdx.x * kQuantChunks + i;
    if (c >= nchunk) break;
    const int64_t frag = (int64_t)blockIdx.y * nchunk + c;
    const int q = *(const int*)(qq + frag * 1024 + (sub >> 2) * 512 + tt * 16 + (sub & 3) * 4);
    const float dh = f16_bits_to_float(*(const uint32_t*)(qs + frag * 128 + tt * 4) & 0xFFFF);
    store4<TYPE>(out, t * out_stride + 32 * c + 4 * sub,
                 make_float4(dh * (float)(int8_t)q, dh * (float)(int8_t)(q >> 8), dh * (float)(int8_t)(q >> 16),
                             dh * (float)(q >> 24)));
  }
}

hipError_t launch_dequantize(const uint8_t* qact, int64_t n_tok, int64_t t_pad, int64_t id, int type, void* out,
                             int64_t out_stride, hipStream_t s) {
  const int64_t nchunk = id / 32;
  const dim3 grid((unsigned)((nchunk + kQuantChunks - 1) / kQuantChunks), (unsigned)((n_tok + 31) / 32));
  const uint8_t* qs = qact + (size_t)t_pad * (size_t)id;
  const auto kernel = type == QMM_F32 ? dequantize_kernel<QMM_F32>
                    : type == QMM_F16 ? dequantize_kernel<QMM_F16> : dequantize_kernel<QMM_BF16>;
  kernel<<<grid, dim3(256), 0, s>>>(qact, qs, (int)n_tok, (int)nchunk, out, out_stride);
  return hipGetLastError();
}

}  // namespace qmm
