/*
 * qmm.h -- C ABI of libqmm: the prefill matrix multiply ("MMQ") of llama.cpp-style
 * k-quant weights (q6_K, q4_K) against activations quantized to q8 blocks of 32,
 * on AMD Instinct MI355X (gfx950).
 *
 *   out[t][j] = sum over k of  weight[j][k] * activation[t][k]
 *
 * computed the way the engineering log "minfer / cuda_optimization_steps"
 * describes it (pages "48 - r45 - cp.async for the q6_K A-side staging",
 * "59 - r56 - q6_K A-side bundle: A cp.async + W_dsc f32 plane", "61 - r58 -
 * q4_K BT spec + cp.async-db2 transplant"): the activations are first quantized
 * by a prepass into q8 blocks with a scale pair (r45 section 1.1), the weights
 * are expanded once at registration into planes the kernel can copy without
 * arithmetic (r56 sections 2.2-2.3, r58 section 3.2), and the GEMM forms exact
 * integer dot products per 32-element block and applies the per-block scales in
 * binary32.
 *
 * Conventions for every entry point:
 *   - Return QMM_OK (0) on success or a negative QMM_E* code; qmm_last_error()
 *     then names the problem.  No entry point ever falls back to another path.
 *   - Every argument is validated before the first HIP call, so invalid calls
 *     fail identically on machines with and without a GPU.
 *   - "stream" is a hipStream_t passed as void* (NULL = the null stream).  Work
 *     is enqueued asynchronously on it; pointers the caller passes must stay
 *     valid until that work completes.  The library keeps no caller pointer past
 *     the call.
 *   - Device pointers belong to the device that is current when the call is
 *     made; a weights handle is bound to the device current at registration and
 *     may only be used while that device is current.
 *   - Handles are immutable after registration: concurrent qmm_mmq calls on
 *     different streams may share one handle.
 */
#ifndef QMM_H
#define QMM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Weight block types. */
#define QMM_Q4_K 4 /* 144-byte blocks of 256 weights: f16 d, f16 dmin, 12 bytes of
                      6-bit scales and mins (8 sub-blocks of 32), 128 bytes of
                      4-bit codes; weight = d*scale*code - dmin*min
                      (r58 sections 2.2, 3.1). */
#define QMM_Q6_K 6 /* 210-byte blocks of 256 weights: ql[128] low 4 bits,
                      qh[64] high 2 bits, int8 scales[16] (one per 16 weights),
                      f16 d; weight = d*scale*(code - 32)
                      (r56 sections 1, 3.2; r58 section 3.2). */
#define QMM_Q4_K_PACKED 14 /* q4_K blocks (the same 144-byte input as QMM_Q4_K)
                      registered with the 4-bit codes kept two per byte in the
                      device plane, as the raw qs bytes hold them (r58 section
                      2.2): 0.5 instead of 1 byte per weight, unpacked by the
                      GEMM.  Results are bit-identical to QMM_Q4_K's. */

/* The rows forms: the same blocks registered for qmm_mmv, kept at the blocks' own
 * size (0.5625 and 0.8203 bytes per weight).  The MMQ needs the
 * types above; a program that runs both registers a matrix twice. */
#define QMM_Q4_K_ROWS 24
#define QMM_Q6_K_ROWS 26

/* Element types of activation tensors. */
#define QMM_F32 0
#define QMM_F16 1
#define QMM_BF16 2
#define QMM_Q8 3 /* as the output or input of a product: q8 blocks, a qact buffer */

/* Return codes. */
#define QMM_OK 0
#define QMM_EINVAL (-1) /* bad argument: type, size, null or misaligned pointer */
#define QMM_ESHAPE (-2) /* buffers that do not belong together (qact vs handle) */
#define QMM_ENOMEM (-3) /* device memory could not be allocated; nothing leaked */
#define QMM_EHIP (-4)   /* a HIP runtime call or kernel launch failed */

/* Size limits (validated): 1 <= od <= QMM_MAX_OD, 256 <= id <= QMM_MAX_ID with
 * id % 256 == 0, 0 <= n_tok <= QMM_MAX_TOKENS.  n_tok == 0 is an empty batch:
 * qmm_qact_bytes gives 0, and qmm_quantize_activations and qmm_mmq (with
 * qact_bytes 0) return QMM_OK without touching any pointer or the device. */
#define QMM_MAX_OD (1 << 21)
#define QMM_MAX_ID (1 << 20)
#define QMM_MAX_TOKENS (1 << 20)

/* Compute units a launch plan (qmm_mmq_plan) may be asked for: 1 .. QMM_MAX_CUS. */
#define QMM_MAX_CUS 65536

/* Largest stride (in elements) from row to row of a strided tensor. */
#define QMM_MAX_STRIDE (1 << 24)

/* Most tokens of one qmm_mmv. */
#define QMM_MV_MAX_TOKENS 16

/* Tokens are padded to a multiple of this many in the qact buffer. */
#define QMM_TOKEN_PAD 128

typedef struct qmm_weights qmm_weights;

typedef struct {
    int type;            /* QMM_Q4_K, QMM_Q4_K_PACKED, QMM_Q6_K, QMM_Q4_K_ROWS or QMM_Q6_K_ROWS */
    int64_t od;          /* output rows */
    int64_t id;          /* inner dimension */
    int64_t od_pad;      /* rows padded with zeros to the row tile (rows forms: to 16) */
    size_t raw_bytes;    /* od * (id/256) * (144 or 210): the k-quant bytes */
    size_t plane_bytes;  /* device memory the handle holds */
    size_t wd_offset;    /* byte offset of the d plane (q6_K; q4_K: == plane_bytes);
                            rows forms: of the plane after the codes */
    size_t sm_offset;    /* byte offset of the stage-record plane of scales, mins,
                            d and dmin (q4_K; q6_K: == plane_bytes); q6_K rows:
                            of the scales (q4_K rows: == plane_bytes) */
} qmm_info;

/*
 * qmm_register_weights -- copy one k-quant weight matrix to the device and
 * expand it once into the planes the GEMM reads (the registration-time planes
 * of r56 section 2.2 and r58 section 3.2; layout: see qmm_weights_export).
 *   type        QMM_Q4_K, QMM_Q4_K_PACKED (q4_K blocks, codes kept packed on
 *               the device) or QMM_Q6_K for the MMQ; QMM_Q4_K_ROWS or
 *               QMM_Q6_K_ROWS for qmm_mmv
 *   od, id      the weight is od rows of id weights; id % 256 == 0.  Any od >= 1
 *               (odd included) is valid: rows are padded with zeros internally.
 *   host_bytes  host memory, od rows * (id/256) blocks, row major, exactly
 *               nbytes = od * (id/256) * (144 for both q4_K types, 210 for
 *               q6_K) bytes.  Copied; the caller
 *               keeps ownership and may free it when the call returns.
 *   stream      the copy and the expansion run on it; the call returns after
 *               both completed (it synchronizes the stream).
 *   out         receives the handle; release with qmm_release_weights.
 * Errors: QMM_EINVAL (type, sizes, nullptrs, nbytes mismatch), QMM_ENOMEM (device
 * memory or the cap of qmm_set_memory_cap), QMM_EHIP.  On error *out is left NULL
 * and no device memory stays allocated.
 */
int qmm_register_weights(int type, int64_t od, int64_t id, const void *host_bytes,
                         size_t nbytes, void *stream, qmm_weights **out);

/* qmm_weights_info -- sizes of a handle.  QMM_EINVAL on null pointers. */
int qmm_weights_info(const qmm_weights *w, qmm_info *out);

/*
 * qmm_weights_export -- copy a handle's device planes to host memory, for
 * inspection and byte-exact tests (the r56 section 4 plane read-back gate).
 * host must hold exactly bytes = info.plane_bytes.  Synchronous.
 * Plane layout (R = od_pad/32 row blocks of 32 rows, nchunk = id/32, nsb =
 * id/256; rows od..od_pad-1 are zero everywhere):
 *   at 0          q6_K: int8 [R][nchunk][2][2][32][16]: the scale-folded weight
 *                 w = scale[k/16] * (code - 32) of (row j, k) as w = 64*hi + lo
 *                 (lo in [0, 63]), hi (plane index p = 0) and lo (p = 1) at byte
 *                 ((j/32*nchunk + k/32)*2 + p)*1024 + ((k%32)/16)*512
 *                 + (j%32)*16 + k%16
 *                 q4_K: int8 [R][nchunk][2][32][16]: the 4-bit code (0..15)
 *                 of (row j, k) at byte (j/32*nchunk + k/32)*1024
 *                 + ((k%32)/16)*512 + (j%32)*16 + k%16
 *                 q4_K packed: uint8 [R][nchunk][2][32][8]: the code of
 *                 (row j, k) in the low nibble (k%16 < 8) or the high nibble
 *                 (k%16 >= 8) of byte (j/32*nchunk + k/32)*512
 *                 + ((k%32)/16)*256 + (j%32)*8 + k%8
 *   at wd_offset  q6_K only: f32 [R][nsb][32]: d of (row j, super-block b) at
 *                 element (j/32*nsb + b)*32 + j%32
 *   at sm_offset  q4_K only (both q4_K types): [R][nchunk/4][1024 bytes], one
 *                 record per (row block, stage g of chunks 4g..4g+3) at byte
 *                 (j/32*nchunk/4 + g)*1024, each holding
 *                 +0    binary16 [32][4]: the 6-bit scale of (row j, chunk
 *                       4g + i) as an integer at element (j%32)*4 + i
 *                 +256  binary16 [2][32][4]: the 6-bit min of (row j, chunk
 *                       8b + 4h + i) of the stage's super-block b = g/2 as an
 *                       integer at element (h*32 + j%32)*4 + i
 *                 +768  f32 [2][32]: d*2^25 (part 0) and -dmin (part 1) of
 *                       (row j, super-block b) at element part*32 + j%32; both
 *                       exact in binary32, zeros stored as +0
 *                 (the two records of a super-block both hold its mins, d and
 *                 dmin)
 * Rows forms: tiles of 16 rows (row j is row n = j%16 of its tile) by nsb blocks;
 * planes start at multiples of 256 bytes.  Byte group g of half h of a block is
 * bytes 64h + 16g .. + 15 of its 128 code bytes.
 *   at 0          [od_pad/16][nsb][h][g][n][16 bytes]: the code bytes, q6_K the low
 *                 code bits
 *   at wd_offset  q4_K [od_pad/16][nsb][n][4 words]: word i from its lowest bit: the
 *                 six-bit scale and min of 32-block 2i, scale and min of 2i + 1, then
 *                 byte i of the block's binary16 d and dmin
 *                 q6_K [od_pad/16][nsb][g][n][h][8 bytes]: the high code bits: bits
 *                 2j, 2j + 1 of byte b are those of the code in the low nibble
 *                 (b < 4) or the high nibble (b >= 4) of the byte group's byte
 *                 4j + b%4, the upper one inverted
 *   at sm_offset  q6_K [od_pad/16][nsb][n][16]: the int8 scales plus 128
 *   after it      q6_K [od_pad/16][nsb][n]: binary16 d
 * Errors: QMM_EINVAL (null pointers, bytes mismatch), QMM_EHIP.
 */
int qmm_weights_export(const qmm_weights *w, void *host, size_t bytes);

/* qmm_release_weights -- free a handle's device memory.  Not safe while work
 * that uses the handle is still in flight: synchronize first.  NULL is a no-op. */
void qmm_release_weights(qmm_weights *w);

/*
 * qmm_set_memory_cap -- upper bound on the device memory (bytes) that all live
 * handles of this process may hold together; registration that would exceed
 * it fails with QMM_ENOMEM before allocating.  0 removes the cap (default).
 * For callers that budget HBM between several consumers.
 */
void qmm_set_memory_cap(size_t bytes);

/*
 * qmm_qact_bytes -- size of the quantized-activation buffer for n_tok tokens of
 * id activations: T_pad * id * 9 / 8 with T_pad = n_tok rounded up to
 * QMM_TOKEN_PAD.  Returns 0 for n_tok == 0 (an empty batch) and if n_tok or
 * id is out of range.
 */
size_t qmm_qact_bytes(int64_t n_tok, int64_t id);

/*
 * qmm_quantize_activations -- the quantize-transpose prepass (r45 section 1.1):
 * f32 activations -> q8 blocks of 32 with a scale pair (r45 section 2.3: 32
 * int8 values plus 4 bytes; r56 section 1: "d/ssum").
 *   x           device f32 [n_tok][id], row major, 16-byte aligned.  Values
 *               must be finite with |x| <= 2046 (so the scaled sum fits f16);
 *               other values give unspecified (but memory-safe) results in their
 *               block: after NaN or an infinity its scale is not finite either, so
 *               that a token which reads it has no finite product.
 *   qact        device buffer of exactly qact_bytes = qmm_qact_bytes(n_tok, id)
 *               bytes, 16-byte aligned, fully overwritten.
 * Per token t and block c of 32 activations x_k:
 *   amax = max |x_k|;  dh = f16(amax / 127)   (binary32 division, f16 round to
 *   nearest even);  q_k = clamp(rint(x_k / dh), -127, 127) (binary32 division,
 *   round half to even) or 0 when dh == 0;  s = f16(dh * sum q_k).
 * Layout of qact (T_pad tokens; tokens >= n_tok are all zero; nchunk = id/32):
 *   q plane at byte 0, 1024-byte fragments per (32-token block tb, chunk c):
 *     q of (t, k) at ((t/32)*nchunk + k/32)*1024 + ((k%32)/16)*512
 *                    + (t%32)*16 + k%16
 *   scale plane at byte T_pad*id, 128 bytes per (tb, c):
 *     (dh, s) of (t, c) at T_pad*id + ((t/32)*nchunk + c)*128 + (t%32)*4,
 *     two little-endian binary16 values, dh first.
 * Errors: QMM_EINVAL (sizes, null/misaligned pointers, qact_bytes mismatch),
 * QMM_EHIP.
 */
int qmm_quantize_activations(const float *x, int64_t n_tok, int64_t id, void *qact,
                             size_t qact_bytes, void *stream);

/*
 * qmm_dequantize_activations -- read a qact buffer back: out[t][k] = dh * q, the
 * number each code stands for, rounded once to the element type (a product of
 * an f16 and a 7-bit integer: exact in f32).
 *   qact, qact_bytes  a buffer for these n_tok and id, 16-byte aligned
 *   type        QMM_F32, QMM_F16 or QMM_BF16
 *   out         device [n_tok] rows of id elements, out_stride elements from
 *               row to row (>= id, a multiple of 4); 16-byte aligned.  Padding
 *               tokens are not written.  Must not overlap qact.
 * Errors: QMM_EINVAL, QMM_EHIP.
 */
int qmm_dequantize_activations(const void *qact, size_t qact_bytes, int64_t n_tok, int64_t id,
                               int type, void *out, int64_t out_stride, void *stream);

/* Norm kinds: over a row x of id elements,
 *   QMM_NORM_RMS    x_k / sqrt(mean(x^2) + eps) * weight_k + bias_k
 *   QMM_NORM_LAYER  (x_k - mean(x)) / sqrt(mean((x - mean(x))^2) + eps) * weight_k + bias_k */
#define QMM_NORM_RMS 0
#define QMM_NORM_LAYER 1

/* What qmm_norm_quantize works on.  Zero the struct, then set what is wanted.
 * Tensors are device memory of n_tok rows of id elements of `type`, a stride
 * (in elements) from row to row: a multiple of 4 in [id, QMM_MAX_STRIDE];
 * pointers 16-byte aligned.  The vectors are f32 [id], 16-byte aligned. */
typedef struct {
    int32_t type;             /* QMM_F32, QMM_F16 or QMM_BF16: h, y, gate, h_out, normed */
    int32_t kind;             /* QMM_NORM_RMS or QMM_NORM_LAYER, both norms */
    float eps;                /* > 0, finite */
    float residual_scale;     /* rs: factor of h in the sum */
    float block_scale;        /* bs: factor of the block's part in the sum */
    const void *h;            /* the residual stream */
    int64_t h_stride;
    const void *y;            /* the block's output, or NULL: nothing is added */
    int64_t y_stride;
    const float *post_weight; /* norm after the block, of y: its weight, or NULL: y as it is */
    const float *post_bias;   /* its bias or NULL (only with post_weight) */
    const void *gate;         /* factor of the block's part, or NULL (only with y): */
    int64_t gate_stride;      /* 0: one row for every token, else a row per token */
    const float *weight;      /* norm before the next block, of the sum: its weight ... */
    const float *bias;        /* ... and bias, or NULL */
    void *h_out;              /* receives the sum, or NULL */
    int64_t h_out_stride;
    void *normed;             /* receives the norm of the sum, or NULL */
    int64_t normed_stride;
    void *qact;               /* receives the norm of the sum as q8 blocks, or NULL */
    size_t qact_bytes;        /* qmm_qact_bytes(n_tok, id), or 0 without qact */
} qmm_norm;

/*
 * qmm_norm_quantize -- what stands between two blocks of a layer, in one pass
 * per row: the norm after a block, its gate, the scaled residual sum, the norm
 * before the next block and its quantization for the next qmm_mmq.
 *   u      = gate * norm(y; post_weight, post_bias)   (each step where given)
 *   s      = rs * h + bs * u, rounded once to `type`  (rs * h without y)
 *   h_out  = s
 *   n      = norm(s; weight, bias)
 *   normed = n rounded to `type`;  qact = the q8 blocks of n, not of its
 *            rounding, as qmm_quantize_activations writes them (padding
 *            tokens zero; |n| <= 2046 as there)
 * At least one of h_out, normed and qact is given; everything is computed in
 * f32, and the second norm is that of s as `type` holds it, whether h_out is
 * stored or not.  A row's result does not depend on the other rows or on which
 * outputs are wanted.  A row whose squares do not add up to a finite f32 (it holds
 * an infinity or NaN, or the sum passes 3.4e38) has NaN as its norm in every
 * element; other rows do not change.
 * An output may be one of the inputs in place (same pointer and stride): h_out
 * may be h or y; normed may be y, or h where h_out is NULL.  Any other overlap
 * of an output with h, y, gate or another output is refused.
 * No workspace; can be captured into a graph.
 * Errors: QMM_EINVAL, QMM_EHIP.  n_tok == 0 is an empty batch.
 */
int qmm_norm_quantize(const qmm_norm *args, int64_t n_tok, int64_t id, void *stream);

/*
 * qmm_mmq -- the GEMM: out[t][j] = sum over 32-blocks c of
 *   q6_K: sum over the block's two 16-groups g of d*sc_g*dh_c*D16_g
 *   q4_K: d*sc_c*dh_c*D32_c - dmin*min_c*s_c
 * with D the exact integer dot of the weight codes (q6_K: code - 32) and the q8
 * codes over the group (r56 section 2.2 for the q6_K d*sc pairs).  The integer
 * parts are exact; the scales are applied and summed in binary32 (error within
 * 1e-4 of the sum of the terms' magnitudes).
 *   w           handle from qmm_register_weights (current device = its device)
 *   qact        buffer written by qmm_quantize_activations for these n_tok and
 *               the handle's id; qact_bytes must equal qmm_qact_bytes(n_tok,
 *               id) or the call fails with QMM_ESHAPE.  16-byte aligned.
 *   out         device f32 [n_tok][od], row major, 4-byte aligned; every element
 *               is overwritten (no accumulation), nothing outside is written.
 * When the output tiles fill the GPU's compute units a whole number of times
 * plus a small remainder, the remainder's tiles are split along the inner
 * dimension into partial sums that a second kernel adds in a fixed order.  Their
 * scratch is one device buffer per (device, stream) of 64 KiB per compute unit
 * (16 MiB on MI355X), allocated with hipMalloc by the first call on that stream
 * that needs it and kept until qmm_stream_release or the end of the process;
 * calls on one stream share it in stream order, also when several threads make
 * them (a call's two kernels are enqueued with nothing in between).  For
 * hipStreamPerThread it is one buffer per (device, thread).  Synchronize a stream
 * before destroying it if an MMQ on it may still run.  Results are deterministic:
 * the same call gives the same bits.
 * Errors: QMM_EINVAL (also for a shape whose tiles exceed one launch: n_tok * od
 * beyond about 6.9e10, i.e. an output of 275 GB), QMM_ESHAPE, QMM_ENOMEM (the
 * scratch), QMM_EHIP.
 */
int qmm_mmq(const qmm_weights *w, const void *qact, size_t qact_bytes, int64_t n_tok,
            float *out, void *stream);

/*
 * qmm_stream_release -- give back the device memory qmm_mmq keeps for `stream`
 * (the tail-partials scratch above, on every device it was allocated for), for
 * callers that create and destroy streams: call it before destroying the
 * stream, with hipStreamPerThread before the thread ends (it gives back the calling
 * thread's).  It synchronizes `stream` first (an MMQ on it may still read the
 * partials), then frees; a later qmm_mmq on the same stream allocates again.
 *   freed_bytes  NULL, or receives the bytes freed (0 if the stream held none).
 * A stream that holds nothing returns QMM_OK without any HIP call.  Not safe
 * concurrently with a qmm_mmq on the same stream from another thread.
 * Errors: QMM_EHIP (the stream's synchronization or the free failed; what was
 * not freed stays held and *freed_bytes counts what was).
 */
int qmm_stream_release(void *stream, size_t *freed_bytes);

/*
 * qmm_mmq_noalloc -- qmm_mmq for callers that cannot allocate device memory:
 * code under HIP graph capture, tight serving loops, harnesses that forbid
 * allocation.  Same arguments, validation, kernels and results (bit for bit)
 * as qmm_mmq; it calls no hipMalloc, hipFree or other allocating routine.  The
 * tail partials (see qmm_mmq) live in a static device array of 16 MiB that
 * every GPU the library runs on holds until the process ends; its address is
 * looked up (hipGetSymbolAddress) on the first call on each device.
 *   - Every call on one GPU shares that GPU's array and leaves the last call's
 *     partials in it: calls that may overlap on one GPU (different streams
 *     without ordering between them) race.  Calls on one stream are ordered, from
 *     one thread or several.
 *   - Nothing in the array needs clearing: each partial is written whole
 *     before it is read.
 *   - A launch that needs more than 16 MiB of partials (only on GPUs with more
 *     than 256 compute units) fails with QMM_EINVAL before any launch.
 * Errors: as qmm_mmq, without QMM_ENOMEM.
 */
int qmm_mmq_noalloc(const qmm_weights *w, const void *qact, size_t qact_bytes, int64_t n_tok,
                    float *out, void *stream);

/* Activations of an epilogue. */
#define QMM_ACT_NONE 0
#define QMM_ACT_RELU 1
#define QMM_ACT_SILU 2      /* x / (1 + exp(-x)) */
#define QMM_ACT_GELU 3      /* x * (1 + erf(x / sqrt(2))) / 2 */
#define QMM_ACT_GELU_TANH 4 /* x * (1 + tanh(sqrt(2/pi) * (x + 0.044715 x^3))) / 2 */

/* What happens to a product's f32 sum v of (token t, row j) before it is stored:
 *   scale * mul[t][j] * act(v + bias[j]) + residual_scale * residual[t][j]
 * each part where given, in f32, rounded once.  Zero the struct, set scale to 1
 * and then what is wanted. */
typedef struct {
    const float *bias;     /* f32 [od], 4-byte aligned, or NULL */
    int32_t act;           /* QMM_ACT_* */
    int32_t type;          /* element type of mul and residual: QMM_F32, QMM_F16, QMM_BF16 */
    float scale;           /* finite */
    float residual_scale;  /* finite */
    const void *mul;       /* device [n_tok] rows of od elements, or NULL */
    int64_t mul_stride;    /* elements from row to row, in [od, QMM_MAX_STRIDE] */
    const void *residual;  /* device [n_tok] rows of od elements, or NULL */
    int64_t residual_stride;
} qmm_epilogue;

/*
 * qmm_mmq_epilogue -- qmm_mmq with an epilogue on its sums, stored in the type
 * and place the next step reads: one kernel instead of the product and an
 * elementwise pass over its output.  The sums are qmm_mmq's: bit for bit where
 * its tiled kernel runs, in another order of their f32 additions for few tokens
 * (up to 64, or a launch that small), which have a kernel of their own.  The same
 * call gives the same bits.
 *   w, qact, qact_bytes, n_tok, stream  as for qmm_mmq
 *   ep          the epilogue, or NULL: the sums themselves, rounded to out_type
 *   out_type    QMM_F32, QMM_F16 or QMM_BF16: out is device [n_tok] rows of od
 *               elements, out_stride elements from row to row (in [od,
 *               QMM_MAX_STRIDE]), aligned to its element.  Only the n_tok x od
 *               elements are written.
 *               QMM_Q8: out is a qact buffer of qmm_qact_bytes(n_tok, od) bytes
 *               (od % 256 == 0; 16-byte aligned) and out_stride is that number;
 *               it receives the q8 blocks of the values, as
 *               qmm_quantize_activations makes them of f32 values, padding
 *               tokens zero -- the next product's input (|values| <= 2046).
 *   work        device memory for the tail partials (see qmm_mmq), 16-byte
 *               aligned, work_bytes of it, at least the plan's scratch_bytes
 *               (qmm_mmq_plan; few tokens need none): the call then allocates
 *               nothing and can be captured, and calls with work memory of their
 *               own may overlap.  Calls that share it have to be on one stream (or
 *               ordered otherwise).
 *               NULL with work_bytes 0: the stream's scratch, as qmm_mmq; a
 *               captured call that needs scratch is then refused, since graphs
 *               replayed side by side would share it.
 * out may be mul or residual in place (same pointer, stride and type); any
 * other overlap of out or work with an input is refused.
 * Errors: as qmm_mmq.
 */
int qmm_mmq_epilogue(const qmm_weights *w, const void *qact, size_t qact_bytes, int64_t n_tok,
                     const qmm_epilogue *ep, int out_type, void *out, int64_t out_stride,
                     void *work, size_t work_bytes, void *stream);

/*
 * qmm_mmv -- the product for up to QMM_MV_MAX_TOKENS tokens straight from the
 * activations, in one kernel: decode steps, a few sequences at once.  The
 * numbers are the MMQ's: x is quantized to the q8 blocks that
 * qmm_quantize_activations writes, block dots are exact, scales are applied and
 * summed in f32 (in another order than qmm_mmq's).
 *   w           a handle of a rows form (current device = its device)
 *   x, x_type   device [n_tok] rows of id activations, QMM_F32, QMM_F16 or
 *               QMM_BF16, x_stride elements from row to row (a multiple of 4 in
 *               [id, QMM_MAX_STRIDE]); aligned to four elements; |x| <= 2046.
 *               Or QMM_Q8: the qact buffer of these tokens (16-byte aligned), as
 *               qmm_norm_quantize and qmm_quantize_activations write it, and
 *               x_stride its qmm_qact_bytes(n_tok, id) bytes; the same results
 *               as from the numbers it was made of, and from about 2^16 values
 *               on in less time than from numbers, with the time of
 *               qmm_quantize_activations counted in
 *   ep, out_type, out, out_stride  as for qmm_mmq_epilogue
 * No workspace; can be captured into a graph.  Deterministic; a token's result
 * may depend in its last bits on how many tokens the call has.
 * Errors: QMM_EINVAL, QMM_ESHAPE (a qact of another size), QMM_EHIP.  n_tok == 0 is
 * an empty batch.
 */
int qmm_mmv(const qmm_weights *w, const void *x, int x_type, int64_t x_stride, int64_t n_tok,
            const qmm_epilogue *ep, int out_type, void *out, int64_t out_stride, void *stream);

/* ---- between the q, k, v products and the output product: positions, a paged cache, attention ---- */

/* A paged cache of keys and values.  A slot holds one token's key (in the pool k)
 * and value (in the pool v) of every head, head_dim channels each; a page holds
 * `page` slots, and each pool n_pages pages of qmm_cache_page_bytes bytes,
 * 16-byte aligned.  The caller owns the pools; nothing in them needs clearing (what
 * no sequence's slot in use holds is never part of a result).  Leftovers that are no
 * finite numbers, in values of tiles that are partly in use, cost time though: attention
 * does such work again (decode steps took up to 2 times as long, prompts and chunks 6 to
 * 20 times), which a pool that was cleared once does not meet.
 *   type     QMM_F16, QMM_BF16, or QMM_Q8: blocks of 32 channels of a slot, int8
 *            codes and an f16 scale as qmm_quantize_activations makes them (the
 *            scaled sum left out; |values| <= 2046 as there), 1.0625 bytes a value
 *   head_dim 64, 96, 128, 192 or 256
 *   page     a power of two in [32, QMM_MAX_PAGE]
 * Layout of a pool (the fragment order of the matrix instructions): pages, in a
 * page heads, in a head tiles of 32 slots.  In a tile, of slot r and channel d,
 * with D = head_dim and m(r) = r with its bits 2 and 3 exchanged,
 *   16 bits  k: element ((d/16*2 + d%16/8)*32 + m(r))*8 + d%8
 *            v: element ((d/32*4 + r/8)*32 + d%32)*8 + r%8
 *   q8       k: byte d/32*1024 + ((d%16/8)*32 + m(r))*16 + d%32/16*8 + d%8
 *            v: byte d/32*1024 + ((r%16/8)*32 + d%32)*16 + r/16*8 + r%8
 *            each the code plus 128; both pools: the f16 scale of block d/32 at
 *            byte 32*D + (d/32*32 + r)*2 */
#define QMM_MAX_PAGE 65536
#define QMM_MAX_HEADS 4096
typedef struct {
    int32_t type;
    int32_t heads;    /* of keys and values, 1 .. QMM_MAX_HEADS */
    int32_t head_dim;
    int32_t page;
    int64_t n_pages;  /* 1 .. 2^31 - 1 */
    void *k, *v;      /* the pools, device memory */
} qmm_cache;

/* qmm_cache_page_bytes -- bytes of one page of one pool; 0 if an argument is out of
 * range. */
size_t qmm_cache_page_bytes(int type, int heads, int head_dim, int page);

/* The sequences of a call.  Sequence s has the call's tokens (rows) starts[s] ..
 * starts[s + 1] - 1, any number of them, none included, and lengths[s] slots in use
 * of the cache, of which its tokens of this call are the last: token i of n has slot
 * lengths[s] - n + i.  Slot j is slot j % page of page table[s][j / page].
 * The arrays are device memory, read when the kernels run.  Whatever they hold,
 * nothing outside the tensors and pools is read or written: a start is taken
 * within [0, n_tok] and as the highest up to it, so that no token has two
 * sequences, lengths within the table's columns; tokens without a slot (more than
 * lengths[s]) and pages outside the pool are not followed: nothing is stored to
 * them, and their keys are not seen.
 * max_new, max_length: the most tokens and the most slots of any sequence, to size
 * the launch by; a result does not go by them, but for its roundings.  Sequences
 * that pass them are worked through all the same, only slower; a max_length far above
 * the lengths is slower too, since attention's parts of the keys are then of the size
 * that they have in a sequence of max_length (one token of 32/8 heads of 128 over
 * 3314 slots: 11.2 us with 3314, 12.9 with 8192, 17.1 with 32768, 25.8 with
 * 131072). */
#define QMM_MAX_SEQS 65535
#define QMM_MAX_SLOTS (1 << 30) /* of a sequence */
typedef struct {
    int32_t n_seq;         /* 1 .. QMM_MAX_SEQS */
    int32_t columns;       /* of the table, >= 1; columns * page <= QMM_MAX_SLOTS */
    const int32_t *starts; /* [n_seq + 1] */
    const int32_t *lengths;/* [n_seq] */
    const int32_t *table;  /* [n_seq] rows of `columns` page numbers */
    int64_t table_stride;  /* elements from row to row, >= columns */
    int64_t max_new;       /* 0 .. QMM_MAX_TOKENS */
    int64_t max_length;    /* 0 .. QMM_MAX_SLOTS */
} qmm_batch;

/* Rotary scalings for long contexts (qmm_rope_frequencies). */
#define QMM_ROPE_PLAIN 0
#define QMM_ROPE_LINEAR 1 /* every frequency divided by factor */
#define QMM_ROPE_BASE 2   /* the base times factor^(n_rot / (n_rot - 2)): the fastest pair stays, the slowest is divided */
#define QMM_ROPE_YARN 3   /* a ramp over the pairs from those that turn `fast` times in the original context, which
                             stay, to those that turn `slow` times, which are divided by factor; its ends are whole
                             pairs; magnitude 0.1 ln(factor) + 1 (1 where factor <= 1) */
#define QMM_ROPE_TURNS 4  /* the same with the ramp over the turns themselves, magnitude 1 */

/*
 * qmm_rope_frequencies -- the angle per position, in radians, of each of the n_rot/2
 * pairs: base^(-2i/n_rot), scaled.  Host arithmetic in 64 bits only; the caller
 * copies them to the device once.
 *   n_rot       a multiple of 16 in [16, 256]
 *   base        > 1, finite
 *   scaling     QMM_ROPE_*; factor > 0; YARN and TURNS: original > 0 (the context
 *               before scaling), fast > slow > 0
 *   frequencies host [n_rot / 2];  magnitude  host, or NULL
 * Errors: QMM_EINVAL.
 */
int qmm_rope_frequencies(int64_t n_rot, double base, int scaling, double factor, double original, double fast,
                         double slow, double *frequencies, float *magnitude);

#define QMM_ROPE_HALF 0        /* pair i: channels i and i + n_rot/2 */
#define QMM_ROPE_INTERLEAVED 1 /* pair i: channels 2i and 2i + 1 */

/* What qmm_rope_cache works on.  Zero the struct, then set what is wanted.  q, k
 * and v are device tensors [n_tok][heads][head_dim] with adjacent channels;
 * strides in elements, of tokens and heads, multiples of 8 in [head_dim,
 * QMM_MAX_STRIDE] (any value where there is one token or one head); 16-byte
 * aligned. */
typedef struct {
    int32_t type;      /* QMM_F32, QMM_F16 or QMM_BF16: q, k, v */
    int32_t out_type;  /* of q_out */
    int32_t q_heads;   /* 1 .. QMM_MAX_HEADS, with q */
    int32_t layout;    /* QMM_ROPE_HALF or QMM_ROPE_INTERLEAVED */
    int32_t n_rot;     /* channels rotated, a multiple of 16 in [0, head_dim] */
    float magnitude;   /* factor of the rotated channels, finite */
    const double *frequencies;  /* device [n_rot / 2] (not with n_rot 0) */
    const int32_t *positions;   /* device [n_tok], or NULL: a token's slot is its position */
    const void *q;              /* queries, or NULL */
    int64_t q_stride, q_head_stride;
    void *q_out;                /* receives them rotated */
    int64_t q_out_stride, q_out_head_stride;
    const void *k;              /* keys, rotated and kept in the cache, or NULL */
    int64_t k_stride, k_head_stride;
    const void *v;              /* values, kept in the cache as they are, or NULL */
    int64_t v_stride, v_head_stride;
} qmm_rope;

/*
 * qmm_rope_cache -- the new tokens' queries and keys turned by their positions, and
 * keys and values kept in their slots, in one pass:
 *   pair (a, b) at position p with frequency f: t = p * f,
 *   (a, b) -> magnitude * (a cos t - b sin t, a sin t + b cos t)
 * t is formed and reduced in 64 bits, the rest is f32; a result is rounded once to
 * the type it is kept in (q8: the blocks of the f32 values).  Channels from n_rot on
 * stay as they are.
 *   cache     k and v, where given, go there; with q alone its head_dim counts
 *   args      at least one of q, k and v
 * q_out may be q in place (same type, pointer and strides); any other overlap of
 * an output with an input is refused.  Rows of tokens of no sequence are left as
 * they are, and slots of other tokens too.  Two tokens of a call never have one
 * slot unless the table names a page twice, in two sequences or in one: what such a
 * slot then holds is open (in q8, codes of one and the scale of the other).
 * No workspace; can be captured into a graph.
 * Errors: QMM_EINVAL, QMM_EHIP.  n_tok == 0 is an empty batch.
 */
int qmm_rope_cache(const qmm_rope *args, const qmm_cache *cache, const qmm_batch *batch, int64_t n_tok, void *stream);

/*
 * qmm_cache_read -- the keys and values that the cache holds for the batch's tokens
 * (their slots as above), as numbers: with starts spaced by the lengths, whole
 * sequences.
 *   type        QMM_F32, QMM_F16 or QMM_BF16
 *   k, v        device [n_tok][heads][head_dim], contiguous, 16-byte aligned; either
 *               may be NULL.  Rows of tokens of no sequence are left as they are;
 *               tokens without a slot, or in a page outside the pool, are zeros.
 * Errors: QMM_EINVAL, QMM_EHIP.
 */
int qmm_cache_read(const qmm_cache *cache, const qmm_batch *batch, int64_t n_tok, int type, void *k, void *v,
                   void *stream);

/* What qmm_attention works on.  Zero the struct, then set what is wanted. */
typedef struct {
    int32_t heads;     /* of q: a multiple of the cache's */
    int32_t causal;    /* 1: a token sees the slots up to its own; 0: all in use (an
                          encoder's states, of a length that has nothing to do with
                          the tokens') */
    int32_t out_type;  /* q's type (QMM_F16, QMM_BF16) or QMM_Q8 */
    float scale;       /* of the scores, in [1e-30, 1e30] */
    int64_t window;    /* causal: of those only the last `window`; 0: all */
    const void *q;     /* device [n_tok][heads][head_dim], adjacent channels, of the
                          cache's type (QMM_F16 with a q8 cache), 16-byte aligned */
    int64_t q_stride, q_head_stride;  /* as in qmm_rope */
    void *out;         /* [n_tok] rows of heads * head_dim elements, out_stride from row
                          to row, a multiple of 8; 16-byte aligned.  QMM_Q8: a qact buffer of
                          qmm_qact_bytes(n_tok, heads * head_dim) bytes, and
                          out_stride that number: the output product's input */
    int64_t out_stride;
} qmm_attn;

/*
 * qmm_attention -- attention of the batch's tokens over the cache: for token i,
 * head h and the keys j that it sees, of cache head h / (heads / cache heads),
 *   p_j = exp(scale * q.k_j - max_j),   out = sum_j p_j v_j / sum_j p_j
 * Products are of 16-bit values summed in f32; maximum and sum are f32; p_j is
 * rounded to q's type for the second product (f16: with weights down to 2^-22 of the
 * largest one in full, smaller ones to 2^-33 of it), q8 keys and values to f16.
 * Scores times scale stay below 2^126 in size, and values times the number of keys
 * below 2^120 (bf16), or are no numbers in what comes of them.  A token that sees no
 * key, or none whose score is above -infinity, gets zeros, whatever the values are.
 * What a token does not see is no part of its result, whatever is stored there.  An
 * output in q8 blocks has its padding tokens zero; rows of tokens of no sequence are
 * left as they are.
 *   work      device memory of at least the plan's work_bytes (qmm_attention_plan),
 *             16-byte aligned; NULL with 0 where it needs none.  Calls that share it
 *             have to be on one stream (or ordered otherwise); nothing in it needs
 *             clearing.
 * The output must not overlap an input or the work memory.  Deterministic: the
 * same call gives the same bits.  Can be captured into a graph.
 * Errors: QMM_EINVAL, QMM_EHIP.  n_tok == 0 is an empty batch.
 */
int qmm_attention(const qmm_attn *args, const qmm_cache *cache, const qmm_batch *batch, int64_t n_tok, void *work,
                  size_t work_bytes, void *stream);

/* How a qmm_attention is launched: the (token, head of its group) pairs of a
 * sequence and a cache head are columns, taken `columns` at a time; the keys of
 * such a tile are split into up to `splits` parts of whole 32-slot tiles, `share` of
 * them each (more where max_length is passed), whose partial results a second
 * kernel joins. */
typedef struct {
    size_t work_bytes;   /* partial results (0: none) */
    int64_t work_groups;
    int32_t few;         /* 1: few columns, the waves of a work-group take turns over
                            the keys; 0: each takes columns of its own */
    int32_t columns;
    int32_t tiles;       /* column tiles of a sequence and cache head with max_new, or
                            as many as work-groups take turns over (many sequences) */
    int32_t splits;
    int32_t share;
} qmm_attn_plan;

/*
 * qmm_attention_plan -- the plan of qmm_attention for these sizes on a GPU with
 * num_cus compute units; host arithmetic only.  Of `cache` type, heads and head_dim
 * count, of `batch` n_seq, max_new and max_length; heads and window as in qmm_attn.
 * Errors: QMM_EINVAL.
 */
int qmm_attention_plan(const qmm_cache *cache, const qmm_batch *batch, int heads, int64_t window, int64_t n_tok,
                       int num_cus, qmm_attn_plan *out);

/* The launch plan of one MMQ (qmm_mmq, qmm_mmq_noalloc): how its output tiles
 * map onto work-groups on a GPU of a given size, and the tail partials it needs.
 * The slots are the work-groups resident at once (per_cu per compute unit).  The
 * tiles of the whole waves, rounded down to whole row tiles (dp_row_tiles of
 * them, all tokens), run one work-group each.  The remaining row tiles' tiles
 * are split along the inner dimension into `split` slices of whole super-blocks,
 * computed by separate work-groups as f32 partial tiles that a second kernel
 * adds, when they form a partial wave: after at most one full wave (none
 * included: a launch filling at most half the GPU splits every tile), or, with
 * one or two work-groups per compute unit, a last wave of at most a quarter of
 * the slots behind several full ones -- and when there are at least two slices
 * to make (every wave group of a slice keeps a super-block). */
typedef struct {
    int64_t work_groups;   /* work-groups of the MMQ launch (0: an empty batch) */
    size_t scratch_bytes;  /* tail partials the call needs, n_tail * split partial
                              tiles of f32 (0: none); qmm_mmq_noalloc refuses a
                              call that needs more than its 16 MiB */
    int32_t threads;       /* threads per work-group */
    int32_t many;          /* 1: the many-tile geometry (several work-groups per
                              compute unit); 0: the few-tile one */
    int32_t tile_rows;     /* output rows per tile */
    int32_t tile_tokens;   /* tokens per tile */
    int32_t k_groups;      /* wave groups per work-group, each taking its share
                              of the work-group's super-blocks */
    int32_t per_cu;        /* work-groups resident per compute unit */
    int32_t row_tiles;     /* tiles covering the od rows ... */
    int32_t tok_tiles;     /* ... and the n_tok tokens */
    int32_t dp_row_tiles;  /* row tiles computed whole (== row_tiles without a tail) */
    int32_t n_tail;        /* tiles split along the inner dimension:
                              (row_tiles - dp_row_tiles) * tok_tiles */
    int32_t split;         /* slices per tail tile (1: no tail) */
    int32_t nsb;           /* super-blocks along the inner dimension, id / 256 */
} qmm_plan;

/*
 * qmm_mmq_plan -- the plan qmm_mmq follows for a handle of this type, od and id
 * at n_tok tokens on a GPU with num_cus compute units (the device attribute
 * hipDeviceAttributeMultiprocessorCount; 256 on MI355X).  Host arithmetic only:
 * no HIP call, no device needed.  For callers that size work ahead, e.g. that
 * check that a qmm_mmq_noalloc call fits its scratch (scratch_bytes).
 *   type, od, id, n_tok  as for qmm_register_weights and qmm_mmq
 *   num_cus     1 .. QMM_MAX_CUS
 *   out         receives the plan (zeroed, nsb set, for n_tok == 0)
 * Errors: QMM_EINVAL (arguments out of range, as the other entry points check
 * them; a shape whose tiles exceed one launch).
 */
int qmm_mmq_plan(int type, int64_t od, int64_t id, int64_t n_tok, int num_cus, qmm_plan *out);

/*
 * qmm_mmq_plan_work -- what work-group wg (0 <= wg < plan->work_groups) of a
 * plan's MMQ launch computes, by the kernel's own mapping: the tile of row tile
 * *row_tile (rows tile_rows * row_tile ...) and token tile *tok_tile, over
 * super-blocks [*sb_begin, *sb_end) of the inner dimension (all nsb of them for
 * a whole tile).  Host arithmetic only.  For inspection and tests of the plan.
 * Errors: QMM_EINVAL (NULL pointers, wg out of range, a plan whose fields do
 * not fit together).
 */
int qmm_mmq_plan_work(const qmm_plan *plan, int64_t wg, int32_t *row_tile, int32_t *tok_tile,
                      int32_t *sb_begin, int32_t *sb_end);

/* qmm_last_error -- message for the calling thread's last failed call ("" if
 * none).  Valid until the thread's next call into the library. */
const char *qmm_last_error(void);

#ifdef __cplusplus
}
#endif
#endif /* QMM_H */
