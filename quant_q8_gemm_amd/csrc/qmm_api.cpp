// qmm_api.cpp -- the C ABI declared in include/qmm.h: argument validation (all of
// it before the first HIP call), weight-handle lifetime, device-memory
// accounting, and the launches.  No compute happens here.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <mutex>
#include <string>
#include <vector>

#include "../../include/qmm.h"
#include "qmm_attention.h"
#include "qmm_epilogue.h"
#include "qmm_internal.h"
#include "qmm_rope.h"

struct qmm_weights {
  qmm::Planes p;
  int device;
  size_t raw_bytes;
  size_t plane_bytes;
  size_t wd_offset;
  size_t sm_offset;
  void* alloc;  // one device allocation holding every plane
};

namespace {

thread_local std::string g_last_error;
std::atomic<size_t> g_held{0};  // device bytes held by live handles
std::atomic<size_t> g_cap{0};   // 0 = no cap

// Scratch for the MMQ's tail partials: one buffer per (device, stream), of the
// largest size any call can need on that device (64 KiB per compute unit).
// Calls on one stream run in order, so they share it; it lives until
// qmm_stream_release(stream) or the process ends.
struct Scratch {
  int device;
  hipStream_t stream;
  uint64_t thread;  // hipStreamPerThread: whose stream (this_thread), else 0
  void* ptr;
  size_t bytes;
};
std::mutex g_scratch_mu;
std::vector<Scratch> g_scratch;

// hipStreamPerThread is one handle for a stream of each thread, whose work
// overlaps.  Numbers are not used again (a thread's scratch may outlive it).
uint64_t this_thread(hipStream_t s) {
  static std::atomic<uint64_t> last{0};
  thread_local const uint64_t mine = ++last;
  return s == hipStreamPerThread ? mine : 0;
}

// Held while a product with a split tail and the kernel that adds its partials
// are enqueued: with another call's product between the two on the stream, the
// second would add that call's partials.  A stream always takes the same one of
// these; two streams that share one wait for each other's launches only.
std::unique_lock<std::mutex> launch_turn(hipStream_t s, size_t scratch_bytes) {
  static std::mutex turns[64];
  if (scratch_bytes == 0) return {};
  const uintptr_t v = (uintptr_t)s;
  return std::unique_lock<std::mutex>(turns[(v ^ (v >> 6) ^ (v >> 12)) % 64]);
}

int fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return code;
}

int fail_hip(hipError_t e, const char* what) {
  return fail(QMM_EHIP, "%s: %s", what, hipGetErrorString(e));
}

void ok() { g_last_error.clear(); }

size_t round_up(size_t v, size_t m) { return (v + m - 1) / m * m; }

size_t block_bytes(int type) { return qmm::is_q4k(type) || type == QMM_Q4_K_ROWS ? 144 : 210; }

const char* type_name(int type) {
  return type == QMM_Q6_K          ? "q6_K"
         : type == QMM_Q4_K        ? "q4_K"
         : type == QMM_Q4_K_PACKED ? "q4_K (codes packed)"
         : type == QMM_Q4_K_ROWS   ? "q4_K (rows)"
                                   : "q6_K (rows)";
}

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

int check_id(int64_t id) {
  if (id < 256 || id > QMM_MAX_ID || id % 256 != 0)
    return fail(QMM_EINVAL, "id must be a multiple of 256 in [256, %d], got %lld", QMM_MAX_ID,
                (long long)id);
  return QMM_OK;
}

// n_tok == 0 is an empty batch: valid, and the call does nothing
int check_tokens(int64_t n_tok) {
  if (n_tok < 0 || n_tok > QMM_MAX_TOKENS)
    return fail(QMM_EINVAL, "n_tok must be in [0, %d], got %lld", QMM_MAX_TOKENS, (long long)n_tok);
  return QMM_OK;
}

int64_t token_pad(int64_t n_tok) { return (n_tok + qmm::kTokenPad - 1) / qmm::kTokenPad * qmm::kTokenPad; }

int check_type(int type) {
  if (type != QMM_Q4_K && type != QMM_Q4_K_PACKED && type != QMM_Q6_K)
    return fail(QMM_EINVAL, "type must be QMM_Q4_K (%d), QMM_Q4_K_PACKED (%d) or QMM_Q6_K (%d)%s, got %d", QMM_Q4_K,
                QMM_Q4_K_PACKED, QMM_Q6_K, qmm::is_rows(type) ? " (a rows form has no MMQ)" : "", type);
  return QMM_OK;
}

int check_od(int64_t od) {
  if (od < 1 || od > QMM_MAX_OD)
    return fail(QMM_EINVAL, "od must be in [1, %d], got %lld", QMM_MAX_OD, (long long)od);
  return QMM_OK;
}

// The geometry part of a handle's planes (no memory): what the plan needs.
qmm::Planes plane_shape(int type, int64_t od, int64_t id) {
  qmm::Planes p{};
  p.type = type;
  p.od = od;
  p.id = id;
  p.od_pad = (int64_t)round_up((size_t)od, qmm::kRowPad);
  p.nsb = id / 256;
  p.nchunk = id / 32;
  return p;
}

// one-dimensional launch: work-groups x threads must stay below 2^32
int check_launch(const qmm::MmqPlan& plan, int64_t n_tok, int64_t od, int num_cus) {
  if ((uint64_t)plan.work_groups * (uint64_t)plan.threads >= (1ull << 32))
    return fail(QMM_EINVAL, "n_tok=%lld x od=%lld needs %lld work-groups, more than one launch holds",
                (long long)n_tok, (long long)od, (long long)plan.work_groups);
  if (plan.scratch_bytes > qmm::mmq_scratch_max_bytes(num_cus))
    return fail(QMM_EINVAL, "internal: tail scratch exceeds its bound");
  return QMM_OK;
}

}  // namespace

extern "C" {

const char* qmm_last_error(void) { return g_last_error.c_str(); }

void qmm_set_memory_cap(size_t bytes) { g_cap.store(bytes); }

size_t qmm_qact_bytes(int64_t n_tok, int64_t id) {
  if (n_tok < 0 || n_tok > QMM_MAX_TOKENS || id < 256 || id > QMM_MAX_ID || id % 256 != 0) return 0;
  return (size_t)token_pad(n_tok) * (size_t)id / 8 * 9;
}

int qmm_register_weights(int type, int64_t od, int64_t id, const void* host_bytes, size_t nbytes,
                         void* stream, qmm_weights** out) {
  if (out == nullptr) return fail(QMM_EINVAL, "out is NULL");
  *out = nullptr;
  const bool rows = qmm::is_rows(type);
  if (!rows)
    if (int rc = check_type(type)) return rc;
  if (int rc = check_od(od)) return rc;
  if (int rc = check_id(id)) return rc;
  if (host_bytes == nullptr) return fail(QMM_EINVAL, "host_bytes is NULL");
  const size_t expect = (size_t)od * (size_t)(id / 256) * block_bytes(type);
  if (nbytes != expect)
    return fail(QMM_EINVAL, "nbytes %zu != od*(id/256)*%zu = %zu", nbytes, block_bytes(type), expect);

  qmm::Planes p = plane_shape(type, od, id);
  // q6_K: codes, d; q4_K: codes, stage records (one of the last two is empty)
  const size_t off_wd = round_up(qmm::wq_bytes(type, p.od_pad, id), 256);
  const size_t off_sm = off_wd + round_up(qmm::wd_bytes(type, p.od_pad, id), 256);
  size_t plane_bytes = off_sm + round_up(qmm::wsm_bytes(type, p.od_pad, id), 256);
  const qmm::RowOffsets at = qmm::row_offsets(type, od, id);
  if (rows) {
    p.od_pad = qmm::row_pad(od);
    plane_bytes = at.bytes;
  }
  // reserve the bytes against the cap before allocating, atomically, so that
  // registrations on several threads cannot overshoot it together; every
  // failure below gives them back
  const size_t cap = g_cap.load();
  size_t held = g_held.load();
  do {
    if (cap != 0 && held + plane_bytes > cap)
      return fail(QMM_ENOMEM, "registration needs %zu device bytes; cap %zu, held %zu", plane_bytes,
                  cap, held);
  } while (!g_held.compare_exchange_weak(held, held + plane_bytes));

  // ---- first HIP call below this line ----
  hipStream_t s = (hipStream_t)stream;
  int device = 0;
  hipError_t e = hipGetDevice(&device);
  if (e != hipSuccess) {
    g_held -= plane_bytes;
    return fail_hip(e, "hipGetDevice");
  }
  void* alloc = nullptr;
  void* raw = nullptr;
  e = hipMalloc(&alloc, plane_bytes);
  if (e != hipSuccess) {
    (void)hipGetLastError();
    g_held -= plane_bytes;
    return e == hipErrorOutOfMemory ? fail(QMM_ENOMEM, "hipMalloc(%zu) failed: out of memory", plane_bytes)
                                    : fail_hip(e, "hipMalloc(planes)");
  }
  e = hipMalloc(&raw, nbytes);
  if (e != hipSuccess) {
    (void)hipGetLastError();
    (void)hipFree(alloc);
    g_held -= plane_bytes;
    return e == hipErrorOutOfMemory ? fail(QMM_ENOMEM, "hipMalloc(%zu) failed: out of memory", nbytes)
                                    : fail_hip(e, "hipMalloc(raw)");
  }
  if (rows) {
    uint8_t* const base = (uint8_t*)alloc;
    p.rows = {base, base + at.heads, base + at.scales, (uint16_t*)(base + at.d)};
  } else {
    p.wq = (int8_t*)alloc;
    p.wd = qmm::is_q4k(type) ? nullptr : (float*)((char*)alloc + off_wd);
    p.wsm = qmm::is_q4k(type) ? (uint8_t*)alloc + off_sm : nullptr;
  }
  int rc = QMM_OK;
  if ((e = hipMemcpyAsync(raw, host_bytes, nbytes, hipMemcpyHostToDevice, s)) != hipSuccess)
    rc = fail_hip(e, "hipMemcpyAsync(weights)");
  else if ((e = rows ? qmm::launch_repack_rows((const uint8_t*)raw, type, od, id, p.rows, s)
                     : qmm::launch_repack((const uint8_t*)raw, p, s)) != hipSuccess)
    rc = fail_hip(e, "repack launch");
  else if ((e = hipStreamSynchronize(s)) != hipSuccess)
    rc = fail_hip(e, "hipStreamSynchronize(registration)");
  (void)hipFree(raw);
  if (rc != QMM_OK) {
    (void)hipFree(alloc);
    g_held -= plane_bytes;
    return rc;
  }
  qmm_weights* w = new qmm_weights;
  w->p = p;
  w->device = device;
  w->raw_bytes = nbytes;
  w->plane_bytes = plane_bytes;
  w->wd_offset = rows ? at.heads : qmm::is_q4k(type) ? plane_bytes : off_wd;
  w->sm_offset = type == QMM_Q6_K_ROWS ? at.scales : qmm::is_q4k(type) ? off_sm : plane_bytes;
  w->alloc = alloc;
  if (getenv("QMM_LOG") != nullptr)
    fprintf(stderr, "qmm: registered %s od=%lld id=%lld od_pad=%lld raw=%zu planes=%zu device=%d\n",
            type_name(type), (long long)od, (long long)id,
            (long long)p.od_pad, nbytes, plane_bytes, device);
  *out = w;
  ok();
  return QMM_OK;
}

int qmm_weights_info(const qmm_weights* w, qmm_info* out) {
  if (w == nullptr || out == nullptr) return fail(QMM_EINVAL, "NULL handle or info pointer");
  out->type = w->p.type;
  out->od = w->p.od;
  out->id = w->p.id;
  out->od_pad = w->p.od_pad;
  out->raw_bytes = w->raw_bytes;
  out->plane_bytes = w->plane_bytes;
  out->wd_offset = w->wd_offset;
  out->sm_offset = w->sm_offset;
  ok();
  return QMM_OK;
}

int qmm_weights_export(const qmm_weights* w, void* host, size_t bytes) {
  if (w == nullptr || host == nullptr) return fail(QMM_EINVAL, "NULL handle or host pointer");
  if (bytes != w->plane_bytes)
    return fail(QMM_EINVAL, "bytes %zu != plane_bytes %zu", bytes, w->plane_bytes);
  int prev = -1;
  hipError_t e = hipGetDevice(&prev);
  if (e != hipSuccess) return fail_hip(e, "hipGetDevice");
  if (prev != w->device && (e = hipSetDevice(w->device)) != hipSuccess) return fail_hip(e, "hipSetDevice");
  e = hipMemcpy(host, w->alloc, bytes, hipMemcpyDeviceToHost);
  if (prev != w->device) (void)hipSetDevice(prev);
  if (e != hipSuccess) return fail_hip(e, "hipMemcpy(planes)");
  ok();
  return QMM_OK;
}

void qmm_release_weights(qmm_weights* w) {
  if (w == nullptr) return;
  int prev = -1;
  if (hipGetDevice(&prev) == hipSuccess && prev != w->device) (void)hipSetDevice(w->device);
  (void)hipFree(w->alloc);
  if (prev >= 0 && prev != w->device) (void)hipSetDevice(prev);
  g_held -= w->plane_bytes;
  delete w;
}

int qmm_quantize_activations(const float* x, int64_t n_tok, int64_t id, void* qact,
                             size_t qact_bytes, void* stream) {
  if (int rc = check_tokens(n_tok)) return rc;
  if (int rc = check_id(id)) return rc;
  if (n_tok == 0) {  // empty batch: no bytes to write, pointers are not used
    if (qact_bytes != 0) return fail(QMM_EINVAL, "qact_bytes %zu != 0 for n_tok = 0", qact_bytes);
    ok();
    return QMM_OK;
  }
  if (x == nullptr || qact == nullptr) return fail(QMM_EINVAL, "x or qact is NULL");
  if (!aligned(x, 16) || !aligned(qact, 16)) return fail(QMM_EINVAL, "x and qact must be 16-byte aligned");
  const size_t need = qmm_qact_bytes(n_tok, id);
  if (qact_bytes != need)
    return fail(QMM_EINVAL, "qact_bytes %zu != qmm_qact_bytes(%lld, %lld) = %zu", qact_bytes,
                (long long)n_tok, (long long)id, need);
  hipError_t e = qmm::launch_quantize(x, n_tok, token_pad(n_tok), id, (uint8_t*)qact,
                                      (hipStream_t)stream);
  if (e != hipSuccess) return fail_hip(e, "quantize launch");
  ok();
  return QMM_OK;
}

}  // extern "C"

namespace {

// ---- qmm_norm_quantize, qmm_dequantize_activations ----

int check_elem(const char* what, int type) {
  if (type != QMM_F32 && type != QMM_F16 && type != QMM_BF16)
    return fail(QMM_EINVAL, "%s must be QMM_F32 (%d), QMM_F16 (%d) or QMM_BF16 (%d), got %d", what, QMM_F32, QMM_F16,
                QMM_BF16, type);
  return QMM_OK;
}

size_t elem_bytes(int type) { return type == QMM_F32 ? 4 : 2; }

// Rows of `cols` elements, `stride` elements apart, accessed four elements at a time.
int check_rows(const char* what, const void* p, int64_t stride, int64_t cols) {
  if (!aligned(p, 16)) return fail(QMM_EINVAL, "%s must be 16-byte aligned", what);
  if (stride < cols || stride % 4 != 0 || stride > QMM_MAX_STRIDE)
    return fail(QMM_EINVAL, "%s_stride must be a multiple of 4 in [%lld, %lld], got %lld", what, (long long)cols,
                (long long)QMM_MAX_STRIDE, (long long)stride);
  return QMM_OK;
}

// A range of device bytes with the layout of its rows.
struct Range {
  const char* what;
  const void* p;
  int64_t stride;  // bytes from row to row
  size_t bytes;    // from the first byte to the last
  size_t row = 0;  // bytes of a row (rows only)
};

Range rows_range(const char* what, const void* p, int64_t stride, int64_t rows, int64_t cols, size_t elem) {
  if (p == nullptr) return {what, p, 0, 0};
  return {what, p, stride * (int64_t)elem, (size_t)((rows - 1) * stride + cols) * elem, (size_t)cols * elem};
}

bool overlap(const Range& a, const Range& b) {
  const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
  if (a.p == nullptr || b.p == nullptr || x >= y + b.bytes || y >= x + a.bytes) return false;
  if (a.row > 0 && b.row > 0 && a.stride == b.stride && a.stride > 0) {
    // columns of one wider tensor: where b's row starts inside a's stride
    const size_t stride = (size_t)a.stride, at = y >= x ? (y - x) % stride : (stride - (x - y) % stride) % stride;
    return at < a.row || at + b.row > stride;
  }
  return true;
}

// Whether an output that overlaps an input is that input in place.
bool same_rows(const Range& a, const Range& b) { return a.p == b.p && a.stride == b.stride && a.bytes == b.bytes; }

int refuse_overlap(const Range& a, const Range& b) {
  return fail(QMM_EINVAL, "%s overlaps %s", a.what, b.what);
}

int check_vector(const char* what, const float* p) {
  return aligned(p, 16) ? QMM_OK : fail(QMM_EINVAL, "%s must be 16-byte aligned", what);
}

}  // namespace

extern "C" {

int qmm_dequantize_activations(const void* qact, size_t qact_bytes, int64_t n_tok, int64_t id, int type, void* out,
                               int64_t out_stride, void* stream) {
  if (int rc = check_tokens(n_tok)) return rc;
  if (int rc = check_id(id)) return rc;
  if (int rc = check_elem("type", type)) return rc;
  const size_t need = qmm_qact_bytes(n_tok, id);
  if (qact_bytes != need)
    return fail(QMM_EINVAL, "qact_bytes %zu != qmm_qact_bytes(%lld, %lld) = %zu", qact_bytes, (long long)n_tok,
                (long long)id, need);
  if (n_tok == 0) {
    ok();
    return QMM_OK;
  }
  if (qact == nullptr || out == nullptr) return fail(QMM_EINVAL, "qact or out is NULL");
  if (!aligned(qact, 16)) return fail(QMM_EINVAL, "qact must be 16-byte aligned");
  if (int rc = check_rows("out", out, out_stride, id)) return rc;
  const Range r = rows_range("out", out, out_stride, n_tok, id, elem_bytes(type)), q{"qact", qact, 0, qact_bytes};
  if (overlap(r, q)) return refuse_overlap(r, q);
  hipError_t e = qmm::launch_dequantize((const uint8_t*)qact, n_tok, token_pad(n_tok), id, type, out, out_stride,
                                        (hipStream_t)stream);
  if (e != hipSuccess) return fail_hip(e, "dequantize launch");
  ok();
  return QMM_OK;
}

int qmm_norm_quantize(const qmm_norm* args, int64_t n_tok, int64_t id, void* stream) {
  if (args == nullptr) return fail(QMM_EINVAL, "args is NULL");
  const qmm_norm& a = *args;
  if (int rc = check_tokens(n_tok)) return rc;
  if (int rc = check_id(id)) return rc;
  if (int rc = check_elem("type", a.type)) return rc;
  if (a.kind != QMM_NORM_RMS && a.kind != QMM_NORM_LAYER)
    return fail(QMM_EINVAL, "kind must be QMM_NORM_RMS (%d) or QMM_NORM_LAYER (%d), got %d", QMM_NORM_RMS,
                QMM_NORM_LAYER, a.kind);
  if (!(a.eps > 0.0f) || !std::isfinite(a.eps)) return fail(QMM_EINVAL, "eps must be positive and finite");
  if (!std::isfinite(a.residual_scale) || !std::isfinite(a.block_scale))
    return fail(QMM_EINVAL, "residual_scale and block_scale must be finite");
  const size_t need = a.qact != nullptr ? qmm_qact_bytes(n_tok, id) : 0;
  if (a.qact_bytes != need)
    return fail(QMM_EINVAL, "qact_bytes %zu != %zu for n_tok=%lld id=%lld %s", a.qact_bytes, need, (long long)n_tok,
                (long long)id, a.qact != nullptr ? "" : "without qact");
  if (n_tok == 0) {  // empty batch: no rows, pointers are not used
    ok();
    return QMM_OK;
  }
  if (a.h == nullptr || a.weight == nullptr) return fail(QMM_EINVAL, "h or weight is NULL");
  if (a.h_out == nullptr && a.normed == nullptr && a.qact == nullptr)
    return fail(QMM_EINVAL, "no output: h_out, normed and qact are NULL");
  if (a.y == nullptr && (a.post_weight != nullptr || a.gate != nullptr))
    return fail(QMM_EINVAL, "post_weight and gate need y");
  if (a.post_weight == nullptr && a.post_bias != nullptr) return fail(QMM_EINVAL, "post_bias needs post_weight");
  if (int rc = check_rows("h", a.h, a.h_stride, id)) return rc;
  if (a.y != nullptr)
    if (int rc = check_rows("y", a.y, a.y_stride, id)) return rc;
  if (a.gate != nullptr)  // a single row of any stride stands for every token when its stride is 0
    if (int rc = check_rows("gate", a.gate, a.gate_stride == 0 ? id : a.gate_stride, id)) return rc;
  if (a.h_out != nullptr)
    if (int rc = check_rows("h_out", a.h_out, a.h_out_stride, id)) return rc;
  if (a.normed != nullptr)
    if (int rc = check_rows("normed", a.normed, a.normed_stride, id)) return rc;
  if (!aligned(a.qact, 16)) return fail(QMM_EINVAL, "qact must be 16-byte aligned");
  if (int rc = check_vector("weight", a.weight)) return rc;
  if (int rc = check_vector("bias", a.bias)) return rc;
  if (int rc = check_vector("post_weight", a.post_weight)) return rc;
  if (int rc = check_vector("post_bias", a.post_bias)) return rc;
  const size_t eb = elem_bytes(a.type);
  const Range h = rows_range("h", a.h, a.h_stride, n_tok, id, eb), y = rows_range("y", a.y, a.y_stride, n_tok, id, eb);
  const Range outs[] = {rows_range("h_out", a.h_out, a.h_out_stride, n_tok, id, eb),
                        rows_range("normed", a.normed, a.normed_stride, n_tok, id, eb),
                        {"qact", a.qact, 0, need}};
  const Range fixed[] = {rows_range("gate", a.gate, a.gate_stride, a.gate_stride == 0 ? 1 : n_tok, id, eb),
                         {"weight", a.weight, 0, (size_t)id * 4},
                         {"bias", a.bias, 0, (size_t)id * 4},
                         {"post_weight", a.post_weight, 0, (size_t)id * 4},
                         {"post_bias", a.post_bias, 0, (size_t)id * 4}};
  for (int i = 0; i < 3; ++i) {
    const bool rows = i < 2;  // h_out and normed may be computed in place
    const bool in_h = rows && (i == 0 || a.h_out == nullptr) && same_rows(outs[i], h);
    const bool in_y = rows && same_rows(outs[i], y);
    if (overlap(outs[i], h) && !in_h) return refuse_overlap(outs[i], h);
    if (overlap(outs[i], y) && !in_y) return refuse_overlap(outs[i], y);
    for (const Range& f : fixed)
      if (overlap(outs[i], f)) return refuse_overlap(outs[i], f);
    for (int k = 0; k < i; ++k)
      if (overlap(outs[i], outs[k])) return refuse_overlap(outs[i], outs[k]);
  }
  hipError_t e = qmm::launch_norm(a, n_tok, a.qact != nullptr ? token_pad(n_tok) : 0, id, (hipStream_t)stream);
  if (e != hipSuccess) return fail_hip(e, "norm launch");
  ok();
  return QMM_OK;
}

}  // extern "C"

namespace {

// The parts of an epilogue that do not depend on the product's sizes.
int check_epilogue(const qmm_epilogue* ep, int out_type) {
  if (out_type != QMM_Q8)
    if (int rc = check_elem("out_type", out_type)) return rc;
  if (ep == nullptr) return QMM_OK;
  if (ep->act < QMM_ACT_NONE || ep->act > QMM_ACT_GELU_TANH)
    return fail(QMM_EINVAL, "act must be one of QMM_ACT_* (0 to %d), got %d", QMM_ACT_GELU_TANH, ep->act);
  if (int rc = check_elem("type of mul and residual", ep->type)) return rc;
  if (!std::isfinite(ep->scale) || !std::isfinite(ep->residual_scale))
    return fail(QMM_EINVAL, "scale and residual_scale must be finite");
  if (!aligned(ep->bias, 4)) return fail(QMM_EINVAL, "bias must be 4-byte aligned");
  const size_t eb = elem_bytes(ep->type);
  if (!aligned(ep->mul, eb) || !aligned(ep->residual, eb))
    return fail(QMM_EINVAL, "mul and residual must be aligned to their element");
  return QMM_OK;
}

int check_stride(const char* what, int64_t stride, int64_t cols) {
  if (stride < cols || stride > QMM_MAX_STRIDE)
    return fail(QMM_EINVAL, "%s_stride must be in [%lld, %lld], got %lld", what, (long long)cols,
                (long long)QMM_MAX_STRIDE, (long long)stride);
  return QMM_OK;
}

// Checks the epilogue and output of a product of n_tok > 0 tokens by od rows and
// writes the kernels' form of them.  `in`: the product's other inputs; *written:
// the range of out.
int resolve_epilogue(const qmm_epilogue* ep, int64_t n_tok, int64_t od, int out_type, void* out, int64_t out_stride,
                     const Range& in, qmm::Epilogue* r, Range* written) {
  static const qmm_epilogue kNone = {nullptr, QMM_ACT_NONE, QMM_F32, 1.0f, 0.0f, nullptr, 0, nullptr, 0};
  if (ep == nullptr) ep = &kNone;
  if (out == nullptr) return fail(QMM_EINVAL, "out is NULL");
  if (out_type == QMM_Q8) {
    const size_t need = qmm_qact_bytes(n_tok, od);
    if (need == 0)
      return fail(QMM_EINVAL, "a q8 output needs od %% 256 == 0 and od <= %d, got od=%lld", QMM_MAX_ID, (long long)od);
    if (out_stride < 0 || (size_t)out_stride != need)
      return fail(QMM_EINVAL, "out_stride %lld != qmm_qact_bytes(%lld, %lld) = %zu", (long long)out_stride,
                  (long long)n_tok, (long long)od, need);
    if (!aligned(out, 16)) return fail(QMM_EINVAL, "a q8 output must be 16-byte aligned");
    *written = {"out", out, 0, need};
  } else {
    if (int rc = check_stride("out", out_stride, od)) return rc;
    if (!aligned(out, elem_bytes(out_type))) return fail(QMM_EINVAL, "out must be aligned to its element");
    *written = rows_range("out", out, out_stride, n_tok, od, elem_bytes(out_type));
  }
  const size_t eb = elem_bytes(ep->type);
  if (ep->mul != nullptr)
    if (int rc = check_stride("mul", ep->mul_stride, od)) return rc;
  if (ep->residual != nullptr)
    if (int rc = check_stride("residual", ep->residual_stride, od)) return rc;
  if (overlap(*written, in)) return refuse_overlap(*written, in);
  const Range bias{"bias", ep->bias, 0, (size_t)od * 4};
  if (overlap(*written, bias)) return refuse_overlap(*written, bias);
  for (const Range& side : {rows_range("mul", ep->mul, ep->mul_stride, n_tok, od, eb),
                            rows_range("residual", ep->residual, ep->residual_stride, n_tok, od, eb)})
    if (overlap(*written, side) && !(out_type == ep->type && same_rows(*written, side)))
      return refuse_overlap(*written, side);
  r->bias = ep->bias;
  r->mul = ep->mul;
  r->residual = ep->residual;
  r->out = out;
  r->mul_stride = (int)ep->mul_stride;
  r->residual_stride = (int)ep->residual_stride;
  r->out_stride = out_type == QMM_Q8 ? 0 : (int)out_stride;
  r->t_pad = token_pad(n_tok);
  r->scale = ep->scale;
  r->residual_scale = ep->residual_scale;
  r->act = ep->act;
  r->side_type = ep->type;
  r->out_type = out_type;
  return QMM_OK;
}

int check_mmq_handle(const qmm_weights* w) {
  if (w == nullptr) return fail(QMM_EINVAL, "NULL weights handle");
  if (qmm::is_rows(w->p.type))
    return fail(QMM_EINVAL, "the handle holds %s weights, the form of qmm_mmv", type_name(w->p.type));
  return QMM_OK;
}

// The current device, which has to be the handle's, and its compute units.
int current_device(const qmm_weights* w, int* device, int* num_cus) {
  hipError_t e = hipGetDevice(device);
  if (e != hipSuccess) return fail_hip(e, "hipGetDevice");
  if (*device != w->device)
    return fail(QMM_EINVAL, "handle belongs to device %d but device %d is current", w->device, *device);
  e = hipDeviceGetAttribute(num_cus, hipDeviceAttributeMultiprocessorCount, *device);
  if (e != hipSuccess) return fail_hip(e, "hipDeviceGetAttribute(multiprocessor count)");
  return QMM_OK;
}

// Validation and launch plan shared by qmm_mmq and qmm_mmq_noalloc.  Returns
// QMM_OK with *launch false for an empty batch (nothing to launch).
int prepare_mmq(const qmm_weights* w, const void* qact, size_t qact_bytes, int64_t n_tok, const float* out,
                qmm::MmqPlan* plan, int* device, int* num_cus, bool* launch) {
  *launch = false;
  if (int rc = check_mmq_handle(w)) return rc;
  if (int rc = check_tokens(n_tok)) return rc;
  if (n_tok == 0) {  // empty batch: an empty output, nothing launched
    if (qact_bytes != 0) return fail(QMM_ESHAPE, "qact_bytes %zu != 0 for n_tok = 0", qact_bytes);
    return QMM_OK;
  }
  if (qact == nullptr || out == nullptr) return fail(QMM_EINVAL, "qact or out is NULL");
  if (!aligned(qact, 16)) return fail(QMM_EINVAL, "qact must be 16-byte aligned");
  if (!aligned(out, 4)) return fail(QMM_EINVAL, "out must be 4-byte aligned");
  const size_t need = qmm_qact_bytes(n_tok, w->p.id);
  if (qact_bytes != need)
    return fail(QMM_ESHAPE, "qact_bytes %zu does not match n_tok=%lld and the handle's id=%lld (%zu)",
                qact_bytes, (long long)n_tok, (long long)w->p.id, need);
  if (int rc = current_device(w, device, num_cus)) return rc;
  *plan = qmm::plan_mmq(w->p, n_tok, *num_cus);
  if (int rc = check_launch(*plan, n_tok, w->p.od, *num_cus)) return rc;
  *launch = true;
  return QMM_OK;
}

// The tail-partials scratch of (device, stream), allocated by its first call.
int stream_scratch(int device, int num_cus, hipStream_t s, void** scratch) {
  const size_t max_bytes = qmm::mmq_scratch_max_bytes(num_cus);
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  for (const Scratch& sc : g_scratch)
    if (sc.device == device && sc.stream == s && sc.thread == this_thread(s)) *scratch = sc.ptr;
  if (*scratch != nullptr) return QMM_OK;
  hipError_t e = hipMalloc(scratch, max_bytes);
  if (e != hipSuccess) {
    (void)hipGetLastError();  // leave no sticky error for the caller's next HIP call
    return e == hipErrorOutOfMemory ? fail(QMM_ENOMEM, "hipMalloc(%zu) for the tail partials failed", max_bytes)
                                    : fail_hip(e, "hipMalloc(tail partials)");
  }
  g_scratch.push_back({device, s, this_thread(s), *scratch, max_bytes});
  return QMM_OK;
}

}  // namespace

extern "C" {

int qmm_mmq(const qmm_weights* w, const void* qact, size_t qact_bytes, int64_t n_tok, float* out,
            void* stream) {
  qmm::MmqPlan plan{};
  int device = -1, num_cus = 0;
  bool launch = false;
  if (int rc = prepare_mmq(w, qact, qact_bytes, n_tok, out, &plan, &device, &num_cus, &launch)) return rc;
  if (!launch) {
    ok();
    return QMM_OK;
  }
  const hipStream_t s = (hipStream_t)stream;
  void* scratch = nullptr;
  if (plan.scratch_bytes > 0)
    if (int rc = stream_scratch(device, num_cus, s, &scratch)) return rc;
  const auto turn = launch_turn(s, plan.scratch_bytes);
  hipError_t e = qmm::launch_mmq(w->p, plan, (const uint8_t*)qact, n_tok, token_pad(n_tok), out,
                                 (float*)scratch, s);
  if (e != hipSuccess) return fail_hip(e, "mmq launch");
  ok();
  return QMM_OK;
}

int qmm_stream_release(void* stream, size_t* freed_bytes) {
  const hipStream_t s = (hipStream_t)stream;
  if (freed_bytes != nullptr) *freed_bytes = 0;
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  bool synced = false;
  int cur = -1;
  for (size_t i = 0; i < g_scratch.size();) {
    if (g_scratch[i].stream != s || g_scratch[i].thread != this_thread(s)) {
      ++i;
      continue;
    }
    // ---- first HIP call below this line (none when the stream holds nothing) ----
    hipError_t e;
    if (!synced) {  // the stream's MMQs may still read the partials
      if ((e = hipStreamSynchronize(s)) != hipSuccess) return fail_hip(e, "hipStreamSynchronize");
      if ((e = hipGetDevice(&cur)) != hipSuccess) return fail_hip(e, "hipGetDevice");
      synced = true;
    }
    if ((e = hipSetDevice(g_scratch[i].device)) != hipSuccess) return fail_hip(e, "hipSetDevice");
    e = hipFree(g_scratch[i].ptr);
    const hipError_t e2 = hipSetDevice(cur);
    if (e != hipSuccess) return fail_hip(e, "hipFree(tail partials)");
    if (e2 != hipSuccess) return fail_hip(e2, "hipSetDevice(restore)");
    if (freed_bytes != nullptr) *freed_bytes += g_scratch[i].bytes;
    g_scratch.erase(g_scratch.begin() + (ptrdiff_t)i);
  }
  ok();
  return QMM_OK;
}

int qmm_mmq_noalloc(const qmm_weights* w, const void* qact, size_t qact_bytes, int64_t n_tok, float* out,
                    void* stream) {
  qmm::MmqPlan plan{};
  int device = -1, num_cus = 0;
  bool launch = false;
  if (int rc = prepare_mmq(w, qact, qact_bytes, n_tok, out, &plan, &device, &num_cus, &launch)) return rc;
  if (!launch) {
    ok();
    return QMM_OK;
  }
  if (plan.scratch_bytes > qmm::kStaticScratchBytes)
    return fail(QMM_EINVAL, "this launch needs %zu bytes of tail scratch; the static scratch holds %zu",
                plan.scratch_bytes, qmm::kStaticScratchBytes);
  float* part = nullptr;
  if (plan.scratch_bytes > 0) {
    hipError_t e = qmm::static_scratch(device, &part);
    if (e != hipSuccess) return fail_hip(e, "hipGetSymbolAddress(static tail scratch)");
  }
  const auto turn = launch_turn((hipStream_t)stream, plan.scratch_bytes);
  hipError_t e = qmm::launch_mmq(w->p, plan, (const uint8_t*)qact, n_tok, token_pad(n_tok), out, part,
                                 (hipStream_t)stream);
  if (e != hipSuccess) return fail_hip(e, "mmq launch");
  ok();
  return QMM_OK;
}

int qmm_mmq_epilogue(const qmm_weights* w, const void* qact, size_t qact_bytes, int64_t n_tok, const qmm_epilogue* ep,
                     int out_type, void* out, int64_t out_stride, void* work, size_t work_bytes, void* stream) {
  if (int rc = check_epilogue(ep, out_type)) return rc;
  if ((work == nullptr) != (work_bytes == 0) || !aligned(work, 16))
    return fail(QMM_EINVAL, "work must be 16-byte aligned and come with its size (NULL with 0)");
  if (int rc = check_mmq_handle(w)) return rc;
  if (int rc = check_tokens(n_tok)) return rc;
  const size_t need = qmm_qact_bytes(n_tok, w->p.id);
  if (qact_bytes != need)
    return fail(QMM_ESHAPE, "qact_bytes %zu does not match n_tok=%lld and the handle's id=%lld (%zu)", qact_bytes,
                (long long)n_tok, (long long)w->p.id, need);
  if (n_tok == 0) {  // empty batch: an empty output, nothing launched
    ok();
    return QMM_OK;
  }
  if (qact == nullptr) return fail(QMM_EINVAL, "qact is NULL");
  if (!aligned(qact, 16)) return fail(QMM_EINVAL, "qact must be 16-byte aligned");
  const Range in{"qact", qact, 0, need}, own{"work", work, 0, work_bytes};
  qmm::Epilogue r{};
  Range written{};
  if (int rc = resolve_epilogue(ep, n_tok, w->p.od, out_type, out, out_stride, in, &r, &written)) return rc;
  if (overlap(own, in)) return refuse_overlap(own, in);
  if (overlap(own, written)) return refuse_overlap(own, written);
  if (ep != nullptr)
    for (const Range& side : {Range{"bias", ep->bias, 0, (size_t)w->p.od * 4},
                              rows_range("mul", ep->mul, ep->mul_stride, n_tok, w->p.od, elem_bytes(ep->type)),
                              rows_range("residual", ep->residual, ep->residual_stride, n_tok, w->p.od,
                                         elem_bytes(ep->type))})
      if (overlap(own, side)) return refuse_overlap(own, side);
  int device = -1, num_cus = 0;
  if (int rc = current_device(w, &device, &num_cus)) return rc;
  const hipStream_t s = (hipStream_t)stream;
  if (qmm::mmq_few_blocks(w->p, n_tok, num_cus) > 0) {  // no scratch
    hipError_t e = qmm::launch_mmq_few(w->p, (const uint8_t*)qact, n_tok, token_pad(n_tok), r, num_cus, s);
    if (e != hipSuccess) return fail_hip(e, "mmq launch");
    ok();
    return QMM_OK;
  }
  const qmm::MmqPlan plan = qmm::plan_mmq(w->p, n_tok, num_cus);
  if (int rc = check_launch(plan, n_tok, w->p.od, num_cus)) return rc;
  if (work != nullptr && work_bytes < plan.scratch_bytes)
    return fail(QMM_EINVAL, "work_bytes %zu, but this launch needs %zu bytes of tail scratch", work_bytes,
                plan.scratch_bytes);
  void* scratch = work;
  if (scratch == nullptr && plan.scratch_bytes > 0) {
    // a captured launch outlives the stream's turn: two graphs would share its scratch
    hipStreamCaptureStatus capture = hipStreamCaptureStatusNone;
    if (hipStreamIsCapturing(s, &capture) != hipSuccess) (void)hipGetLastError();
    if (capture != hipStreamCaptureStatusNone)
      return fail(QMM_EINVAL, "a captured call of this shape needs %zu bytes of work memory of its own",
                  plan.scratch_bytes);
    if (int rc = stream_scratch(device, num_cus, s, &scratch)) return rc;
  }
  const auto turn = launch_turn(s, plan.scratch_bytes);
  hipError_t e = qmm::launch_mmq_epilogue(w->p, plan, (const uint8_t*)qact, n_tok, token_pad(n_tok), r,
                                          (float*)scratch, s);
  if (e != hipSuccess) return fail_hip(e, "mmq launch");
  ok();
  return QMM_OK;
}

int qmm_mmv(const qmm_weights* w, const void* x, int x_type, int64_t x_stride, int64_t n_tok, const qmm_epilogue* ep,
            int out_type, void* out, int64_t out_stride, void* stream) {
  if (int rc = check_epilogue(ep, out_type)) return rc;
  if (x_type != QMM_Q8)
    if (int rc = check_elem("x_type", x_type)) return rc;
  if (n_tok < 0 || n_tok > QMM_MV_MAX_TOKENS)
    return fail(QMM_EINVAL, "n_tok must be in [0, %d], got %lld", QMM_MV_MAX_TOKENS, (long long)n_tok);
  if (n_tok > 0 && x == nullptr) return fail(QMM_EINVAL, "x is NULL");
  const bool q8 = x_type == QMM_Q8;
  const size_t xb = q8 ? 1 : elem_bytes(x_type);
  if (q8 ? !aligned(x, 16) : !aligned(x, 4 * xb) || x_stride % 4 != 0)
    return fail(QMM_EINVAL, "x and its rows must be aligned to four elements, a q8 x to 16 bytes");
  if (w == nullptr) return fail(QMM_EINVAL, "NULL weights handle");
  if (!qmm::is_rows(w->p.type))
    return fail(QMM_EINVAL, "the handle holds %s weights, qmm_mmv reads the rows forms", type_name(w->p.type));
  Range in{};
  if (q8) {
    const size_t need = qmm_qact_bytes(n_tok, w->p.id);
    if (x_stride < 0 || (size_t)x_stride != need)
      return fail(QMM_ESHAPE, "x_stride %lld does not match a qact of n_tok=%lld and the handle's id=%lld (%zu bytes)",
                  (long long)x_stride, (long long)n_tok, (long long)w->p.id, need);
    in = {"x", x, 0, need};
  }
  if (n_tok == 0) {  // empty batch: an empty output, nothing launched
    ok();
    return QMM_OK;
  }
  if (!q8) {
    if (int rc = check_stride("x", x_stride, w->p.id)) return rc;
    in = rows_range("x", x, x_stride, n_tok, w->p.id, xb);
  }
  qmm::Epilogue r{};
  Range written{};
  if (int rc = resolve_epilogue(ep, n_tok, w->p.od, out_type, out, out_stride, in, &r, &written)) return rc;
  int device = -1, num_cus = 0;
  if (int rc = current_device(w, &device, &num_cus)) return rc;
  hipError_t e = qmm::launch_mmv(w->p, x, x_type, q8 ? token_pad(n_tok) * w->p.id : x_stride, (int)n_tok, r, num_cus,
                                 (hipStream_t)stream);
  if (e != hipSuccess) return fail_hip(e, "mmv launch");
  ok();
  return QMM_OK;
}

int qmm_mmq_plan(int type, int64_t od, int64_t id, int64_t n_tok, int num_cus, qmm_plan* out) {
  if (out == nullptr) return fail(QMM_EINVAL, "out is NULL");
  std::memset(out, 0, sizeof *out);
  if (int rc = check_type(type)) return rc;
  if (int rc = check_od(od)) return rc;
  if (int rc = check_id(id)) return rc;
  if (int rc = check_tokens(n_tok)) return rc;
  if (num_cus < 1 || num_cus > QMM_MAX_CUS)
    return fail(QMM_EINVAL, "num_cus must be in [1, %d], got %d", QMM_MAX_CUS, num_cus);
  out->nsb = (int32_t)(id / 256);
  if (n_tok == 0) {  // an empty batch launches nothing
    ok();
    return QMM_OK;
  }
  const qmm::MmqPlan plan = qmm::plan_mmq(plane_shape(type, od, id), n_tok, num_cus);
  if (int rc = check_launch(plan, n_tok, od, num_cus)) return rc;
  out->work_groups = plan.work_groups;
  out->scratch_bytes = plan.scratch_bytes;
  out->threads = plan.threads;
  out->many = plan.many ? 1 : 0;
  out->tile_rows = plan.tile_rows;
  out->tile_tokens = plan.tile_tokens;
  out->k_groups = plan.k_groups;
  out->per_cu = plan.per_cu;
  out->row_tiles = plan.row_tiles;
  out->tok_tiles = plan.tok_tiles;
  out->dp_row_tiles = plan.dp_row_tiles;
  out->n_tail = plan.n_tail;
  out->split = plan.split;
  ok();
  return QMM_OK;
}

int qmm_mmq_plan_work(const qmm_plan* plan, int64_t wg, int32_t* row_tile, int32_t* tok_tile, int32_t* sb_begin,
                      int32_t* sb_end) {
  if (plan == nullptr || row_tile == nullptr || tok_tile == nullptr || sb_begin == nullptr || sb_end == nullptr)
    return fail(QMM_EINVAL, "plan or an output pointer is NULL");
  const qmm_plan& q = *plan;
  const bool consistent = q.nsb >= 1 && q.tok_tiles >= 1 && q.dp_row_tiles >= 0 && q.n_tail >= 0 &&
                          q.split >= 1 && (q.n_tail > 0) == (q.split > 1) && q.split <= q.nsb &&
                          q.n_tail % q.tok_tiles == 0 && q.dp_row_tiles + q.n_tail / q.tok_tiles == q.row_tiles &&
                          q.work_groups == (int64_t)q.dp_row_tiles * q.tok_tiles + (int64_t)q.n_tail * q.split &&
                          q.work_groups < ((int64_t)1 << 31);
  if (!consistent) return fail(QMM_EINVAL, "plan is not one qmm_mmq_plan wrote");
  if (wg < 0 || wg >= q.work_groups)
    return fail(QMM_EINVAL, "work-group %lld outside the launch's %lld", (long long)wg, (long long)q.work_groups);
  qmm::MmqPlan p{};
  p.row_tiles = q.row_tiles;
  p.tok_tiles = q.tok_tiles;
  p.dp_row_tiles = q.dp_row_tiles;
  p.n_tail = q.n_tail;
  p.split = q.split;
  int rt = 0, tt = 0, s0 = 0, s1 = 0;
  qmm::plan_work(p, q.nsb, wg, &rt, &tt, &s0, &s1);
  *row_tile = rt;
  *tok_tile = tt;
  *sb_begin = s0;
  *sb_end = s1;
  ok();
  return QMM_OK;
}

}  // extern "C"

namespace {

// ---- qmm_rope_cache, qmm_cache_read, qmm_attention ----

bool head_dim_ok(int dim) { return dim == 64 || dim == 96 || dim == 128 || dim == 192 || dim == 256; }

int check_cache_shape(const qmm_cache& c) {
  if (c.type != QMM_F16 && c.type != QMM_BF16 && c.type != QMM_Q8)
    return fail(QMM_EINVAL, "a cache's type must be QMM_F16 (%d), QMM_BF16 (%d) or QMM_Q8 (%d), got %d", QMM_F16, QMM_BF16,
                QMM_Q8, c.type);
  if (c.heads < 1 || c.heads > QMM_MAX_HEADS)
    return fail(QMM_EINVAL, "a cache's heads must be in [1, %d], got %d", QMM_MAX_HEADS, c.heads);
  if (!head_dim_ok(c.head_dim)) return fail(QMM_EINVAL, "head_dim must be 64, 96, 128, 192 or 256, got %d", c.head_dim);
  return QMM_OK;
}

bool page_ok(int page) { return page >= 32 && page <= QMM_MAX_PAGE && (page & (page - 1)) == 0; }

// The cache and the batch, as the kernels take them.  Pools that a call does not use may be
// NULL (use: 1 k, 2 v).
int check_cache(const qmm_cache* cache, const qmm_batch* batch, int64_t n_tok, int use, qmm::Pools* p, qmm::Batch* b) {
  if (cache == nullptr || batch == nullptr) return fail(QMM_EINVAL, "cache or batch is NULL");
  const qmm_cache& c = *cache;
  if (int rc = check_cache_shape(c)) return rc;
  if (!page_ok(c.page)) return fail(QMM_EINVAL, "page must be a power of two in [32, %d], got %d", QMM_MAX_PAGE, c.page);
  if (c.n_pages < 1 || c.n_pages > INT32_MAX)
    return fail(QMM_EINVAL, "n_pages must be in [1, 2^31 - 1], got %lld", (long long)c.n_pages);
  if (((use & 1) != 0 && c.k == nullptr) || ((use & 2) != 0 && c.v == nullptr))
    return fail(QMM_EINVAL, "a pool of the cache is NULL");
  if (!aligned(c.k, 16) || !aligned(c.v, 16)) return fail(QMM_EINVAL, "the cache's pools must be 16-byte aligned");
  if (c.n_pages > (INT64_MAX >> 1) / (int64_t)qmm_cache_page_bytes(c.type, c.heads, c.head_dim, c.page))
    return fail(QMM_EINVAL, "the pools' bytes pass 2^62");
  const qmm_batch& q = *batch;
  if (q.n_seq < 1 || q.n_seq > QMM_MAX_SEQS)
    return fail(QMM_EINVAL, "n_seq must be in [1, %d], got %d", QMM_MAX_SEQS, q.n_seq);
  if (q.columns < 1 || (int64_t)q.columns * c.page > QMM_MAX_SLOTS)
    return fail(QMM_EINVAL, "columns must be at least 1 and columns * page at most %d, got %d * %d", QMM_MAX_SLOTS, q.columns, c.page);
  if (q.table_stride < q.columns || q.table_stride > INT32_MAX)
    return fail(QMM_EINVAL, "table_stride must be in [%d, 2^31), got %lld", q.columns, (long long)q.table_stride);
  if (q.max_new < 0 || q.max_new > QMM_MAX_TOKENS || q.max_length < 0 || q.max_length > QMM_MAX_SLOTS)
    return fail(QMM_EINVAL, "max_new must be in [0, %d] and max_length in [0, %d], got %lld and %lld", QMM_MAX_TOKENS,
                QMM_MAX_SLOTS, (long long)q.max_new, (long long)q.max_length);
  if (q.starts == nullptr || q.lengths == nullptr || q.table == nullptr)
    return fail(QMM_EINVAL, "starts, lengths or table is NULL");
  if (!aligned(q.starts, 4) || !aligned(q.lengths, 4) || !aligned(q.table, 4))
    return fail(QMM_EINVAL, "starts, lengths and table must be 4-byte aligned");
  int shift = 0;
  while ((1 << shift) < c.page) ++shift;
  *p = {(uint8_t*)c.k, (uint8_t*)c.v, c.heads, c.head_dim, shift, c.type, (int32_t)c.n_pages};
  *b = {q.starts, q.lengths, q.table, q.table_stride, q.n_seq, q.columns, (int32_t)n_tok};
  return QMM_OK;
}

// A tensor [n_tok][heads][dim] with adjacent channels; *range: its bytes.
int check_heads(const char* what, const void* p, int64_t stride, int64_t head_stride, int64_t n_tok, int64_t heads,
                int64_t dim, size_t elem, qmm::Rows* rows, Range* range) {
  if (!aligned(p, 16)) return fail(QMM_EINVAL, "%s must be 16-byte aligned", what);
  if (n_tok == 1) stride = 0;
  if (heads == 1) head_stride = 0;
  const auto ok_stride = [&](int64_t s) { return s >= dim && s <= QMM_MAX_STRIDE && s % 8 == 0; };
  if ((n_tok > 1 && !ok_stride(stride)) || (heads > 1 && !ok_stride(head_stride)))
    return fail(QMM_EINVAL, "%s's strides must be multiples of 8 in [%lld, %d], got %lld and %lld", what, (long long)dim,
                QMM_MAX_STRIDE, (long long)stride, (long long)head_stride);
  *rows = {p, stride, head_stride};
  *range = {what, p, 0, (size_t)((n_tok - 1) * stride + (heads - 1) * head_stride + dim) * elem};
  return QMM_OK;
}

// Whether elements of a tensor fall on one another: one stride has to step over all that the other spans.
bool folds(const qmm::Rows& r, int64_t n_tok, int64_t heads, int64_t dim) {
  const int64_t row = (heads - 1) * r.head_stride + dim, column = (n_tok - 1) * r.stride + dim;
  return n_tok > 1 && heads > 1 && r.stride < row && r.head_stride < column;
}

// Columns of one wider row, e.g. q, k and v of a joint product: rows of equal stride that
// do not reach into each other.
void as_rows(const qmm::Rows& r, int64_t n_tok, int64_t heads, int64_t dim, size_t elem, Range* range) {
  const int64_t row = (heads - 1) * r.head_stride + dim;
  if (n_tok > 1 && row <= r.stride) {
    range->stride = r.stride * (int64_t)elem;
    range->row = (size_t)row * elem;
  }
}

Range pool_range(const char* what, const void* p, const qmm_cache& c) {
  return {what, p, 0, p == nullptr ? 0 : (size_t)c.n_pages * qmm_cache_page_bytes(c.type, c.heads, c.head_dim, c.page)};
}

// The batch's arrays, which no output may overlap.
struct BatchRanges {
  Range r[3];
  explicit BatchRanges(const qmm_batch& b)
      : r{{"starts", b.starts, 0, (size_t)(b.n_seq + 1) * 4},
          {"lengths", b.lengths, 0, (size_t)b.n_seq * 4},
          {"table", b.table, 0, ((size_t)(b.n_seq - 1) * b.table_stride + b.columns) * 4}} {}
};

}  // namespace

extern "C" {

size_t qmm_cache_page_bytes(int type, int heads, int head_dim, int page) {
  if ((type != QMM_F16 && type != QMM_BF16 && type != QMM_Q8) || heads < 1 || heads > QMM_MAX_HEADS ||
      !head_dim_ok(head_dim) || !page_ok(page))
    return 0;
  return (size_t)heads * (page / qmm::kTileSlots) * qmm::tile_bytes(type, head_dim);
}

int qmm_rope_frequencies(int64_t n_rot, double base, int scaling, double factor, double original, double fast, double slow,
                         double* frequencies, float* magnitude) {
  if (n_rot < 16 || n_rot > 256 || n_rot % 16 != 0)
    return fail(QMM_EINVAL, "n_rot must be a multiple of 16 in [16, 256], got %lld", (long long)n_rot);
  if (!(base > 1.0) || !std::isfinite(base)) return fail(QMM_EINVAL, "base must be above 1 and finite");
  if (scaling < QMM_ROPE_PLAIN || scaling > QMM_ROPE_TURNS)
    return fail(QMM_EINVAL, "scaling must be one of QMM_ROPE_* (0 to %d), got %d", QMM_ROPE_TURNS, scaling);
  if (scaling != QMM_ROPE_PLAIN && (!(factor > 0.0) || !std::isfinite(factor)))
    return fail(QMM_EINVAL, "factor must be positive and finite");
  const bool ramp = scaling == QMM_ROPE_YARN || scaling == QMM_ROPE_TURNS;
  if (ramp && (!(original > 0.0) || !std::isfinite(original) || !(slow > 0.0) || !(fast > slow) || !std::isfinite(fast)))
    return fail(QMM_EINVAL, "original must be positive, and fast above slow above 0, all finite");
  if (frequencies == nullptr) return fail(QMM_EINVAL, "frequencies is NULL");
  const double n = (double)n_rot, kTurn = 6.283185307179586477;
  if (scaling == QMM_ROPE_BASE) base *= std::pow(factor, n / (n - 2.0));
  // the pair that turns `turns` times in the original context
  const auto pair = [&](double turns) { return n * std::log(original / (turns * kTurn)) / (2.0 * std::log(base)); };
  const double low = ramp ? std::fmax(0.0, std::floor(pair(fast))) : 0.0;
  const double high = ramp ? std::fmin(n - 1.0, std::ceil(pair(slow))) : 0.0;
  for (int64_t i = 0; i < n_rot / 2; ++i) {
    double f = std::pow(base, -2.0 * (double)i / n), keep = 1.0;
    if (scaling == QMM_ROPE_LINEAR) keep = 0.0;
    if (scaling == QMM_ROPE_YARN) keep = 1.0 - std::fmin(1.0, std::fmax(0.0, ((double)i - low) / std::fmax(high - low, 0.001)));
    if (scaling == QMM_ROPE_TURNS) keep = std::fmin(1.0, std::fmax(0.0, (original * f / kTurn - slow) / (fast - slow)));
    if (keep < 1.0) f = f / factor * (1.0 - keep) + f * keep;
    frequencies[i] = f;
  }
  if (magnitude != nullptr) *magnitude = scaling == QMM_ROPE_YARN && factor > 1.0 ? (float)(0.1 * std::log(factor) + 1.0) : 1.0f;
  ok();
  return QMM_OK;
}

int qmm_rope_cache(const qmm_rope* args, const qmm_cache* cache, const qmm_batch* batch, int64_t n_tok, void* stream) {
  if (args == nullptr) return fail(QMM_EINVAL, "args is NULL");
  const qmm_rope& a = *args;
  if (int rc = check_tokens(n_tok)) return rc;
  if (int rc = check_elem("type", a.type)) return rc;
  if (a.q != nullptr)
    if (int rc = check_elem("out_type", a.out_type)) return rc;
  qmm::Pools pools{};
  qmm::Batch b{};
  if (int rc = check_cache(cache, batch, n_tok, (a.k != nullptr ? 1 : 0) | (a.v != nullptr ? 2 : 0), &pools, &b)) return rc;
  const int64_t dim = cache->head_dim;
  if (a.layout != QMM_ROPE_HALF && a.layout != QMM_ROPE_INTERLEAVED)
    return fail(QMM_EINVAL, "layout must be QMM_ROPE_HALF (%d) or QMM_ROPE_INTERLEAVED (%d), got %d", QMM_ROPE_HALF,
                QMM_ROPE_INTERLEAVED, a.layout);
  if (a.n_rot < 0 || a.n_rot > dim || a.n_rot % 16 != 0)
    return fail(QMM_EINVAL, "n_rot must be a multiple of 16 in [0, %lld], got %d", (long long)dim, a.n_rot);
  if (!std::isfinite(a.magnitude)) return fail(QMM_EINVAL, "magnitude must be finite");
  if (a.q != nullptr && (a.q_heads < 1 || a.q_heads > QMM_MAX_HEADS))
    return fail(QMM_EINVAL, "q_heads must be in [1, %d], got %d", QMM_MAX_HEADS, a.q_heads);
  if (n_tok == 0) {  // empty batch: pointers are not used
    ok();
    return QMM_OK;
  }
  if (a.q == nullptr && a.k == nullptr && a.v == nullptr) return fail(QMM_EINVAL, "nothing to do: q, k and v are NULL");
  if (a.n_rot > 0 && a.frequencies == nullptr) return fail(QMM_EINVAL, "frequencies is NULL");
  if (!aligned(a.frequencies, 8) || !aligned(a.positions, 4))
    return fail(QMM_EINVAL, "frequencies must be 8-byte aligned and positions 4-byte aligned");
  qmm::RopeArgs r{};
  r.frequencies = a.frequencies;
  r.positions = a.positions;
  r.type = a.type;
  r.out_type = a.out_type;
  r.layout = a.layout;
  r.n_rot = a.n_rot;
  r.magnitude = a.magnitude;
  const size_t eb = elem_bytes(a.type);
  Range q{}, q_out{}, k{}, v{};
  if (a.q != nullptr) {
    if (a.q_out == nullptr) return fail(QMM_EINVAL, "q_out is NULL");
    r.q_heads = a.q_heads;
    if (int rc = check_heads("q", a.q, a.q_stride, a.q_head_stride, n_tok, a.q_heads, dim, eb, &r.q, &q)) return rc;
    if (int rc = check_heads("q_out", a.q_out, a.q_out_stride, a.q_out_head_stride, n_tok, a.q_heads, dim,
                             elem_bytes(a.out_type), &r.q_out, &q_out))
      return rc;
    if (folds(r.q_out, n_tok, a.q_heads, dim)) return fail(QMM_EINVAL, "q_out's strides put rows on one another");
    as_rows(r.q, n_tok, a.q_heads, dim, eb, &q);
    as_rows(r.q_out, n_tok, a.q_heads, dim, elem_bytes(a.out_type), &q_out);
  }
  if (a.k != nullptr) {
    if (int rc = check_heads("k", a.k, a.k_stride, a.k_head_stride, n_tok, pools.heads, dim, eb, &r.k, &k)) return rc;
    as_rows(r.k, n_tok, pools.heads, dim, eb, &k);
  }
  if (a.v != nullptr) {
    if (int rc = check_heads("v", a.v, a.v_stride, a.v_head_stride, n_tok, pools.heads, dim, eb, &r.v, &v)) return rc;
    as_rows(r.v, n_tok, pools.heads, dim, eb, &v);
  }
  const bool in_place = a.q != nullptr && a.type == a.out_type && r.q.p == r.q_out.p && r.q.stride == r.q_out.stride &&
                        r.q.head_stride == r.q_out.head_stride;
  const Range outs[] = {q_out, pool_range("the cache's k", a.k != nullptr ? cache->k : nullptr, *cache),
                        pool_range("the cache's v", a.v != nullptr ? cache->v : nullptr, *cache)};
  const Range ins[] = {q, k, v, {"frequencies", a.frequencies, 0, (size_t)a.n_rot * 4},
                       {"positions", a.positions, 0, (size_t)n_tok * 4}};
  const BatchRanges fixed(*batch);
  for (int i = 0; i < 3; ++i) {
    for (int j = 0; j < 5; ++j)
      if (overlap(outs[i], ins[j]) && !(i == 0 && j == 0 && in_place)) return refuse_overlap(outs[i], ins[j]);
    for (const Range& f : fixed.r)
      if (overlap(outs[i], f)) return refuse_overlap(outs[i], f);
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i], outs[j])) return refuse_overlap(outs[i], outs[j]);
  }
  hipError_t e = qmm::launch_rope(r, pools, b, std::min(batch->max_new, n_tok), (hipStream_t)stream);
  if (e != hipSuccess) return fail_hip(e, "rope launch");
  ok();
  return QMM_OK;
}

int qmm_cache_read(const qmm_cache* cache, const qmm_batch* batch, int64_t n_tok, int type, void* k, void* v, void* stream) {
  if (int rc = check_tokens(n_tok)) return rc;
  if (int rc = check_elem("type", type)) return rc;
  qmm::Pools pools{};
  qmm::Batch b{};
  if (int rc = check_cache(cache, batch, n_tok, 3, &pools, &b)) return rc;
  if (n_tok == 0) {
    ok();
    return QMM_OK;
  }
  if (k == nullptr && v == nullptr) return fail(QMM_EINVAL, "k and v are NULL");
  if (!aligned(k, 16) || !aligned(v, 16)) return fail(QMM_EINVAL, "k and v must be 16-byte aligned");
  const size_t bytes = (size_t)n_tok * cache->heads * cache->head_dim * elem_bytes(type);
  const Range outs[] = {{"k", k, 0, k == nullptr ? 0 : bytes}, {"v", v, 0, v == nullptr ? 0 : bytes}};
  const BatchRanges fixed(*batch);
  for (const Range& o : outs) {
    for (const Range& f : {pool_range("the cache's k", cache->k, *cache), pool_range("the cache's v", cache->v, *cache),
                           fixed.r[0], fixed.r[1], fixed.r[2]})
      if (overlap(o, f)) return refuse_overlap(o, f);
  }
  if (overlap(outs[0], outs[1])) return refuse_overlap(outs[0], outs[1]);
  hipError_t e = qmm::launch_cache_read(pools, b, std::min(batch->max_new, n_tok), type, k, v, (hipStream_t)stream);
  if (e != hipSuccess) return fail_hip(e, "cache read launch");
  ok();
  return QMM_OK;
}

}  // extern "C"

namespace {

// What the plan needs of an attention's sizes.
int check_attention_sizes(const qmm_cache& c, int heads, int64_t n_tok) {
  if (heads < 1 || heads > QMM_MAX_HEADS || heads % c.heads != 0)
    return fail(QMM_EINVAL, "heads must be a multiple of the cache's %d up to %d, got %d", c.heads, QMM_MAX_HEADS, heads);
  if (n_tok * heads > INT32_MAX / 2)
    return fail(QMM_EINVAL, "n_tok * heads must be below 2^30, got %lld * %d", (long long)n_tok, heads);
  return QMM_OK;
}

}  // namespace

extern "C" {

int qmm_attention_plan(const qmm_cache* cache, const qmm_batch* batch, int heads, int64_t window, int64_t n_tok, int num_cus,
                       qmm_attn_plan* out) {
  if (out == nullptr) return fail(QMM_EINVAL, "out is NULL");
  std::memset(out, 0, sizeof *out);
  if (cache == nullptr || batch == nullptr) return fail(QMM_EINVAL, "cache or batch is NULL");
  if (int rc = check_tokens(n_tok)) return rc;
  if (int rc = check_cache_shape(*cache)) return rc;
  if (int rc = check_attention_sizes(*cache, heads, n_tok)) return rc;
  const qmm_batch& b = *batch;
  if (b.n_seq < 1 || b.n_seq > QMM_MAX_SEQS)
    return fail(QMM_EINVAL, "n_seq must be in [1, %d], got %d", QMM_MAX_SEQS, b.n_seq);
  if (b.max_new < 0 || b.max_new > QMM_MAX_TOKENS || b.max_length < 0 || b.max_length > QMM_MAX_SLOTS)
    return fail(QMM_EINVAL, "max_new must be in [0, %d] and max_length in [0, %d], got %lld and %lld", QMM_MAX_TOKENS,
                QMM_MAX_SLOTS, (long long)b.max_new, (long long)b.max_length);
  if (window < 0) return fail(QMM_EINVAL, "window must not be negative, got %lld", (long long)window);
  if (num_cus < 1 || num_cus > QMM_MAX_CUS)
    return fail(QMM_EINVAL, "num_cus must be in [1, %d], got %d", QMM_MAX_CUS, num_cus);
  if (n_tok > 0) {
    const qmm::AttnPlan plan = qmm::plan_attention(cache->type, heads, cache->heads, cache->head_dim, b.n_seq, n_tok,
                                                   b.max_new, b.max_length, window, num_cus);
    *out = {plan.work_bytes, plan.work_groups, plan.few ? 1 : 0, plan.columns, plan.tiles, plan.splits, plan.share};
  }
  ok();
  return QMM_OK;
}

int qmm_attention(const qmm_attn* args, const qmm_cache* cache, const qmm_batch* batch, int64_t n_tok, void* work,
                  size_t work_bytes, void* stream) {
  if (args == nullptr) return fail(QMM_EINVAL, "args is NULL");
  const qmm_attn& a = *args;
  if (int rc = check_tokens(n_tok)) return rc;
  qmm::Pools pools{};
  qmm::Batch b{};
  if (int rc = check_cache(cache, batch, n_tok, 3, &pools, &b)) return rc;
  if (int rc = check_attention_sizes(*cache, a.heads, n_tok)) return rc;
  const int type = cache->type == QMM_BF16 ? QMM_BF16 : QMM_F16;
  const int64_t dim = cache->head_dim, id = dim * a.heads;
  if (a.out_type != type && a.out_type != QMM_Q8)
    return fail(QMM_EINVAL, "out_type must be that of q (%d with this cache) or QMM_Q8 (%d), got %d", type, QMM_Q8, a.out_type);
  if (a.causal != 0 && a.causal != 1) return fail(QMM_EINVAL, "causal must be 0 or 1, got %d", a.causal);
  if (!(a.scale >= 1e-30f) || !(a.scale <= 1e30f))  // its multiples of a few stay normal numbers
    return fail(QMM_EINVAL, "scale must be in [1e-30, 1e30]");
  if (a.window < 0 || (a.window > 0 && a.causal == 0))
    return fail(QMM_EINVAL, "window must be 0, or positive with causal, got %lld", (long long)a.window);
  if ((work == nullptr) != (work_bytes == 0) || !aligned(work, 16))
    return fail(QMM_EINVAL, "work must be 16-byte aligned and come with its size (NULL with 0)");
  const size_t need = a.out_type == QMM_Q8 ? qmm_qact_bytes(n_tok, id) : 0;
  if (a.out_type == QMM_Q8) {
    if (id % 256 != 0 || id > QMM_MAX_ID)
      return fail(QMM_EINVAL, "a q8 output needs heads * head_dim %% 256 == 0 and at most %d, got %lld", QMM_MAX_ID, (long long)id);
    if (a.out_stride < 0 || (size_t)a.out_stride != need)
      return fail(QMM_EINVAL, "out_stride %lld != qmm_qact_bytes(%lld, %lld) = %zu", (long long)a.out_stride, (long long)n_tok,
                  (long long)id, need);
  }
  if (n_tok == 0) {  // empty batch: pointers are not used
    ok();
    return QMM_OK;
  }
  if (a.q == nullptr || a.out == nullptr) return fail(QMM_EINVAL, "q or out is NULL");
  if (!aligned(a.out, 16)) return fail(QMM_EINVAL, "out must be 16-byte aligned");
  if (a.out_type != QMM_Q8 && (a.out_stride < id || a.out_stride > QMM_MAX_STRIDE || a.out_stride % 8 != 0))
    return fail(QMM_EINVAL, "out_stride must be a multiple of 8 in [%lld, %d], got %lld", (long long)id, QMM_MAX_STRIDE,
                (long long)a.out_stride);
  qmm::Rows rows{};
  Range q{};
  if (int rc = check_heads("q", a.q, a.q_stride, a.q_head_stride, n_tok, a.heads, dim, 2, &rows, &q)) return rc;
  as_rows(rows, n_tok, a.heads, dim, 2, &q);
  const Range out = need > 0 ? Range{"out", a.out, 0, need} : rows_range("out", a.out, a.out_stride, n_tok, id, 2);
  const Range own{"work", work, 0, work_bytes};
  const BatchRanges fixed(*batch);
  for (const Range& in : {q, pool_range("the cache's k", cache->k, *cache), pool_range("the cache's v", cache->v, *cache),
                          fixed.r[0], fixed.r[1], fixed.r[2]}) {
    if (overlap(out, in)) return refuse_overlap(out, in);
    if (overlap(own, in)) return refuse_overlap(own, in);
  }
  if (overlap(own, out)) return refuse_overlap(own, out);
  int device = -1, num_cus = 0;
  hipError_t e = hipGetDevice(&device);
  if (e != hipSuccess) return fail_hip(e, "hipGetDevice");
  e = hipDeviceGetAttribute(&num_cus, hipDeviceAttributeMultiprocessorCount, device);
  if (e != hipSuccess) return fail_hip(e, "hipDeviceGetAttribute(multiprocessor count)");
  const qmm::AttnPlan plan = qmm::plan_attention(cache->type, a.heads, cache->heads, cache->head_dim, batch->n_seq, n_tok,
                                                 batch->max_new, batch->max_length, a.window, num_cus);
  if (work_bytes < plan.work_bytes)
    return fail(QMM_EINVAL, "work_bytes %zu, but this launch needs %zu bytes of work memory (qmm_attention_plan)", work_bytes,
                plan.work_bytes);
  qmm::AttnArgs r{};
  r.q = a.q;
  r.q_stride = rows.stride;
  r.q_head_stride = rows.head_stride;
  r.out = a.out;
  r.out_stride = a.out_type == QMM_Q8 ? 0 : a.out_stride;
  r.part = (float*)work;
  r.sums = (float2*)((float*)work + (plan.work_bytes > 0 ? (size_t)plan.splits * n_tok * id : 0));
  r.window = a.window;
  r.heads = a.heads;
  r.group = a.heads / cache->heads;
  r.by_group = qmm::Divisor(r.group);
  r.causal = a.causal;
  r.q8_out = a.out_type == QMM_Q8;
  r.splits = plan.splits;
  r.share = plan.share;
  r.columns = plan.columns;
  r.tiles = plan.tiles;
  r.t_pad = token_pad(n_tok);
  r.scale2 = (float)(a.scale * 1.4426950408889634074);
  const auto turn = launch_turn((hipStream_t)stream, plan.work_bytes);
  e = qmm::launch_attention(r, pools, b, plan, (hipStream_t)stream);
  if (e != hipSuccess) return fail_hip(e, "attention launch");
  ok();
  return QMM_OK;
}

}  // extern "C"
