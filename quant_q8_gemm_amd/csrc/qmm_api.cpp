// qmm_api.cpp -- the C ABI declared in include/qmm.h: argument validation (all of
// it before the first HIP call), weight-handle lifetime, device-memory
// accounting, and the launches.  No compute happens here.
#include <hip/hip_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <mutex>
#include <string>
#include <vector>

#include "../../include/qmm.h"
#include "qmm_epilogue.h"
#include "qmm_internal.h"

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
