// Records what libqmm launches when two threads call it: the HIP runtime's calls are
// answered here (this program's symbols come before the runtime's), so no GPU is used.
// Behind every launch of a product the thread sleeps, which lets the other thread
// launch in between where nothing stops it.
//
//   launch_order <libqmm.so> <mmq | noalloc | epilogue | work> <stream | per_thread>
//
// One stream: every product has to be followed by its own second kernel, which reads
// the partial sums that the product left.  hipStreamPerThread names a stream of each
// thread: no two of them may leave their partials in the same place.
#include <hip/hip_runtime_api.h>

#include <dlfcn.h>

#include <barrier>
#include <chrono>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <mutex>
#include <thread>
#include <vector>

#include "../../include/qmm.h"

namespace {

struct Launch {
  int thread;
  const void* kernel;
  const void* part;  // of a product: its partial sums
};
std::mutex g_mu;
std::vector<Launch> g_launches;
const void* g_product = nullptr;
thread_local int t_thread = 0;

constexpr int kPartArg = 14;  // of mmq_kernel

}  // namespace

extern "C" {

// what <<<>>> keeps between itself and the launch
hipError_t __hipPushCallConfiguration(dim3, dim3, size_t, hipStream_t) { return hipSuccess; }
hipError_t __hipPopCallConfiguration(dim3*, dim3*, size_t*, hipStream_t*) { return hipSuccess; }
hipError_t hipLaunchKernel(const void* f, dim3, dim3, void** args, size_t, hipStream_t) {
  {
    std::lock_guard<std::mutex> lock(g_mu);
    g_launches.push_back({t_thread, f, f == g_product ? *(void**)args[kPartArg] : nullptr});
  }
  if (f == g_product) std::this_thread::sleep_for(std::chrono::microseconds(300));
  return hipSuccess;
}
hipError_t hipMalloc(void** p, size_t n) {
  *p = aligned_alloc(4096, (n + 4095) / 4096 * 4096);
  return *p != nullptr ? hipSuccess : hipErrorOutOfMemory;
}
hipError_t hipFree(void* p) {
  free(p);
  return hipSuccess;
}
hipError_t hipGetDevice(int* d) {
  *d = 0;
  return hipSuccess;
}
hipError_t hipSetDevice(int) { return hipSuccess; }
hipError_t hipDeviceGetAttribute(int* v, hipDeviceAttribute_t, int) {
  *v = 256;  // compute units
  return hipSuccess;
}
hipError_t hipMemcpyAsync(void*, const void*, size_t, hipMemcpyKind, hipStream_t) { return hipSuccess; }
hipError_t hipStreamSynchronize(hipStream_t) { return hipSuccess; }
hipError_t hipStreamIsCapturing(hipStream_t, hipStreamCaptureStatus* s) {
  *s = hipStreamCaptureStatusNone;
  return hipSuccess;
}
hipError_t hipGetLastError() { return hipSuccess; }
hipError_t hipFuncSetAttribute(const void*, hipFuncAttribute, int) { return hipSuccess; }
hipError_t hipGetSymbolAddress(void** p, const void*) {
  static char place[16];
  *p = place;
  return hipSuccess;
}

}  // extern "C"

int main(int argc, char** argv) {
  if (argc != 4) return 2;
  void* lib = dlopen(argv[1], RTLD_NOW);
  if (lib == nullptr) {
    fprintf(stderr, "%s\n", dlerror());
    return 2;
  }
#define ENTRY(name) const auto name = (decltype(&::name))dlsym(lib, #name)
  ENTRY(qmm_register_weights);
  ENTRY(qmm_qact_bytes);
  ENTRY(qmm_mmq);
  ENTRY(qmm_mmq_noalloc);
  ENTRY(qmm_mmq_epilogue);
  ENTRY(qmm_mmq_plan);
  ENTRY(qmm_stream_release);
  ENTRY(qmm_last_error);
#undef ENTRY
  const bool per_thread = strcmp(argv[3], "per_thread") == 0;
  const hipStream_t stream = per_thread ? hipStreamPerThread : (hipStream_t)0x1000;
  constexpr int64_t kOd = 4352, kId = 2048, kTok = 509;
  qmm_plan plan;
  if (qmm_mmq_plan(QMM_Q6_K, kOd, kId, kTok, 256, &plan) != QMM_OK || plan.n_tail == 0) {
    fprintf(stderr, "the shape has no split tail\n");
    return 2;
  }
  const std::vector<char> raw(kOd * (kId / 256) * 210);
  qmm_weights* w = nullptr;
  if (qmm_register_weights(QMM_Q6_K, kOd, kId, raw.data(), raw.size(), stream, &w) != QMM_OK) {
    fprintf(stderr, "%s\n", qmm_last_error());
    return 2;
  }
  const size_t bytes = qmm_qact_bytes(kTok, kId);
  char* const base = (char*)(1ull << 40);  // addresses that nothing reads
  auto call = [&](int thread) {
    char* const out = base + ((size_t)(1 + thread) << 30);
    if (strcmp(argv[2], "mmq") == 0) return qmm_mmq(w, base, bytes, kTok, (float*)out, stream);
    if (strcmp(argv[2], "noalloc") == 0) return qmm_mmq_noalloc(w, base, bytes, kTok, (float*)out, stream);
    const bool work = strcmp(argv[2], "work") == 0;
    return qmm_mmq_epilogue(w, base, bytes, kTok, nullptr, QMM_F32, out, kOd, work ? base + ((size_t)9 << 30) : nullptr,
                            work ? plan.scratch_bytes : 0, stream);
  };
  g_launches.clear();
  if (call(0) != QMM_OK || g_launches.size() != 2) {
    fprintf(stderr, "not a product and its second kernel: %zu launches, %s\n", g_launches.size(), qmm_last_error());
    return 2;
  }
  g_product = g_launches[0].kernel;
  const void* const second = g_launches[1].kernel;
  g_launches.clear();

  constexpr int kThreads = 2, kCalls = 20;
  std::barrier start(kThreads), done(kThreads);
  std::vector<std::thread> threads;
  size_t freed[kThreads] = {};
  for (int i = 0; i < kThreads; ++i)
    threads.emplace_back([&, i] {
      t_thread = i;
      start.arrive_and_wait();
      for (int k = 0; k < kCalls; ++k)
        if (call(i) != QMM_OK) fprintf(stderr, "%s\n", qmm_last_error());
      done.arrive_and_wait();
      if (per_thread && qmm_stream_release(stream, &freed[i]) != QMM_OK) fprintf(stderr, "%s\n", qmm_last_error());
    });
  for (auto& t : threads) t.join();

  if (g_launches.size() != 2 * kThreads * kCalls) {
    fprintf(stderr, "%zu launches\n", g_launches.size());
    return 1;
  }
  if (per_thread) {
    for (const Launch& a : g_launches)
      for (const Launch& b : g_launches)
        if (a.thread != b.thread && a.part != nullptr && a.part == b.part) {
          fprintf(stderr, "two threads' streams share their partial sums\n");
          return 1;
        }
    for (size_t f : freed)
      if (f != (size_t)256 * 64 * 1024) {
        fprintf(stderr, "a thread released %zu bytes\n", f);
        return 1;
      }
    return 0;
  }
  for (size_t i = 0; i < g_launches.size(); i += 2)
    if (g_launches[i].kernel != g_product || g_launches[i + 1].kernel != second ||
        g_launches[i].thread != g_launches[i + 1].thread) {
      fprintf(stderr, "launch %zu: another call's kernel between a product and its second kernel\n", i);
      return 1;
    }
  return 0;
}
