// The lookups of the attention kernels, compiled for the host, in the order in which the kernels make them: every tile
// of a share, by waves or groups that take turns, looked up ahead, in two passes.  Each place is that of the table, or
// -1 behind the end and for pages outside the pool.  Prints the number of checks.
#include <algorithm>
#include <cstdio>
#include <memory>
#include <random>

#include "../../quant_q8_gemm_amd/csrc/qmm_pages.h"

namespace {

long checks = 0;

bool good(const qmm::Batch& b, const qmm::Pools& p, int s, int h, int t, int end, int64_t at, const char* what) {
  ++checks;
  const int64_t want = t < end ? qmm::tile_offset(b, p, s, h, t) : -1;
  if (at == want) return true;
  std::fprintf(stderr, "%s: tile %d of %d at %lld, expected %lld\n", what, t, end, (long long)at, (long long)want);
  return false;
}

// as few_kernel: a tile, the next one, then two ahead
bool few(const qmm::Batch& b, const qmm::Pools& p, int s, int h, int from, int end, int wave, int waves) {
  qmm::Pages pages(b, p, s, h);
  for (int pass = 0; pass < 2; ++pass) {
    int t = from + wave;
    int64_t at = pages.place(t, end), next = pages.place(t + waves, end);
    for (; t < end; t += waves) {
      if (!good(b, p, s, h, t, end, at, "few")) return false;
      at = next;
      next = pages.place(t + 2 * waves, end);
    }
  }
  return true;
}

// as many_kernel: stages of KB tiles, `ahead` of them on their way
template <int KB>
bool many(const qmm::Batch& b, const qmm::Pools& p, int s, int h, int from, int end, int group, int groups, int ahead) {
  qmm::Pages pages(b, p, s, h);
  const int step = KB * groups;
  for (int pass = 0; pass < 2; ++pass) {
    qmm::Places<KB> next;
    const auto right = [&](int t) {
      uint32_t here = 0;
      for (int k = 0; k < KB; ++k) {
        if (!good(b, p, s, h, t + k, end, next.at[k], "many")) return false;
        here |= (uint32_t)(next.at[k] >= 0) << k;
      }
      return here == next.here();
    };
    for (int i = 0; i <= ahead; ++i) {
      next.find(pages, from + group * KB + i * step, end);
      if (!right(from + group * KB + i * step)) return false;
    }
    for (int round = from; round < end; round += step) {
      const int t = round + group * KB + (ahead + 1) * step;
      next.find(pages, t, end);
      if (!right(t)) return false;
    }
  }
  return true;
}

}  // namespace

int main() {
  std::mt19937 rng(3);
  const int dims[] = {64, 96, 128, 192, 256}, types[] = {QMM_F16, QMM_BF16, QMM_Q8}, wild[] = {-1, INT32_MIN, INT32_MAX, 1 << 30};
  for (int round = 0; round < 6000; ++round) {
    const int n_seq = 1 + rng() % 3, shift = 5 + rng() % 4, columns = 1 + rng() % (rng() % 3 == 0 ? 400 : 80);
    // some pools are past 4 GiB
    const qmm::Pools p{nullptr, nullptr, (int)(1 + rng() % 70), dims[rng() % 5], shift, types[rng() % 3],
                       (int)(1 + rng() % (rng() % 2 == 0 ? 50 : 2000000))};
    const int64_t stride = columns + rng() % 3;
    const size_t size = (size_t)((n_seq - 1) * stride + columns);
    const std::unique_ptr<int32_t[]> table(new int32_t[size]);  // of its exact size
    for (size_t i = 0; i < size; ++i)
      table[i] = rng() % 20 == 0 ? wild[rng() % 4] : rng() % 20 == 0 ? p.n_pages : (int)(rng() % (unsigned)p.n_pages);
    const qmm::Batch b{nullptr, nullptr, table.get(), stride, n_seq, columns, 1};
    const int tiles = columns << (shift - 5), s = rng() % n_seq, h = rng() % p.heads;
    for (int i = 0; i < 3; ++i) {
      const int end = 1 + rng() % tiles, from = rng() % (end + 1), even = from & ~1;
      if (!few(b, p, s, h, from, end, rng() % 4, 4) || !few(b, p, s, h, from, end, rng() % 2, 2)) return 1;
      const int groups = 1 + rng() % 2, group = rng() % groups, ahead = 1 + rng() % 3;
      if (!many<1>(b, p, s, h, from, end, group, groups, ahead) || !many<2>(b, p, s, h, even, end, group, groups, ahead)) return 1;
    }
  }
  std::printf("%ld\n", checks);
  return 0;
}
