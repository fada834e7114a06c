// Which sequence has which rows, compiled for the host: whatever the starts hold, a sequence's rows begin at the
// highest start up to its own, so that no row has two sequences and the last one's end is the end of all.
// Prints the number of checks.
#include <algorithm>
#include <cstdio>
#include <random>
#include <vector>

#include "../../quant_q8_gemm_amd/csrc/qmm_cache.h"

int main() {
  std::mt19937 rng(2);
  const int wild[] = {0, 1, -1, 1000000, INT32_MAX, INT32_MIN};
  long checks = 0;
  for (int round = 0; round < 20000; ++round) {
    const int n_seq = 1 + rng() % (rng() % 8 == 0 ? 300 : 6), n_tok = 1 + rng() % 300;
    std::vector<int32_t> starts(n_seq + 1), lengths(n_seq, 7), table(n_seq, 0);
    for (int& v : starts) v = rng() % 10 == 0 ? wild[rng() % 6] : (int)(rng() % (unsigned)(n_tok + 1));
    if (rng() % 2 == 0) {  // in order but for one
      std::sort(starts.begin(), starts.end());
      starts[rng() % (n_seq + 1)] = (int)(rng() % (unsigned)(n_tok + 1));
    }
    const qmm::Batch b{starts.data(), lengths.data(), table.data(), 1, n_seq, 1, n_tok};
    std::vector<int> owner(n_tok, -1);
    int end = 0;
    for (int s = 0; s <= n_seq; ++s) {
      end = std::max(end, std::min(std::max(starts[s], 0), n_tok));
      if (s == n_seq) break;
      const qmm::Sequence q = qmm::sequence(b, 5, s);
      if (q.first != end || q.count < 0 || q.first + q.count > n_tok) {
        std::fprintf(stderr, "sequence %d: rows %d + %d, expected to begin at %d\n", s, q.first, q.count, end);
        return 1;
      }
      for (int row = q.first; row < q.first + q.count; ++row, ++checks) {
        if (owner[row] >= 0) {
          std::fprintf(stderr, "row %d of sequences %d and %d\n", row, owner[row], s);
          return 1;
        }
        owner[row] = s;
      }
    }
    for (int row = std::min(std::max(starts[0], 0), n_tok); row < end; ++row, ++checks)
      if (owner[row] < 0) return 1;
    if (qmm::first_row(b, n_seq) != end) return 1;
  }
  std::printf("%ld\n", checks);
  return 0;
}
