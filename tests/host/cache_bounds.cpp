// Where the kernels look for a sequence's rows, slots and tiles, compiled for the host:
// with arrays that hold anything, rows stay rows of the call, slots have a column, and
// a tile's place is inside its pool or -1.  Prints the number of checks.
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "../../quant_q8_gemm_amd/csrc/qmm_cache.h"

int main() {
  std::mt19937 rng(1);
  const int wild[] = {0, 1, -1, 31, 32, 33, 1000, -1000, 1 << 30, -(1 << 30), INT32_MAX, INT32_MIN};
  const auto any = [&](int high) {
    return rng() % 4 == 0 ? wild[rng() % 12] : (int)(rng() % (unsigned)(high + 2)) - (rng() % 8 == 0 ? 1 : 0);
  };
  const int dims[] = {64, 96, 128, 192, 256}, types[] = {QMM_F16, QMM_BF16, QMM_Q8};
  long checks = 0;
  for (int round = 0; round < 20000; ++round) {
    const int n_seq = 1 + rng() % 5, columns = 1 + rng() % 7, n_tok = 1 + rng() % 300, shift = 5 + rng() % 4;
    qmm::Pools p{nullptr, nullptr, (int)(1 + rng() % 9), dims[rng() % 5], shift, types[rng() % 3], (int)(1 + rng() % 50)};
    const int64_t stride = columns + rng() % 3;
    std::vector<int32_t> starts(n_seq + 1), lengths(n_seq), table((n_seq - 1) * stride + columns);
    for (int& v : starts) v = any(n_tok);
    for (int& v : lengths) v = any(columns << shift);
    for (int& v : table) v = any(p.n_pages);
    const qmm::Batch b{starts.data(), lengths.data(), table.data(), stride, n_seq, columns, n_tok};
    const int64_t page = (int64_t)p.heads * (1 << (shift - 5)) * qmm::tile_bytes(p.type, p.dim);
    if (page != (int64_t)p.heads * (1 << shift) * p.dim * (p.type == QMM_Q8 ? 34 : 64) / 32) return 1;
    for (int s = 0; s < n_seq; ++s) {
      const qmm::Sequence q = qmm::sequence(b, shift, s);
      if (q.first < 0 || q.count < 0 || q.first + q.count > n_tok || q.length < 0 || q.length > columns << shift) {
        std::fprintf(stderr, "sequence: %d + %d of %d, length %d\n", q.first, q.count, n_tok, q.length);
        return 1;
      }
      for (int tile = 0; 32 * tile < q.length; ++tile)
        for (int h = 0; h < p.heads; ++h, ++checks) {
          const int64_t at = qmm::tile_offset(b, p, s, h, tile);
          const int id = table[s * stride + (tile >> (shift - 5))];
          if ((at < 0) != (id < 0 || id >= p.n_pages) || at + qmm::tile_bytes(p.type, p.dim) > page * p.n_pages) {
            std::fprintf(stderr, "tile %d of page %d of %d at %lld\n", tile, id, p.n_pages, (long long)at);
            return 1;
          }
        }
    }
  }
  // every element of a tile has a place of its own
  for (int dim : dims) {
    std::vector<char> k(32 * dim), v(32 * dim), kc(34 * dim), vc(34 * dim);
    for (int r = 0; r < 32; ++r)
      for (int d = 0; d < dim; ++d, checks += 4)
        if (k[qmm::key_at(r, d)]++ || v[qmm::value_at(r, d)]++ || kc[qmm::key_code_at(r, d)]++ || vc[qmm::value_code_at(r, d)]++)
          return 1;
    for (int r = 0; r < 32; ++r)
      for (int c = 0; c < dim / 32; ++c)
        for (int i = 0; i < 2; ++i)
          if (kc[qmm::scale_at(dim, r, c) + i]++) return 1;
    for (char c : kc)
      if (c != 1) return 1;
  }
  std::printf("%ld\n", checks);
  return 0;
}
