// The blocks of rows of lists, against a walk over the sequences; and offsets of any contents, which must give rows
// inside the packed ones.  Prints how many rows it looked at.
#include <cstdio>
#include <random>
#include <vector>

#include "../../nvfp4_activation_quantize_gb300/csrc/h3q_blocks.cuh"

int main() {
  std::mt19937 rng(5);
  long looked = 0;
  for (int round = 0; round < 3000; ++round) {
    const int shift = 6 + rng() % 3, size = 1 << shift;
    const int batch = rng() % 7;
    std::vector<int32_t> cu(batch + 1);
    for (int b = 0; b < batch; ++b) {
      const int kind = rng() % 4;
      cu[b + 1] = cu[b] + (kind == 0 ? 0 : kind == 1 ? 1 + rng() % 3 : kind == 2 ? size - 1 + rng() % 3 : rng() % 900);
    }
    const int64_t total = cu[batch] + rng() % 200;
    const int64_t rows = total / size + batch;
    std::vector<int> seen(cu[batch] + 1, 0);
    for (int64_t r = 0; r < rows; ++r, ++looked) {
      const h3q::BlockPlace p = h3q::block_at(cu.data(), batch, total, shift, r);
      if (p.rows == 0) continue;
      const int b = p.sequence;
      if (p.rows < 0 || p.rows > size || p.row0 != cu[b] + static_cast<int64_t>(p.index) * size) return 1;
      if (p.row0 + p.rows > cu[b + 1] || (p.row0 + p.rows < cu[b + 1] && p.rows != size)) return 2;
      if (r != (cu[b] >> shift) + b + p.index) return 3;
      for (int i = 0; i < p.rows; ++i) ++seen[p.row0 + i];
    }
    for (int i = 0; i < cu[batch]; ++i)
      if (seen[i] != 1) return 4;
    // any offsets
    for (int b = 0; b <= batch; ++b) cu[b] = rng() % 3 ? static_cast<int32_t>(rng()) : static_cast<int32_t>(rng() % 2000) - 500;
    for (int64_t r = 0; r < rows; ++r, ++looked) {
      const h3q::BlockPlace p = h3q::block_at(cu.data(), batch, total, shift, r);
      if (p.rows != 0 && (p.rows < 0 || p.rows > size || p.row0 < 0 || p.row0 + p.rows > total)) return 5;
      if (p.rows != 0 && (cu[p.sequence] >> shift) + p.sequence + p.index != r) return 6;
    }
    for (int b = 0; b < batch; ++b) {
      const int64_t n = h3q::rows_of(cu.data(), b, total);
      if (n < 0 || (n > 0 && (cu[b] < 0 || cu[b] + n > total))) return 7;
      // its block rows are among the lists
      if (n > 0 && (cu[b] >> shift) + static_cast<int64_t>(b) + (n + size - 1) / size > rows) return 8;
    }
  }
  std::printf("%ld\n", looked);
  return 0;
}
