// Every position around a sequence's pages, with page numbers that exist and that do not: the place
// that h3q_pages.h gives is inside the cache and is the layout's, or it is "none".
#include <cstdint>
#include <cstdio>
#include <limits>
#include <vector>

#include "../../nvfp4_activation_quantize_gb300/csrc/h3q_pages.h"

int main() {
  long checked = 0;
  const int32_t lo = std::numeric_limits<int32_t>::min(), hi = std::numeric_limits<int32_t>::max();
  for (int shift = 4; shift <= 7; ++shift)
    for (int64_t pages : {int64_t{1}, int64_t{5}, int64_t{hi}})
      for (int64_t heads : {int64_t{1}, int64_t{7}, int64_t{1} << 18}) {
        const std::vector<int32_t> table = {0, static_cast<int32_t>(pages - 1), -1, lo, hi, 4};
        const int64_t page = int64_t{1} << shift;
        for (int64_t p = -2 * page; p < 8 * page; ++p) {
          const int64_t got = h3q::cache_row_of(p, table.data(), static_cast<int64_t>(table.size()), pages, heads, shift);
          int64_t want = -1;
          if (p >= 0 && p / page < static_cast<int64_t>(table.size())) {
            const int64_t n = table[p / page];
            if (n >= 0 && n < pages) want = n * heads * page + p % page;
          }
          if (got != want || got >= pages * heads * page) {
            std::printf("p %ld: %ld, wanted %ld\n", long(p), long(got), long(want));
            return 1;
          }
          ++checked;
        }
        for (int64_t p : {int64_t{lo} * 2, int64_t{hi} * 2, int64_t{1} << 60})
          if (h3q::cache_row_of(p, table.data(), static_cast<int64_t>(table.size()), pages, heads, shift) != -1) return 2;
      }
  std::printf("%ld\n", checked);
  return 0;
}
