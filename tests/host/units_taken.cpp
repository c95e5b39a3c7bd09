// A launch of more blocks than there are units, its blocks started and given away in any order: with next_block
// every unit is taken exactly once.
#include <cstdint>
#include <cstdio>
#include <random>
#include <vector>

#include "../../nvfp4_activation_quantize_gb300/csrc/h3q_units.h"

int main() {
  std::mt19937 rng(11);
  long checked = 0, surplus_first = 0;
  for (int trial = 0; trial < 4000; ++trial) {
    const int64_t units = rng() % 12, blocks = units + rng() % 9;
    const int sms = 1 + rng() % 4;
    std::vector<int64_t> pending(blocks), running;
    for (int64_t i = 0; i < blocks; ++i) pending[i] = i;
    std::vector<int> done(units, 0);
    auto any = [&]() {   // a block that has not started, in no order
      const size_t i = trial % 3 == 0 ? 0 : rng() % pending.size();
      const int64_t b = pending[i];
      pending.erase(pending.begin() + static_cast<long>(i));
      return b;
    };
    while (!pending.empty() || !running.empty()) {
      while (static_cast<int>(running.size()) < sms && !pending.empty()) running.push_back(any());
      const size_t c = rng() % running.size();
      const int64_t b = running[c];
      const bool taken = !pending.empty() && rng() % 8 != 0;
      const int64_t x = taken ? any() : 0;
      const bool had = b < units;
      if (had) ++done[static_cast<size_t>(b)];
      surplus_first += !had && taken && x < units;
      const int64_t next = h3q::next_block(taken, x, had, units);
      if (next >= 0)
        running[c] = next;
      else
        running.erase(running.begin() + static_cast<long>(c));
    }
    for (int64_t u = 0; u < units; ++u) {
      if (done[static_cast<size_t>(u)] != 1)
        return std::printf("unit %ld of %ld taken %d times\n", long(u), long(units), done[static_cast<size_t>(u)]), 1;
      ++checked;
    }
  }
  if (surplus_first < 100) return std::printf("the order was never at stake\n"), 2;
  std::printf("%ld\n", checked);
  return 0;
}
