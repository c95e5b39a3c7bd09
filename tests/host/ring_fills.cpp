// A ring of buffers with a barrier each (a phase that flips when a fill's bytes have landed), filled and read for
// random times and given up at any moment: after the waits that h3q_ring.h names no fill is under way.
#include <cstdint>
#include <cstdio>
#include <random>
#include <vector>

#include "../../nvfp4_activation_quantize_gb300/csrc/h3q_ring.h"

int main() {
  std::mt19937 rng(7);
  long checked = 0;
  for (uint32_t slots = 1; slots <= 5; ++slots)
    for (int trial = 0; trial < 3000; ++trial) {
      std::vector<uint32_t> issued(slots, 0), landed(slots, 0);   // fills of each slot
      uint32_t n = 0, taken = 0;                                  // fills issued, and read and given back
      auto land = [&](uint32_t s) { landed[s] += landed[s] < issued[s]; };
      auto arrived = [&](uint32_t k) {   // the wait: the phase of this parity is over
        return (landed[h3q::fill_slot(k, slots)] & 1u) != h3q::fill_parity(k, slots);
      };
      const int steps = static_cast<int>(rng() % 40);
      for (int i = 0; i < steps; ++i) {
        switch (rng() % 3) {
          case 0:   // the next fill, where its slot was given back
            if (n < taken + slots) ++issued[h3q::fill_slot(n, slots)], ++n;
            break;
          case 1: land(rng() % slots); break;
          default:
            if (taken < n && arrived(taken)) ++taken;
        }
      }
      // given up: what is waited for
      for (uint32_t k = h3q::first_fill_under_way(n, slots); k < n; ++k)
        for (int t = 0; !arrived(k); ++t) {
          if (t > 3) return std::printf("fill %u of %u in %u slots never arrives\n", k, n, slots), 1;
          land(h3q::fill_slot(k, slots));
        }
      for (uint32_t s = 0; s < slots; ++s)
        if (landed[s] != issued[s]) return std::printf("slot %u of %u: a fill is under way\n", s, slots), 1;
      ++checked;
    }
  std::printf("%ld\n", checked);
  return 0;
}
