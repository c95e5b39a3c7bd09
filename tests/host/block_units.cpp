// Prints, for each "units sms" line of stdin, "ok" if the blocks of a launch cover every unit once: whole, or in both
// halves, these last and all in one turn.
#include <cinttypes>
#include <cstdio>
#include <vector>

#include "h3q_units.h"

int main() {
  int64_t units;
  int sms;
  while (std::scanf("%" SCNd64 " %d", &units, &sms) == 2) {
    std::vector<int> seen(units, 0);
    const int64_t blocks = h3q::part_of(0, units, sms).blocks;
    bool ok = blocks >= units && blocks <= units + sms / 2;
    int64_t halves = 0;
    for (int64_t b = 0; b < blocks && ok; ++b) {
      const h3q::UnitPart p = h3q::part_of(b, units, sms);
      ok = p.unit >= 0 && p.unit < units && p.blocks == blocks && p.half >= -1 && p.half <= 1;
      if (!ok) break;
      ok = (seen[p.unit] & (p.half < 0 ? 3 : 1 << p.half)) == 0 && (p.half >= 0 || halves == 0);
      seen[p.unit] |= p.half < 0 ? 3 : 1 << p.half;
      halves += p.half >= 0;
    }
    for (int s : seen) ok = ok && s == 3;
    for (int64_t b = blocks; b < blocks + 3; ++b) ok = ok && h3q::part_of(b, units, sms).unit >= units;
    for (int64_t more = 0; more < 12 && sms > 0; ++more) {   // launches for at most so many units
      const int64_t halves_at_most = h3q::most_halves(units, units + more, sms);
      for (int64_t u = units; u <= units + more; ++u) {
        const int64_t need = h3q::part_of(0, u, sms).blocks;
        ok = ok && need <= units + more + (halves_at_most > 0 ? halves_at_most : 0);
        ok = ok && (halves_at_most > 0 || need == u);
      }
      // (also where the sequences hold fewer rows than there are)
      for (int64_t u = 0; u < units && units < 1000; ++u)
        ok = ok && (halves_at_most == 0 || h3q::part_of(0, u, sms).blocks <= units + more + halves_at_most);
    }
    std::puts(ok && halves <= (sms > 0 ? sms : 0) ? "ok" : "bad");
  }
}
