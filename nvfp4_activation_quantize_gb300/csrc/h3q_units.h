// h3q_units.h -- which block's unit a persistent CTA takes next: plain C++, compiled into the kernel and into
// a host program of the tests.
#pragma once

#include <cstdint>

#include "h3q_pages.h"

namespace h3q {

// A CTA that works for block b asks the launch for a block that has not started.  `taken`: it was given block
// x, which then never starts by itself.  Blocks [0, units) have a unit, those above none, and no order is
// promised in which blocks start or are given away: also a CTA whose own block has none (`had` false, and
// `units` known) may be given one that has.  Returns the block to go on with, or -1.
H3Q_HOST_DEVICE int64_t next_block(bool taken, int64_t x, bool had, int64_t units) {
  return taken && (had || x < units) ? x : -1;
}

// A unit, or half of one: block b of a launch whose units fill `sms` CTAs and leave `units % sms` for the last turn.
// Where these fit in halves, they are halves: of unit `unit`, `half` 0 or 1 (-1: whole).  Blocks [0, blocks) have one.
struct UnitPart {
  int64_t unit;
  int half;
  int64_t blocks;
};
H3Q_HOST_DEVICE UnitPart part_of(int64_t b, int64_t units, int sms) {
  UnitPart p{b, -1, units};
  const int64_t last = sms > 0 ? units % sms : 0, first = units - last;
  if (2 * last > sms) return p;
  p.blocks = units + last;
  if (b >= first) {
    p.unit = first + (b - first) / 2;
    p.half = static_cast<int>((b - first) & 1);
  }
  return p;
}

// How many blocks more than `most` a launch of at least `least` and at most `most` units needs for such halves (0:
// no number of units between has any).
H3Q_HOST_DEVICE int64_t most_halves(int64_t least, int64_t most, int sms) {
  if (least / sms == most / sms) return 2 * (least % sms) > sms ? 0 : most % sms < sms / 2 ? most % sms : sms / 2;
  return sms / 2;
}

}  // namespace h3q
