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

}  // namespace h3q
