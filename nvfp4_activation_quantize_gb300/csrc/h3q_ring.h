// h3q_ring.h -- which fills of a ring of buffers may be under way, and the parities that their barriers
// are waited for with: plain C++, compiled into the kernels and into a host program of the tests.
//
// Fill k goes to slot k % slots, where it is the (k / slots)-th: its barrier's phase of parity (k / slots) & 1
// completes when the bytes are there.
#pragma once

#include <cstdint>

#include "h3q_pages.h"

namespace h3q {

H3Q_HOST_DEVICE uint32_t fill_slot(uint32_t k, uint32_t slots) { return k % slots; }
H3Q_HOST_DEVICE uint32_t fill_parity(uint32_t k, uint32_t slots) { return (k / slots) & 1u; }

// The first of n fills that may still be under way: the last of each slot (one before it was waited for by
// whoever read the slot and gave it back).  A CTA that gives up waits for the fills from this one on before
// it ends, for its shared memory is the next one's then.
H3Q_HOST_DEVICE uint32_t first_fill_under_way(uint32_t n, uint32_t slots) { return n < slots ? 0 : n - slots; }

}  // namespace h3q
