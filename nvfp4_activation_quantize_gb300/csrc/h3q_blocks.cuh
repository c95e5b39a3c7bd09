// h3q_blocks.cuh -- which rows a block of a packed sequence holds (include/h3q.h, h3q_block_rows), shared by
// the calls that attend over blocks.
#pragma once

#include <cstdint>

#include "h3q_pages.h"

namespace h3q {

// A block of consecutive rows of a sequence; rows = 0: none.
struct BlockPlace {
  int sequence;
  int index;       // number of the block in its sequence
  int64_t row0;    // its first packed row
  int rows;
};

// Rows of sequence b among `total` packed ones: as many as are there, whatever the list holds.
H3Q_HOST_DEVICE int64_t rows_of(const int32_t* cu, int b, int64_t total) {
  const int64_t at = cu[b];
  int64_t n = static_cast<int64_t>(cu[b + 1]) - at;
  if (at < 0) return 0;
  if (n > total - at) n = total - at;
  return n < 0 ? 0 : n;
}

// The block of block row r: sequence b is the last with cu[b] / size + b <= r.  (Sequences' block rows
// cannot meet: a sequence of n rows from row c on has at most (c + n) / size - c / size + 1 blocks.)  `shift`:
// size = 1 << shift.  Lists that decrease give some block or none.
H3Q_HOST_DEVICE BlockPlace block_at(const int32_t* cu, int batch, int64_t total, int shift, int64_t r) {
  BlockPlace p{0, 0, 0, 0};
  if (batch == 0) return p;
  int lo = 0, hi = batch;   // the first sequence past r is in (lo, hi]
  while (hi - lo > 1) {
    const int mid = lo + (hi - lo) / 2;
    if ((cu[mid] >> shift) + static_cast<int64_t>(mid) <= r) {
      lo = mid;
    } else {
      hi = mid;
    }
  }
  const int64_t i = r - (cu[lo] >> shift) - lo;
  const int64_t n = rows_of(cu, lo, total);
  if (i < 0 || i << shift >= n) return p;
  p.sequence = lo;
  p.index = static_cast<int>(i);
  p.row0 = cu[lo] + (i << shift);
  const int64_t left = n - (i << shift);
  p.rows = static_cast<int>(left < (int64_t{1} << shift) ? left : int64_t{1} << shift);
  return p;
}

H3Q_HOST_DEVICE int log2_of(int size) { return size == 64 ? 6 : size == 128 ? 7 : 8; }   // 64, 128 or 256

}  // namespace h3q
