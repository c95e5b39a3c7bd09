// h3q_pages.h -- where a position of a sequence lives in the paged cache: plain C++,
// compiled into the kernels and into a host program of the tests.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define H3Q_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define H3Q_HOST_DEVICE inline
#endif

namespace h3q {

// The page that holds position p of a sequence whose page list is table_row, or -1
// where there is none: p negative or past the list, or the list names no page of
// [0, num_pages).
H3Q_HOST_DEVICE int64_t page_of(int64_t p, const int32_t* table_row, int64_t max_pages, int64_t num_pages,
                                int page_shift) {
  if (p < 0) return -1;
  const int64_t at = p >> page_shift;
  if (at >= max_pages) return -1;
  const int64_t page = table_row[at];
  return page >= 0 && page < num_pages ? page : -1;
}

// Row of the cache (page, head 0, row in page) of position p, in rows of one head, or -1.
H3Q_HOST_DEVICE int64_t cache_row_of(int64_t p, const int32_t* table_row, int64_t max_pages, int64_t num_pages,
                                     int64_t kv_heads, int page_shift) {
  const int64_t page = page_of(p, table_row, max_pages, num_pages, page_shift);
  if (page < 0) return -1;
  return ((page * kv_heads) << page_shift) + (p & ((int64_t{1} << page_shift) - 1));
}

}  // namespace h3q
