// h3q_cache.cuh -- the paged NVFP4 key/value cache as the kernels see it.
//
// codes [num_pages, kv_heads, page_size, head_dim/2] and scales [num_pages,
// kv_heads, page_size, head_dim/16], keys and values apart: the rows of one head in
// one page are contiguous (64 bytes of codes a row at head_dim 128), so a page is
// one copy for the reader, and its scales are another.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "h3q_device.cuh"
#include "h3q_pages.h"

namespace h3q {

struct PagedCache {
  uint8_t* codes[2];   // keys, values
  uint8_t* scales[2];
  int64_t num_pages;
  int kv_heads;
  int head_dim;
  int page_shift;      // page_size = 1 << page_shift
};

// Which sequence holds which of the packed rows, and where in the cache: the n rows
// cu[b] .. cu[b + 1] - 1 of sequence b stand at its last n positions
// kv_len[b] - n .. kv_len[b] - 1, position p in page table[b * max_pages + p / page_size].
struct PagedRows {
  const int32_t* cu;
  const int32_t* kv_len;
  const int32_t* table;
  int64_t max_pages;
  int batch;
};

// The sequence of packed row r: the last b of [0, batch) with cu[b] <= r < cu[b + 1],
// or -1 when the row belongs to none.  The whole warp searches: 32 probes a step, so
// two dependent loads for a thousand sequences.  Any contents of cu end the search.
__device__ __forceinline__ int warp_find_sequence(const int32_t* cu, int batch, int64_t r) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = batch;
  while (n > 1) {
    const int step = (n + 31) >> 5;
    const int at = lo + lane * step;
    const bool le = lane * step < n && static_cast<int64_t>(cu[at]) <= r;
    const int cnt = __popc(__ballot_sync(0xffffffffu, le));
    if (cnt == 0) return -1;
    const int skip = (cnt - 1) * step;
    lo += skip;
    n = n - skip < step ? n - skip : step;
  }
  return static_cast<int64_t>(cu[lo]) <= r && r < static_cast<int64_t>(cu[lo + 1]) ? lo : -1;
}

// A launch that may begin while the stream's work before it ends: its CTAs are there when that is done.
// Every thread of the kernel calls after_stream() before it reads or writes memory, and no load is .nc: memory may
// change while the kernel is resident.  (A token's write and attention at 777 positions, from a graph: 12.3 us,
// with plain launches 12.8; with the kernels letting the next one in as they begin 12.5.)
template <class... P, class... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

__device__ __forceinline__ void after_stream() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// load_stream and load16_reused (h3q_device.cuh) for such kernels: what they read may change while they are
// resident, which .nc promises it does not.
__device__ __forceinline__ void load_fresh(const void* p, Block16& b) {
  asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(b.w[0]), "=r"(b.w[1]), "=r"(b.w[2]), "=r"(b.w[3]), "=r"(b.w[4]),
                 "=r"(b.w[5]), "=r"(b.w[6]), "=r"(b.w[7])
               : "l"(p));
}

__device__ __forceinline__ uint4 load16_fresh(const void* p) {
  uint4 v;
  asm volatile("ld.global.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

}  // namespace h3q
