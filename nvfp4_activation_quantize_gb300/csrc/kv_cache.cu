// kv_cache.cu -- new key and value rows quantized into the paged NVFP4 cache, and
// rows of the cache read back as bf16.
//
// Write: the block quantize of the other producers (h3q_device.cuh) on every 16
// elements of a head, stored where the page table says.  Read: bf16(fl((E2M1value *
// E4M3value) / gsf)).  Both are bound by memory: 4 bytes of bf16 and 1.125 bytes of
// cache per element pair (key and value).
//
// A warp owns 512 / head_dim rows (4 at head_dim 128) and walks heads: a lane is one
// block of one row, so the rows' sequence, page and place are looked up once and
// serve every head, and neighbouring rows of a sequence leave as one contiguous piece
// of a page (4 x 64 bytes of codes, one 32-byte sector of scales).  Some
// heads' loads are in flight before the first is converted.  How many heads a warp
// takes follows from the work: all of a unit's heads cost one lookup, but a decoding
// step of 64 rows x 8 heads has only 16 units if each warp takes them all, so heads
// are dealt out until every SM has its warps.
//
// Measured: 65,280 rows x 56 heads x 128 written in 0.354 ms (0.354 is the bytes' time at the
// copy rate; heads per warp at most 4: 0.361, 16: 0.369 ms); the 160,272 rows x 8 heads x 128 of 32
// prefixes read in 0.142 ms (0.124; heads per warp at most 8: 0.144, 2: 0.152; four heads' loads in
// flight, not two: 0.158, occupancy 4 CTAs a SM instead of 5).  Units go round the warps: with a
// contiguous range for each, 0.370 and 0.171 ms.
#include "h3q_cache.cuh"
#include "h3q_device.cuh"
#include "h3q_internal.h"

namespace h3q {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kWriteUnroll = 4;   // heads whose loads are in flight
constexpr int kReadUnroll = 2;
constexpr int kWriteHeads = 8;    // heads of a unit, at most
constexpr int kReadHeads = 4;

struct RowsArgs {
  PagedCache cache;
  PagedRows at;
  const uint16_t* in[2];   // bf16 rows (write)
  uint16_t* out[2];        // bf16 rows (read), [rows, kv_heads, head_dim]
  int64_t ld[2];
  const float* gsf[2];
  int64_t rows;
  int heads_per_unit;
  int64_t head_units;      // units along the heads
  int64_t units;           // row groups x head units
};

// Where this lane's row lives: the offset of (page, head 0, row in page) in rows of
// the cache, or -1 for a row of no sequence, of a position before its first or past
// its table, or of a page that does not exist.  The warp looks the first row's sequence up
// together; the others' are that one or soon after, so each lane steps on by itself.
template <int ROWS_PER_WARP>
__device__ __forceinline__ int64_t locate(const RowsArgs& a, int64_t row0, int mine, bool* owned) {
  *owned = false;
  int b = warp_find_sequence(a.at.cu, a.at.batch, row0);
  const int64_t r = row0 + mine;
  if (b < 0) {   // the first row is no sequence's: look for every row
#pragma unroll
    for (int i = 1; i < ROWS_PER_WARP; ++i) {
      const int c = warp_find_sequence(a.at.cu, a.at.batch, row0 + i);
      if (i == mine) b = c;
    }
  }
  if (b < 0 || r >= a.rows) return -1;
  int64_t end = a.at.cu[b + 1];
  while (r >= end) {
    if (++b >= a.at.batch) return -1;
    end = a.at.cu[b + 1];
  }
  if (a.at.cu[b] > r) return -1;   // (lists out of order)
  *owned = true;
  const int64_t p = static_cast<int64_t>(a.at.kv_len[b]) - end + r;
  return cache_row_of(p, a.at.table + b * a.at.max_pages, a.at.max_pages, a.cache.num_pages, a.cache.kv_heads,
                      a.cache.page_shift);
}

template <int HD>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(const RowsArgs a) {
  constexpr int kBlocks = HD / 16;             // lanes per row
  constexpr int kRows = 32 / kBlocks;          // rows per warp
  __shared__ float inv_table[2][128];
  const int lane = threadIdx.x & 31;
  const int mine = lane / kBlocks, blk = lane % kBlocks;
  after_stream();
  const float gsf[2] = {*a.gsf[0], *a.gsf[1]};
  fill_inverse_scales(inv_table[0], gsf[0]);
  fill_inverse_scales(inv_table[1], gsf[1]);
  __syncthreads();
  const int64_t nwarps = static_cast<int64_t>(gridDim.x) * kWarps;
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); u < a.units; u += nwarps) {
    const int64_t group = u / a.head_units;
    const int h0 = static_cast<int>(u - group * a.head_units) * a.heads_per_unit;
    const int h1 = h0 + a.heads_per_unit < a.cache.kv_heads ? h0 + a.heads_per_unit : a.cache.kv_heads;
    bool owned;
    const int64_t slot = locate<kRows>(a, group * kRows, mine, &owned);
    const int64_t r = group * kRows + mine;
#pragma unroll 1
    for (int t = 0; t < 2; ++t) {
      const uint16_t* src = (t == 0 ? a.in[0] : a.in[1]) + r * (t == 0 ? a.ld[0] : a.ld[1]) + blk * 16;
      uint8_t* codes = t == 0 ? a.cache.codes[0] : a.cache.codes[1];
      uint8_t* scales = t == 0 ? a.cache.scales[0] : a.cache.scales[1];
      const float g = t == 0 ? gsf[0] : gsf[1];
      for (int h = h0; h < h1; h += kWriteUnroll) {
        Block16 x[kWriteUnroll];
#pragma unroll
        for (int i = 0; i < kWriteUnroll; ++i) {
          if (slot >= 0 && h + i < h1) {
            load_fresh(src + static_cast<int64_t>(h + i) * HD, x[i]);
          } else {
#pragma unroll
            for (int w = 0; w < 8; ++w) x[i].w[w] = 0;
          }
        }
#pragma unroll
        for (int i = 0; i < kWriteUnroll; ++i) {
          if (h + i >= h1) break;  // warp-uniform
          const Quantized q = quantize_block(x[i], g, inv_table[t]);
          const int64_t at = slot + (static_cast<int64_t>(h + i) << a.cache.page_shift);
          // four lanes' scale bytes leave as one word
          uint32_t word = q.sf << (8 * (lane & 3));
          word |= __shfl_xor_sync(0xffffffffu, word, 1);
          word |= __shfl_xor_sync(0xffffffffu, word, 2);
          if (slot >= 0) {
            store_codes(codes + at * (HD / 2) + blk * 8, q.codes_lo, q.codes_hi);
            if ((lane & 3) == 0) store_word(scales + at * kBlocks + blk, word);
          }
        }
      }
    }
  }
}

// bf16 magnitudes of the eight E2M1 codes under one scale byte, 16 bytes: the low
// bytes of codes 0..7, then their high bytes, so that a byte permute whose selectors
// are the codes themselves looks four of them up at once.  (Eight copies of each, so that
// no two lanes' lookups meet in a bank, were no faster: 151 us against 148 for 32 prefixes.)
__device__ __forceinline__ void fill_magnitudes(uint4* tab, float gsf) {
  for (int s = threadIdx.x; s < 128; s += blockDim.x) {
    uint32_t w[4] = {0, 0, 0, 0};
    const float sv = e4m3_value(static_cast<uint32_t>(s));
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const float m = c < 2 ? 0.5f * c : static_cast<float>((2 + (c & 1)) << (c >> 1)) * 0.25f;
      const uint32_t b = float2_to_bf16x2(make_float2(__fdiv_rn(__fmul_rn(m, sv), gsf), 0.0f)) & 0xffffu;
      w[c >> 2] |= (b & 0xffu) << (8 * (c & 3));
      w[2 + (c >> 2)] |= (b >> 8) << (8 * (c & 3));
    }
    tab[s] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// Eight codes -> eight bf16 (four words).
__device__ __forceinline__ void values8(uint32_t codes, const uint4& m, uint32_t* out) {
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const uint32_t c = half == 0 ? codes : codes >> 16;
    const uint32_t sel = c & 0x7777u;
    const uint32_t lo = __byte_perm(m.x, m.y, sel);
    const uint32_t hi = __byte_perm(m.z, m.w, sel);
    // the codes' sign bits 3, 7 (11, 15) go to bits 15 and 31 of the words
    out[2 * half] = __byte_perm(lo, hi, 0x5140) | ((c << 12) & 0x8000u) | ((c << 24) & 0x80000000u);
    out[2 * half + 1] = __byte_perm(lo, hi, 0x7362) | ((c << 4) & 0x8000u) | ((c << 16) & 0x80000000u);
  }
}

template <int HD>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const RowsArgs a) {
  constexpr int kBlocks = HD / 16;
  constexpr int kRows = 32 / kBlocks;
  __shared__ uint4 tab[2][128];
  const int lane = threadIdx.x & 31;
  const int mine = lane / kBlocks, blk = lane % kBlocks;
  after_stream();
  fill_magnitudes(tab[0], *a.gsf[0]);
  fill_magnitudes(tab[1], *a.gsf[1]);
  __syncthreads();
  const int64_t nwarps = static_cast<int64_t>(gridDim.x) * kWarps;
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); u < a.units; u += nwarps) {
    const int64_t group = u / a.head_units;
    const int h0 = static_cast<int>(u - group * a.head_units) * a.heads_per_unit;
    const int h1 = h0 + a.heads_per_unit < a.cache.kv_heads ? h0 + a.heads_per_unit : a.cache.kv_heads;
    bool owned;
    const int64_t slot = locate<kRows>(a, group * kRows, mine, &owned);
    const int64_t r = group * kRows + mine;
#pragma unroll 1
    for (int t = 0; t < 2; ++t) {
      const uint8_t* codes = t == 0 ? a.cache.codes[0] : a.cache.codes[1];
      const uint8_t* scales = t == 0 ? a.cache.scales[0] : a.cache.scales[1];
      uint16_t* dst = (t == 0 ? a.out[0] : a.out[1]) + r * a.cache.kv_heads * HD + blk * 16;
      for (int h = h0; h < h1; h += kReadUnroll) {
        uint32_t lo[kReadUnroll], hi[kReadUnroll], sf[kReadUnroll];
#pragma unroll
        for (int i = 0; i < kReadUnroll; ++i) {
          lo[i] = hi[i] = sf[i] = 0;  // a row that the cache does not hold reads as zero
          if (slot >= 0 && h + i < h1) {
            const int64_t at = slot + (static_cast<int64_t>(h + i) << a.cache.page_shift);
            asm volatile("ld.global.L1::no_allocate.v2.b32 {%0,%1}, [%2];"
                         : "=r"(lo[i]), "=r"(hi[i])
                         : "l"(codes + at * (HD / 2) + blk * 8));
            sf[i] = scales[at * kBlocks + blk] & 0x7fu;
          }
        }
#pragma unroll
        for (int i = 0; i < kReadUnroll; ++i) {
          if (!owned || h + i >= h1) continue;
          const uint4 m = tab[t][sf[i]];
          Block16 v;
          values8(lo[i], m, v.w);
          values8(hi[i], m, v.w + 4);
          asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst + static_cast<int64_t>(h + i) * HD),
                       "r"(v.w[0]), "r"(v.w[1]), "r"(v.w[2]), "r"(v.w[3]), "r"(v.w[4]), "r"(v.w[5]), "r"(v.w[6]),
                       "r"(v.w[7])
                       : "memory");
        }
      }
    }
  }
}

// Heads per warp and the units that follow: as many heads as keep 16 warps on each of
// 152 SMs busy, at most `most`.
void plan_units(RowsArgs& a, int rows_per_warp, int most) {
  const int64_t groups = (a.rows + rows_per_warp - 1) / rows_per_warp;
  int64_t per = groups * a.cache.kv_heads / (152 * 16);
  per = per < 1 ? 1 : per > most ? most : per;
  if (per > a.cache.kv_heads) per = a.cache.kv_heads;
  a.heads_per_unit = static_cast<int>(per);
  a.head_units = (a.cache.kv_heads + per - 1) / per;
  a.units = groups * a.head_units;
}

template <int HD>
cudaError_t launch_rows(RowsArgs a, bool write, cudaStream_t stream) {
  plan_units(a, 512 / HD, write ? kWriteHeads : kReadHeads);
  const void* kernel = write ? reinterpret_cast<const void*>(&cache_write_kernel<HD>)
                             : reinterpret_cast<const void*>(&cache_read_kernel<HD>);
  int blocks = 0;
  cudaError_t err = persistent_blocks(kernel, kThreads, 0, (a.units + kWarps - 1) / kWarps, &blocks);
  if (err != cudaSuccess) return err;
  return launch_early(write ? &cache_write_kernel<HD> : &cache_read_kernel<HD>, blocks, kThreads, 0, stream, a);
}

cudaError_t dispatch(const RowsArgs& a, bool write, cudaStream_t stream) {
  switch (a.cache.head_dim) {
    case 64: return launch_rows<64>(a, write, stream);
    case 128: return launch_rows<128>(a, write, stream);
    default: return launch_rows<256>(a, write, stream);
  }
}

}  // namespace

cudaError_t launch_cache_write(const PagedCache& cache, const PagedRows& at, const uint16_t* const x[2],
                               const int64_t ld[2], const float* const gsf[2], int64_t rows, cudaStream_t stream) {
  RowsArgs a{};
  a.cache = cache;
  a.at = at;
  a.rows = rows;
  for (int t = 0; t < 2; ++t) {
      a.in[t] = x[t];
      a.ld[t] = ld[t];
      a.gsf[t] = gsf[t];
  }
  return dispatch(a, true, stream);
}

cudaError_t launch_cache_read(const PagedCache& cache, const PagedRows& at, uint16_t* const out[2],
                              const float* const gsf[2], int64_t rows, cudaStream_t stream) {
  RowsArgs a{};
  a.cache = cache;
  a.at = at;
  a.rows = rows;
  for (int t = 0; t < 2; ++t) {
      a.out[t] = out[t];
      a.gsf[t] = gsf[t];
  }
  return dispatch(a, false, stream);
}

}  // namespace h3q
