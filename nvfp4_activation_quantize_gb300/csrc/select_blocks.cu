// select_blocks.cu -- the blocks of keys that each block of queries attends to.
//
// Score of query block i and key block j of a key head: (sum of the block's query rows, over the
// heads of the group) . (sum of the block's keys) / (keys of the block).  The `top` highest
// are kept; of equal ones those with the lowest numbers.
//
// Two kernels.
//   pool    sums the rows of each block of q and of k: every input byte is read once, which is
//           the bound (DRAM).  The sums are kept as hi + lo, two fp32.  A running sum begins at a
//           constant that is larger than all that can come (S. M. Rump, T. Ogita and S. Oishi,
//           "Accurate floating-point summation part I", SIAM J. Sci. Comput. 31(1), 2008): what its
//           rounding leaves of each value is exact and goes to a sum of its own, four packed
//           additions a pair of values (65,280 rows of 56 + 56 heads of 128 in 280 us, 6.9 TB/s with what is
//           written).  A sum of
//           up to 256 values is exact where they lie within a factor of 2^18 of each other, and else off by
//           2^-20 of the largest at most (both 2^-1 for each doubling of their number).
//   score   16 query blocks a CTA against all key blocks of their sequence, with mma.sync m16n8k16 (16 rows are
//           what there is; scores go straight to the choice), on two fp16 parts of each sum, scaled: three
//           products are as good as fp32's.  q's operands are in shared memory, k's come from L2 in the order
//           that a lane wants, a load of 16 bytes for three products.  Then a warp per query block takes its
//           scores into registers and looks for the top-th highest.  65,280 tokens' 510 x 510 scores of 56
//           heads, of which 64 a row are kept: 145 us (284 with fp32 products from tiles in shared memory).
//           Bound: latency with 24 warps an SM, of the products' loads (80 us) and the choice's steps (55).
//
// What these products cannot tell apart is told apart by fp32 pairs: a score is off by at most
// delta = 176 * 2^-24 * |q| |k|, of the largest |k|.  (Parts and the product of two second parts: 3 * 2^-22.  A
// product of 16 values adds 17 terms, of each of which it may cut what is below 2^-23 of the largest, and rounds,
// 36 * 2^-24 at most: M. Fasi, N. J. Higham, M. Mikaitis and S. Pranesh, "Numerical behavior of NVIDIA tensor
// cores", PeerJ Comput. Sci. 7, 2021.  Four of them follow each other in each of two sums, 144; in the other two, of
// second parts, they are 2^-10 of that.  Sums, mean: 6.)  Where the top-th score is more than 2 delta above the next, the
// choice is the exact one.  Where it is not (one list in forty for unrelated blocks), the scores within 2 delta of it
// are formed again from hi + lo in pairs of fp32, and the places that are left go to the highest of those.  What is
// compared is their distance from the border, 3 delta at most, in fp32: 2^-39 of |q| |k|; the pairs' own error is 2^-40
// (some 18 sums of rests that come to 10 * 2^-24 at most, each rounded).
#include <cuda_fp16.h>

#include <cfloat>
#include <cmath>

#include "h3q_blocks.cuh"
#include "h3q_device.cuh"
#include "h3q_internal.h"

namespace h3q {
namespace {

// ---------------------------------------------------------------------------- pool

constexpr int kPoolThreads = 128;

// The workspace: hi and lo parts of q and of k, [kv_heads][block rows][head_dim], for each block the length of its sums
// as a vector (infinity where one is no number), and k once more as two fp16 parts for the products, scaled by
// a power of two that takes the block's size to 2^14: [8 rows of all heads'][16 dimensions][row][4 dimensions], for
// these the first parts and the second ones, so that a load of 16 bytes a lane is an operand of the products.
struct Sums {
  float* hi[2];
  float* lo[2];
  float* size[2];
  uint4* parts;
  int64_t rows[2];   // block rows
  uint32_t* far;     // rows of scores that no CTA holds, one for each of kFarRows CTAs at most, or nullptr
  int64_t far_row;   // scores of such a row
};

Sums carve(const BlockShape& s, uint8_t* workspace) {
  Sums w{};
  w.rows[0] = s.rows_q / s.block_q + s.batch;
  w.rows[1] = s.rows_k / s.block_k + s.batch;
  float* at = reinterpret_cast<float*>(workspace);
  for (int t = 0; t < 2; ++t) {
    const int64_t n = w.rows[t] * s.kv_heads * s.head_dim;
    w.hi[t] = at;
    w.lo[t] = at + n;
    at += 2 * n;
  }
  w.parts = reinterpret_cast<uint4*>(at);   // (16-byte aligned: head_dim is a multiple of 4)
  at += (w.rows[1] * s.kv_heads + 7) / 8 * 8 * s.head_dim;
  for (int t = 0; t < 2; ++t) {
    w.size[t] = at;
    at += w.rows[t] * s.kv_heads;
  }
  if (s.rows_k / s.block_k > kNearBlocks) {
    w.far = reinterpret_cast<uint32_t*>(at);
    w.far_row = (s.rows_k / s.block_k + 32) / 32 * 32;
  }
  return w;
}

// block_at for up to 32 sequences, a lane for each: one wait for memory, where halving waits for every step.  Whole warp.
__device__ __forceinline__ BlockPlace block_at_once(const int32_t* cu, int batch, int64_t total, int shift, int64_t r) {
  const int lane = threadIdx.x & 31;
  BlockPlace p{0, 0, 0, 0};
  if (batch == 0) return p;
  int first = 0, end = 0;
  if (lane < batch) {
    first = cu[lane];
    end = cu[lane + 1];
  }
  const uint32_t upto = __ballot_sync(0xffffffffu, lane < batch && (first >> shift) + static_cast<int64_t>(lane) <= r);
  p.sequence = upto != 0u ? 31 - __clz(upto) : 0;
  first = __shfl_sync(0xffffffffu, first, p.sequence);
  end = __shfl_sync(0xffffffffu, end, p.sequence);
  int64_t n = static_cast<int64_t>(end) - first;
  if (n > total - first) n = total - first;
  const int64_t i = r - (first >> shift) - p.sequence, left = n - (i << shift);
  if (first < 0 || i < 0 || left <= 0) return p;
  p.index = static_cast<int>(i);
  p.row0 = first + (i << shift);
  p.rows = static_cast<int>(left < (int64_t{1} << shift) ? left : int64_t{1} << shift);
  return p;
}

struct PoolArgs {
  const uint16_t* x[2];
  int64_t ld[2];
  const int32_t* cu[2];
  int64_t total[2];
  int shift[2];
  int group[2];      // heads that are summed together
  int batch, kv_heads;
  Sums sums;
};

__device__ __forceinline__ float2 sub2(float2 a, float2 b) { return fma2(b, make_float2(-1.0f, -1.0f), a); }

// (hi, lo) += x: hi + error = hi + x without rounding (D. E. Knuth's two-sum, The Art of Computer Programming
// vol. 2, 4.2.2).
__device__ __forceinline__ void add_to(float2& hi, float2& lo, float2 x) {
  const float2 s = add2(hi, x);
  const float2 y = sub2(s, hi);
  lo = add2(lo, add2(sub2(hi, sub2(s, y)), sub2(x, y)));
  hi = s;
}

// Powers of two that take numbers up to `size` (and not above 2^-112) below 2^15, and back.
__device__ __forceinline__ uint32_t exponent_of(float size) { return max(__float_as_uint(size) >> 23, 15u); }
__device__ __forceinline__ float scale_up(float size) { return __uint_as_float((268u - exponent_of(size)) << 23); }
__device__ __forceinline__ float scale_down(float size) { return __uint_as_float((exponent_of(size) - 14u) << 23); }

// x, scaled, as two fp16 parts: to 2^-22 of it (and 2^-25).
__device__ __forceinline__ void halves_of(float2 x, float scale, uint32_t& first, uint32_t& second) {
  x = mul2(x, make_float2(scale, scale));
  const __half2 h = __float22half2_rn(x);
  const __half2 rest = __float22half2_rn(sub2(x, __half22float2(h)));
  first = *reinterpret_cast<const uint32_t*>(&h);
  second = *reinterpret_cast<const uint32_t*>(&rest);
}

template <int HD>
__global__ void __launch_bounds__(kPoolThreads, 6) pool_kernel(const __grid_constant__ PoolArgs a) {
  constexpr int kLanes = HD / 8;            // lanes of a row of a head, 8 values each
  constexpr int kRows = 32 / kLanes;        // rows of a head that a load of the warp takes
  constexpr int kUnroll = 4;                // loads under way while as many are summed
  const int lane = threadIdx.x & 31;
  const int c = lane % kLanes;
  const uint32_t unit = blockIdx.x * (kPoolThreads / 32) + (threadIdx.x >> 5);   // (below 2^31, see the API)
  const uint32_t row_of_unit = unit / static_cast<uint32_t>(a.kv_heads);
  const int head = static_cast<int>(unit - row_of_unit * a.kv_heads);
  int64_t r = row_of_unit;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // (they wait for this kernel's end)
  if (r >= a.sums.rows[0] + a.sums.rows[1]) return;
  const int t = r >= a.sums.rows[0];
  if (t) r -= a.sums.rows[0];
  const BlockPlace p = a.batch <= 32 ? block_at_once(a.cu[t], a.batch, a.total[t], a.shift[t], r)
                                     : block_at(a.cu[t], a.batch, a.total[t], a.shift[t], r);
  if (p.rows == 0) return;   // (never read)
  const int group = a.group[t], items = p.rows * group;   // rows of single heads
  const int64_t ld = a.ld[t];
  const uint16_t* const x = a.x[t] + p.row0 * ld + static_cast<int64_t>(head) * group * HD + c * 8;
  // hi: sums and `offset`, which is 1.5 * 2^k with 2^k at least 4 times what `items` values below `limit` can
  // come to, so that all of them have the same last place.
  float2 hi[4], lo[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) hi[i] = lo[i] = make_float2(0.0f, 0.0f);
  float offset = 0.0f, limit = 0.0f;
  const int growth = 36 - __clz(items);   // 2^growth > 16 * items: 4, and values up to 4 times the exponent's
  bool finite = true;
  // (seldom more than once: a larger value has come)
  auto raise = [&](float most) {
    const int e = max(static_cast<int>(__float_as_uint(most) >> 23), 1) + growth;
    if (e >= 254) {
      finite = false;
      return;
    }
    const float to = __uint_as_float(static_cast<uint32_t>(max(e, 30)) << 23 | 0x400000u);
    const float2 from2 = make_float2(offset, offset), to2 = make_float2(to, to);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = sub2(hi[i], from2);
      hi[i] = add2(to2, v);
      lo[i] = add2(lo[i], sub2(v, sub2(hi[i], to2)));
    }
    offset = to;
    limit = __uint_as_float(static_cast<uint32_t>(max(e - growth + 2, 3)) << 23);
  };
  // The lane's next item: row item / group, head item % group.
  int item = lane / kLanes, item_head = item % group;
  const uint16_t* from = x + item / group * ld + item_head * HD;
  const int heads_on = kRows % group;
  const int64_t step = kRows / group * ld + heads_on * HD, wrap = ld - group * HD;
  auto one = [&]() {
    const uint4 w = load16_stream(from);
    from += step;
    item_head += heads_on;
    if (item_head >= group) {
      item_head -= group;
      from += wrap;
    }
    return w;
  };
  auto load = [&](uint4 (&w)[kUnroll]) {
    if (item + (kUnroll - 1) * kRows < items) {
#pragma unroll
      for (int n = 0; n < kUnroll; ++n) w[n] = one();
    } else {   // the last, or past them
#pragma unroll
      for (int n = 0; n < kUnroll; ++n) {
        w[n] = make_uint4(0u, 0u, 0u, 0u);
        if (item + n * kRows < items) w[n] = one();
      }
    }
    item += kUnroll * kRows;
  };
  auto sum = [&](const uint4 (&w)[kUnroll]) {
    uint32_t most = 0u;
#pragma unroll
    for (int n = 0; n < kUnroll; ++n)
      most = absmax_bf16x2(most, absmax_bf16x2(absmax_bf16x2(w[n].x, w[n].y), absmax_bf16x2(w[n].z, w[n].w)));
    const float largest = halves_amax(most);
    if (!(largest < limit)) raise(largest);
#pragma unroll
    for (int n = 0; n < kUnroll; ++n) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 v = bf16x2_to_float2(i == 0 ? w[n].x : i == 1 ? w[n].y : i == 2 ? w[n].z : w[n].w);
        const float2 s = add2(hi[i], v);
        lo[i] = add2(lo[i], sub2(v, sub2(s, hi[i])));
        hi[i] = s;
      }
    }
  };
  uint4 w0[kUnroll], w1[kUnroll];
  constexpr int kStep = kRows * kUnroll;
  load(w0);
  for (int i0 = lane / kLanes; i0 < items; i0 += 2 * kStep) {   // (zeros past the last change nothing)
    load(w1);
    sum(w0);
    load(w0);
    sum(w1);
  }
  // Values near fp32's end, infinities or values that are no numbers, in any lane: by two-sums, at 2^-32 of their
  // size, so that sums may pass fp32's end on the way.
  constexpr float kDown = 0x1p-32f, kUp = 0x1p32f;
  const bool scaled = !__all_sync(0xffffffffu, finite);
  if (!scaled) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 rest = lo[i];
      hi[i] = sub2(hi[i], make_float2(offset, offset));
      lo[i] = make_float2(0.0f, 0.0f);
      add_to(hi[i], lo[i], rest);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) hi[i] = lo[i] = make_float2(0.0f, 0.0f);
#pragma unroll 1
    for (int i0 = lane / kLanes; i0 < items; i0 += kRows) {
      const uint4 w = load16_stream(x + i0 / group * ld + (i0 % group) * HD);
      add_to(hi[0], lo[0], mul2(bf16x2_to_float2(w.x), make_float2(kDown, kDown)));
      add_to(hi[1], lo[1], mul2(bf16x2_to_float2(w.y), make_float2(kDown, kDown)));
      add_to(hi[2], lo[2], mul2(bf16x2_to_float2(w.z), make_float2(kDown, kDown)));
      add_to(hi[3], lo[3], mul2(bf16x2_to_float2(w.w), make_float2(kDown, kDown)));
    }
  }
  // the other rows' lanes
#pragma unroll
  for (int o = kLanes; o < 32; o <<= 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 h = make_float2(__shfl_xor_sync(0xffffffffu, hi[i].x, o), __shfl_xor_sync(0xffffffffu, hi[i].y, o));
      const float2 l = make_float2(__shfl_xor_sync(0xffffffffu, lo[i].x, o), __shfl_xor_sync(0xffffffffu, lo[i].y, o));
      add_to(hi[i], lo[i], h);
      lo[i] = add2(lo[i], l);
    }
  }
  if (scaled) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      hi[i] = mul2(hi[i], make_float2(kUp, kUp));
      lo[i] = mul2(lo[i], make_float2(kUp, kUp));
    }
  }
  // hi = the sum rounded to fp32, lo = the rest (none where hi is no number)
  float size = 0.0f;
  float h[8], l[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float a0 = i & 1 ? hi[i / 2].y : hi[i / 2].x, b0 = i & 1 ? lo[i / 2].y : lo[i / 2].x;
    h[i] = __fadd_rn(a0, b0);
    l[i] = __fsub_rn(b0, __fsub_rn(h[i], a0));
    if (!(fabsf(a0) <= FLT_MAX)) {
      h[i] = a0;
      l[i] = 0.0f;
    }
    size = fmaxf(size, fabsf(h[i]));
  }
  // (a maximum passes over what is no number)
  bool odd = !(size <= FLT_MAX);
#pragma unroll
  for (int i = 0; i < 8; ++i) odd = odd || h[i] != h[i];
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) size = fmaxf(size, __shfl_xor_sync(0xffffffffu, size, o));
  {   // the length of the sums, and a little more
    const float up = scale_up(size);
    float squares = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float y = __fmul_rn(h[i], up);
      squares = __fmaf_rn(y, y, squares);
    }
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) squares = __fadd_rn(squares, __shfl_xor_sync(0xffffffffu, squares, o));
    const float length = __fmul_rn(__fmul_rn(__fsqrt_rn(squares), 1.0f + 0x1p-18f), scale_down(size));
    size = fmaxf(size, length);
  }
  if (__any_sync(0xffffffffu, odd || !(size <= FLT_MAX))) size = INFINITY;
  const int64_t rows = a.sums.rows[t], at = static_cast<int64_t>(head) * rows + r;
  if (lane == 0) a.sums.size[t][at] = size;
  if (lane < kLanes) {
    float4* const hd = reinterpret_cast<float4*>(a.sums.hi[t] + at * HD) + 2 * c;
    float4* const ld4 = reinterpret_cast<float4*>(a.sums.lo[t] + at * HD) + 2 * c;
    hd[0] = make_float4(h[0], h[1], h[2], h[3]);
    hd[1] = make_float4(h[4], h[5], h[6], h[7]);
    ld4[0] = make_float4(l[0], l[1], l[2], l[3]);
    ld4[1] = make_float4(l[4], l[5], l[6], l[7]);
    if (t) {
      const float s = scale_up(size <= FLT_MAX ? size : 1.0f);
      uint4* const to = a.sums.parts + (at / 8 * (HD / 16) + c / 2) * 32 + at % 8 * 4 + c % 2 * 2;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint4 w;
        halves_of(make_float2(h[4 * i], h[4 * i + 1]), s, w.x, w.z);
        halves_of(make_float2(h[4 * i + 2], h[4 * i + 3]), s, w.y, w.w);
        to[i] = w;
      }
    }
  }
}

// ---------------------------------------------------------------------------- score

// R = 16: 256 threads a CTA, three CTAs an SM.  R = 32: 512, one.
template <int R>
constexpr int kScoreThreads = R <= 16 ? 256 : 512;
constexpr int kRows = 16;         // query blocks of a CTA at most: the rows of a product
// A row of scores begins so much past a multiple of 32 words: the eight rows that a warp stores to are in other banks.
constexpr int kRowPad = 8;
__host__ __device__ constexpr int width_of(int candidates) { return (candidates + 31) / 32 * 32 + kRowPad; }
// Scores that a CTA holds: 16 query blocks against 1,024 key blocks, or fewer against more.
constexpr int kScores = kRows * width_of(1024);
static_assert(width_of(static_cast<int>(kNearBlocks) + 1) <= kScores, "one query block against so many");

struct ScoreArgs {
  BlockShape s;
  Sums sums;
  int shift_q, shift_k;
  int rows;          // query blocks of a CTA
  int first;
  int32_t* blocks;
  float* scores;     // or nullptr
};

// A float's place in the order of all, as an unsigned number; no number is the lowest.
__device__ __forceinline__ uint32_t order_of_number(float x) {
  const uint32_t u = __float_as_uint(__fadd_rn(x, 0.0f));   // (-0 counts as 0)
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ uint32_t order_of(float x) { return x != x ? 0u : order_of_number(x); }
__device__ __forceinline__ float value_of(uint32_t order) {
  return __uint_as_float(order & 0x80000000u ? order & 0x7fffffffu : ~order);
}

// A query block's orders as the lanes of a warp have them, that of key block 32 r + lane in round r: in R
// registers, or (R = 0) in shared memory.
template <int R>
struct Orders {
  uint32_t held[R > 0 ? R : 1];
  uint32_t* at;
  int count;
  template <typename F>
  __device__ __forceinline__ void each(F f) {
    const int lane = threadIdx.x & 31;
    if constexpr (R > 0) {
#pragma unroll
      for (int r = 0; r < R; ++r) f(32 * r + lane, held[r]);
    } else {
      for (int j = lane; j < count; j += 32) f(j, at[j]);
    }
  }
  // each, in step: all lanes call f in every round
  template <typename F>
  __device__ __forceinline__ void in_step(F f) {
    const int lane = threadIdx.x & 31;
    if constexpr (R > 0) {
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (32 * r < count) f(32 * r + lane, held[r]);
    } else {
      for (int j = lane; j < count + lane; j += 32) {
        uint32_t x = j < count ? at[j] : 0u;
        f(j, x);
        if (j < count) at[j] = x;
      }
    }
  }
};

// Where a row is cut: `border` is the n-th highest of its orders (0 if fewer than n are above 0), `next` the
// highest that is not among the n, border itself where more than those have it (`tied`: then `above` are higher).
struct Cut {
  uint32_t border, next;
  bool tied;
  int above;
};

// Rounds of counting what is at least some value: the first ones at the place that normally distributed scores of
// the row's mean and deviation would have it, corrected by what was counted (four for 510 such scores, where
// halves of the interval take nine), then halves of the interval of values, at last of orders.  Whole warp.
template <int R>
__device__ __forceinline__ Cut cut_at(Orders<R>& row, int n) {
  uint32_t lowest = 0xffffffffu, highest = 0u;
  int any = 0, over = 0;   // above 0; of the highest order, which is no score
  float sum = 0.0f, squares = 0.0f;
  row.each([&](int, uint32_t x) {
    any += x != 0u;
    over += x == 0xffffffffu;
    lowest = min(lowest, x - 1u);   // (0 last)
    highest = max(highest, x);
    const float v = x + 1u > 1u ? value_of(x) : 0.0f;
    sum = __fadd_rn(sum, v);
    squares = __fmaf_rn(v, v, squares);
  });
  any = __reduce_add_sync(0xffffffffu, any);
  if (any < n) return {0u, 0u, true, any};
  over = __reduce_add_sync(0xffffffffu, over);
  uint32_t lo = __reduce_min_sync(0xffffffffu, lowest) + 1u, hi = __reduce_max_sync(0xffffffffu, highest);
  // at least n are >= lo, fewer than n are > hi
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, o));
    squares = __fadd_rn(squares, __shfl_xor_sync(0xffffffffu, squares, o));
  }
  const float per = __fdividef(1.0f, static_cast<float>(max(any - over, 1))), mean = __fmul_rn(sum, per);
  const float deviation = sqrtf(fmaxf(__fmaf_rn(-mean, mean, __fmul_rn(squares, per)), 0.0f));
  float guess;   // (the normal quantile to 3e-3: C. Hastings, "Approximations for Digital Computers", 1955)
  {
    const float share = __fmul_rn(static_cast<float>(n - over), per), tail = fminf(share, __fsub_rn(1.0f, share));
    const float r = sqrtf(__fmul_rn(-2.0f, __logf(fmaxf(tail, 1e-6f))));
    const float z = __fsub_rn(r, __fdividef(__fmaf_rn(0.27061f, r, 2.30753f),
                                            __fmaf_rn(__fmaf_rn(0.04481f, r, 0.99229f), r, 1.0f)));
    guess = __fmaf_rn(share < 0.5f ? z : -z, deviation, mean);
  }
  for (int round = 0; lo < hi; ++round) {
    uint32_t mid = lo + (hi - lo) / 2 + 1;
    if (round < 24) {
      const uint32_t at = order_of(round < 6 ? guess : __fmul_rn(0.5f, __fadd_rn(value_of(lo), value_of(hi))));
      if (at > lo && at <= hi) mid = at;
    }
    int mine = 0;
    row.each([&](int, uint32_t x) { mine += x >= mid; });
    const int got = __reduce_add_sync(0xffffffffu, mine);
    if (got == n) {   // exactly these: the lowest of them, and the highest of the others
      uint32_t least = 0xffffffffu, most = 0u;
      row.each([&](int, uint32_t x) {
        least = min(least, x >= mid ? x : 0xffffffffu);
        most = max(most, x >= mid ? 0u : x);
      });
      return {__reduce_min_sync(0xffffffffu, least), __reduce_max_sync(0xffffffffu, most), false, 0};
    }
    if (got < n) {
      hi = mid - 1;
    } else {
      lo = mid;
    }
    if (round < 5) {   // a score more is sqrt(2 pi) e^(z^2 / 2) deviations over the scores further down
      const float z = __fdividef(__fsub_rn(guess, mean), deviation);
      const float step = __fmul_rn(__fmul_rn(2.5066f * per, deviation), __expf(fminf(__fmul_rn(0.5f * z, z), 20.0f)));
      guess = __fmaf_rn(static_cast<float>(got - n), step, guess);
    }
  }
  int more = 0;
  row.each([&](int, uint32_t x) { more += x > lo; });
  return {lo, lo, true, static_cast<int>(__reduce_add_sync(0xffffffffu, more))};
}

struct RowPlace {
  BlockPlace block;
  int candidates;    // key blocks that may be chosen: the first of them
  int own;           // those from here on always are (causal)
  float delta;       // how far a score may be off
};

// One query block's choice among the first p.candidates key blocks, whose scores' orders are at `scored`.
// `q_at`, `k_at`: where its sums and those of its sequence's key blocks begin in a.sums; `len`: keys.  Whole warp.
template <int HD, int R>
__device__ __forceinline__ void choose(const ScoreArgs& a, const RowPlace& p, uint32_t* scored, int64_t q_at,
                                       int64_t k_at, int64_t len, int64_t list) {
  const int lane = threadIdx.x & 31;
  const int m = p.candidates, top = a.s.top;
  auto kept = [&](int j) { return j < a.first || j >= p.own; };
  Orders<R> row;
  row.at = scored;
  row.count = m;
  if constexpr (R > 0) {   // those that are always chosen stand above all, those past m below
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int j = 32 * r + lane;
      const uint32_t x = scored[j < m ? j : 0];
      row.held[r] = j >= m ? 0u : kept(j) ? 0xffffffffu : x;
    }
  } else {
    row.in_step([&](int j, uint32_t& x) {
      if (kept(j)) x = 0xffffffffu;
    });
    __syncwarp();
  }
  // The score of key block j from hi + lo, less `from`: a lane has 4 or 2 dimensions.  In pairs of fp32, whose
  // products and sums keep their rounding errors (T. J. Dekker, "A floating-point technique for extending the
  // available precision", Numer. Math. 18, 1971), as far as those cannot underflow; else in fp64, of which an
  // SM does two a clock.  (The worst, 65,280 tokens of equal blocks, all of which tie: 4.1 ms.)
  constexpr int kEach = HD / 32;
  float qh[kEach], ql[kEach];
  bool has_q = false;
  const bool pairs = p.delta > 0x1p-80f && p.delta < 0x1p80f;
  auto exact = [&](int j, float from) {
    if (!has_q) {
#pragma unroll
      for (int z = 0; z < kEach; ++z) {
        qh[z] = a.sums.hi[0][q_at + lane * kEach + z];
        ql[z] = a.sums.lo[0][q_at + lane * kEach + z];
      }
      has_q = true;
    }
    const int64_t at = k_at + static_cast<int64_t>(j) * HD + lane * kEach;
    const int64_t left = len - (static_cast<int64_t>(j) << a.shift_k);
    const int keys = left < a.s.block_k ? static_cast<int>(left) : a.s.block_k;
    if (pairs) {
      float s = 0.0f, rest = 0.0f;
      auto add = [&](float x) {   // s + rest += x
        const float sum = __fadd_rn(s, x), y = __fsub_rn(sum, s);
        rest = __fadd_rn(rest, __fadd_rn(__fsub_rn(s, __fsub_rn(sum, y)), __fsub_rn(x, y)));
        s = sum;
      };
#pragma unroll
      for (int z = 0; z < kEach; ++z) {
        const float kh = a.sums.hi[1][at + z], kl = a.sums.lo[1][at + z];
        const float product = __fmul_rn(qh[z], kh);
        rest = __fadd_rn(rest, __fadd_rn(__fmaf_rn(qh[z], kh, -product), __fmaf_rn(qh[z], kl, __fmul_rn(ql[z], kh))));
        add(product);
      }
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) {
        const float other = __shfl_xor_sync(0xffffffffu, s, o), its = __shfl_xor_sync(0xffffffffu, rest, o);
        rest = __fadd_rn(rest, its);
        add(other);
      }
      const float n = static_cast<float>(keys), mean = __fdiv_rn(s, n);
      if (!(fabsf(mean) <= FLT_MAX)) return __fsub_rn(mean, from);   // (an infinity has no rest)
      return __fadd_rn(__fsub_rn(mean, from), __fdiv_rn(__fadd_rn(__fmaf_rn(-mean, n, s), rest), n));
    }
    double sum = 0.0;
#pragma unroll
    for (int z = 0; z < kEach; ++z)
      sum = fma(static_cast<double>(qh[z]) + static_cast<double>(ql[z]),
                static_cast<double>(a.sums.hi[1][at + z]) + static_cast<double>(a.sums.lo[1][at + z]), sum);
#pragma unroll
    for (int z = 16; z >= 1; z >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, z);
    return static_cast<float>(sum / static_cast<double>(keys) - static_cast<double>(from));
  };

  Cut cut{0u, 0u, false, 0};   // all at least at the border are chosen (tied: all above it, and the first of those at it)
  if (m > top) {
    cut = cut_at(row, top);
    const float t = value_of(cut.border), reach = __fmul_rn(p.delta, 2.0f);
    if (cut.border != 0u && cut.border != 0xffffffffu && cut.next != 0u && reach > 0.0f && reach <= FLT_MAX &&
        __fsub_rn(t, value_of(cut.next)) <= reach) {
      // Those within reach of the border compete by their exact scores (less t, so that fp32 holds them to
      // 2^-24 of delta) for the places that those above leave; what is beyond reach keeps its side.
      auto sort_out = [&](uint32_t& x) {   // whether it is within reach; else above or below all
        const bool may = x != 0u && x != 0xffffffffu;
        const float from_t = may ? __fsub_rn(value_of(x), t) : 0.0f;
        const bool close = may && fabsf(from_t) <= reach;
        if (may && !close) x = from_t > reach ? 0xffffffffu : 0u;
        return close;
      };
      if constexpr (R > 0) {
        uint32_t near = 0u;   // a bit for each round
#pragma unroll
        for (int r = 0; r < R; ++r) near |= static_cast<uint32_t>(sort_out(row.held[r])) << r;
        for (uint32_t lanes; (lanes = __ballot_sync(0xffffffffu, near != 0u)) != 0u;) {
          const int i = __ffs(lanes) - 1, r = __shfl_sync(0xffffffffu, __ffs(near) - 1, i);
          const uint32_t x = order_of(exact(32 * r + i, t));
          if (lane != i) continue;
          near &= near - 1;
#pragma unroll
          for (int z = 0; z < R; ++z)
            if (z == r) row.held[z] = x;
        }
      } else {
        row.in_step([&](int j, uint32_t& x) {
          uint32_t todo = __ballot_sync(0xffffffffu, sort_out(x));
          while (todo) {
            const int i = __ffs(todo) - 1;
            todo &= todo - 1;
            const float s = exact(j - lane + i, t);
            if (lane == i) x = order_of(s);
          }
        });
      }
      __syncwarp();
      cut = cut_at(row, top);
    }
  }
  int written = 0, ties = cut.tied ? top - cut.above : m;   // places; of those at the border
  const uint32_t before = (1u << lane) - 1u;
  const float rows_f = static_cast<float>(p.block.rows) * static_cast<float>(a.s.heads / a.s.kv_heads);
  int32_t* const blocks = a.blocks + list;
  float* const scores = a.scores != nullptr ? a.scores + list : nullptr;
  auto is_chosen = [&](int j, uint32_t x) {
    bool in = j < m && x >= cut.border;
    if (cut.tied) {
      const uint32_t at_border = __ballot_sync(0xffffffffu, j < m && x == cut.border);
      in = in && (x > cut.border || __popc(at_border & before) < ties);
      ties -= __popc(at_border);
    }
    return in;
  };
  if constexpr (R > 0) {
    // Which are chosen, a bit for each round; lane r has round r's lanes, and how many were chosen before.  Then
    // each lane writes its own: two of 32 rounds' bits, mostly.
    static_assert(R <= 32, "a lane for each round");
    const float per_row = __fdiv_rn(1.0f, rows_f);
    uint32_t mine = 0u, lanes = 0u;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (32 * r >= m) break;   // (uniform)
      const bool in = is_chosen(32 * r + lane, row.held[r]);
      const uint32_t all = __ballot_sync(0xffffffffu, in);
      if (lane == r) lanes = all;
      mine |= static_cast<uint32_t>(in) << r;
    }
    int upto = __popc(lanes);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    written = __shfl_sync(0xffffffffu, upto, 31);
    upto -= __popc(lanes);
    while (__any_sync(0xffffffffu, mine != 0u)) {
      const int r = mine != 0u ? __ffs(mine) - 1 : 0;
      const int place = __shfl_sync(0xffffffffu, upto, r) + __popc(__shfl_sync(0xffffffffu, lanes, r) & before);
      if (mine != 0u && place < top) {
        blocks[place] = 32 * r + lane;
        if (scores != nullptr) scores[place] = __fmul_rn(value_of(scored[32 * r + lane]), per_row);
      }
      mine &= mine - 1u;
    }
  } else {
    row.in_step([&](int j, uint32_t& x) {
      const bool in = is_chosen(j, x);
      uint32_t chosen = __ballot_sync(0xffffffffu, in);
      const int place = written + __popc(chosen & before);
      written += __popc(chosen);
      if (in && place < top) blocks[place] = j;
      while (scores != nullptr && chosen) {   // (the scores are no longer there)
        const int i = __ffs(chosen) - 1;
        chosen &= chosen - 1;
        const float s = exact(j - lane + i, 0.0f);
        if (lane == i && place < top) scores[place] = __fdiv_rn(s, rows_f);
      }
    });
  }
  for (int place = written + lane; place < top; place += 32) {
    a.blocks[list + place] = -1;
    if (a.scores != nullptr) a.scores[list + place] = -INFINITY;
  }
}

// acc += A B: 16 query blocks by 8 key blocks over 16 dimensions.
__device__ __forceinline__ void product(float (&acc)[4], const uint4& x, uint32_t y0, uint32_t y1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(acc[0]), "+f"(acc[1]), "+f"(acc[2]), "+f"(acc[3])
      : "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w), "r"(y0), "r"(y1));
}

// FAR: for calls where a sequence's scores may pass what a CTA holds, which are then in the workspace (an instance of its
// own: with both ways in one, 16 tokens took 47 us for 43).
template <int HD, int R, bool FAR>
__global__ void __launch_bounds__(kScoreThreads<R>, R <= 16 ? 3 : 1) score_kernel(const __grid_constant__ ScoreArgs a) {
  constexpr int kThreads = kScoreThreads<R>, kWarps = kThreads / 32;
  extern __shared__ __align__(16) uint32_t smem[];
  constexpr int kSteps = HD / 16;
  uint4* const q_parts = reinterpret_cast<uint4*>(smem);   // [step][first, second][lane]
  uint32_t* const scored = smem + kSteps * 2 * 32 * 4;     // orders [rows of a pass][width]
  __shared__ RowPlace places[kRows];
  __shared__ float most_k;
  __shared__ int odd;          // some sums are no numbers
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t lists = a.sums.rows[0], kb_rows = a.sums.rows[1];
  const int64_t chunks = (lists + a.rows - 1) / a.rows;
  // (a CTA's only one, but where it has a row of the workspace)
  int64_t block = blockIdx.x;
  do {
    const int head = static_cast<int>(block / chunks);
    const int64_t r0 = (block - head * chunks) * a.rows;
    const int rows = static_cast<int>(lists - r0 < a.rows ? lists - r0 : a.rows);

    // (the lists of rows are older than the sums: they are looked at before those are there)
    if (threadIdx.x < rows) {
      RowPlace p{};
      p.block = block_at(a.s.cu_q, a.s.batch, a.s.rows_q, a.shift_q, r0 + threadIdx.x);
      if (p.block.rows > 0) {
        const int b = p.block.sequence;
        const int64_t n = rows_of(a.s.cu_q, b, a.s.rows_q), len = rows_of(a.s.cu_k, b, a.s.rows_k);
        const int64_t from = len - n + (static_cast<int64_t>(p.block.index) << a.shift_q);   // its first query's position
        int64_t end = len;
        if (a.s.causal && from + p.block.rows < end) end = from + p.block.rows < 0 ? 0 : from + p.block.rows;
        p.candidates = static_cast<int>((end + (int64_t{1} << a.shift_k) - 1) >> a.shift_k);
        p.own = !a.s.causal ? p.candidates : from < 0 ? 0 : static_cast<int>(from >> a.shift_k);
      }
      places[threadIdx.x] = p;
    }
    if (threadIdx.x == 0) {
      most_k = 0.0f;
      odd = 0;
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");   // the sums are written
    __syncthreads();

    for (int seg = 0; seg < rows;) {
      // rows of one sequence, as many as the scores have room for
      const RowPlace first = places[seg];
      const bool far = FAR && width_of(first.candidates) > kScores;   // (one query block, see the loop below)
      uint32_t* const far_row = a.sums.far + blockIdx.x * a.sums.far_row;
      int most = first.candidates, n = 1, width = width_of(most);
      while (seg + n < rows && first.block.rows > 0 && places[seg + n].block.rows > 0 &&
             places[seg + n].block.sequence == first.block.sequence) {
        const int other = max(places[seg + n].candidates, most);
        const int w = width_of(other);
        if ((n + 1) * w > kScores) break;
        most = other;
        width = w;
        ++n;
      }
      const int b = first.block.sequence;
      const int64_t q_at = (static_cast<int64_t>(head) * lists + r0 + seg) * HD;
      int64_t k_at = 0, len = 0;
      if (most > 0) {
        const int64_t kb0 = (a.s.cu_k[b] >> a.shift_k) + static_cast<int64_t>(b);   // the sequence's key block rows
        len = rows_of(a.s.cu_k, b, a.s.rows_k);
        const int64_t k_row = static_cast<int64_t>(head) * kb_rows + kb0;   // among all heads'
        k_at = k_row * HD;
        const float* const k_size = a.sums.size[1] + k_row;
        const float* const q_size = a.sums.size[0] + static_cast<int64_t>(head) * lists + r0 + seg;
        auto keys_of = [&](int j) {
          const int64_t left = len - (static_cast<int64_t>(j) << a.shift_k);
          return static_cast<float>(left < a.s.block_k ? left : a.s.block_k);
        };
        {
          float m = 0.0f;
          for (int i = threadIdx.x; i < most; i += kThreads) {
            const float size = k_size[i];
            if (size <= FLT_MAX) {
              m = fmaxf(m, __fdiv_rn(size, keys_of(i)));
            } else {
              odd = 1;
            }
          }
          if (threadIdx.x < n && !(q_size[threadIdx.x] <= FLT_MAX)) odd = 1;
#pragma unroll
          for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
          if (lane == 0) atomicMax(reinterpret_cast<int*>(&most_k), __float_as_int(m));   // (none is negative)
        }
        // The products: a lane's operand of q is two query blocks (lane / 4 and 8 on), four of 16 dimensions each, which
        // the warps make together; a warp takes every eighth group of 8 key blocks.
        float q_down[2];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int block = lane / 4 + 8 * y;
          const float size = block < n ? q_size[block] : INFINITY;
          const bool there = size <= FLT_MAX;
          const float s = scale_up(there ? size : 1.0f);
          q_down[y] = scale_down(there ? size : 1.0f);
          for (int z = warp; z < kSteps; z += kWarps) {
            const float4 v = there ? reinterpret_cast<const float4*>(a.sums.hi[0] + q_at + block * HD)[4 * z + lane % 4]
                                   : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            uint32_t* const to = reinterpret_cast<uint32_t*>(q_parts + 2 * z * 32 + lane) + y;
            halves_of(make_float2(v.x, v.y), s, to[0], to[32 * 4]);
            halves_of(make_float2(v.z, v.w), s, to[2], to[32 * 4 + 2]);
          }
        }
        const int last = static_cast<int>((len - 1) >> a.shift_k);   // the sequence's last block, which may be shorter
        const float per_full = __fdiv_rn(1.0f, static_cast<float>(a.s.block_k)), per_last = __fdiv_rn(1.0f, keys_of(last));
        const int64_t group0 = k_row / 8;
        const int before = static_cast<int>(k_row - group0 * 8);   // rows of other sequences in the first group
        const int groups = (before + most + 7) / 8;
        // Steps whose operands are asked for before the group is begun: half, where there are registers for them.
        constexpr int kAhead = R > 16 ? kSteps / 2 : 0;
        const uint4* from = a.sums.parts + (group0 + warp) * (kSteps * 32) + lane;
        uint4 k[kSteps];
        if (warp < groups) {
#pragma unroll
          for (int z = 0; z < kAhead; ++z) k[z] = from[z * 32];
        }
        __syncthreads();
        uint32_t* const my_scores = scored + lane / 4 * width;
        for (int g = warp; g < groups; g += kWarps) {
#pragma unroll
          for (int z = kAhead; z < kSteps; ++z) k[z] = from[z * 32];
          if (g + kWarps < groups) from += kWarps * kSteps * 32;
          const int j = 8 * g - before + lane % 4 * 2;
          float size[2];
#pragma unroll
          for (int x = 0; x < 2; ++x) size[x] = static_cast<uint32_t>(j + x) < static_cast<uint32_t>(most) ? k_size[j + x] : 0.0f;
          // (four sums, so that none is long: first parts of even and odd steps, the rest)
          float even[4] = {}, uneven[4] = {}, rest[4] = {}, other[4] = {};
#pragma unroll
          for (int z = 0; z < kSteps; ++z) {
            const uint4 first = q_parts[2 * z * 32 + lane], second = q_parts[(2 * z + 1) * 32 + lane];
            product(z & 1 ? uneven : even, first, k[z].x, k[z].y);
            product(rest, first, k[z].z, k[z].w);
            product(other, second, k[z].x, k[z].y);
            if (z < kAhead) k[z] = from[z * 32];   // (after the last group: any)
          }
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (static_cast<uint32_t>(j + x) >= static_cast<uint32_t>(most)) continue;
            const float per_key = j + x == last ? per_last : per_full, k_down = scale_down(size[x]);
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const int i = 2 * y + x;
              const float sum = __fadd_rn(__fadd_rn(even[i], uneven[i]), __fadd_rn(rest[i], other[i]));
              // (the smaller factor first: nothing is too large on the way that is not so at the end)
              const float s = __fmul_rn(__fmul_rn(__fmul_rn(sum, per_key), fminf(q_down[y], k_down)), fmaxf(q_down[y], k_down));
              if (lane / 4 + 8 * y >= n) continue;
              if (far) {
                far_row[j + x] = order_of_number(s);
              } else {
                my_scores[8 * y * width + j + x] = order_of_number(s);
              }
            }
          }
        }
        __syncthreads();
        if (odd) {   // scores with sums that are no numbers: as fp32 has them
          for (int i = threadIdx.x; i < n * most; i += kThreads) {
            const int y = i / most, j = i - y * most;
            if (q_size[y] <= FLT_MAX && k_size[j] <= FLT_MAX) continue;
            const float* const qv = a.sums.hi[0] + q_at + y * HD;
            const float* const kv = a.sums.hi[1] + k_at + static_cast<int64_t>(j) * HD;
            float s = 0.0f;
            for (int d = 0; d < HD; ++d) s = __fmaf_rn(qv[d], kv[d], s);
            if (far) {
              far_row[j] = order_of(__fdiv_rn(s, keys_of(j)));
            } else {
              scored[y * width + j] = order_of(__fdiv_rn(s, keys_of(j)));
            }
          }
        }
        if (threadIdx.x < n) {   // (0: queries or keys of zeros, whose scores are exact)
          const float q_sum = q_size[threadIdx.x];
          // (2^-145: what scaled sums below 2^-112 may lose)
          const float off = fmaxf(fmaxf(__fmul_rn(q_sum, fmaxf(__fmul_rn(most_k, 0x1.6p-17f), 0x1p-145f)),
                                        __fmul_rn(most_k, 0x1p-145f)), 0x1p-140f);
          places[seg + threadIdx.x].delta = q_sum == 0.0f || most_k == 0.0f ? 0.0f : off;
        }
        __syncthreads();
      }
      if (threadIdx.x == 0) {
        most_k = 0.0f;
        odd = 0;
      }
      // the choice: a warp for each query block
      for (int y = warp; y < n; y += kWarps) {
        const RowPlace p = places[seg + y];
        const int64_t list = (static_cast<int64_t>(head) * lists + r0 + seg + y) * a.s.top;
        uint32_t* const row = scored + y * width;
        const int64_t q_row = q_at + static_cast<int64_t>(y) * HD;
        if (far) {
          choose<HD, 0>(a, p, far_row, q_row, k_at, len, list);
        } else if (p.candidates <= 512) {
          choose<HD, 16>(a, p, row, q_row, k_at, len, list);
        } else if (R > 16 && p.candidates <= 1024) {
          choose<HD, (R > 16 ? 32 : 0)>(a, p, row, q_row, k_at, len, list);
        } else {
          choose<HD, 0>(a, p, row, q_row, k_at, len, list);
        }
      }
      seg += n;
      __syncthreads();   // the scores, and places' deltas, are overwritten
    }
    block += gridDim.x;
  } while (FAR && block < chunks * a.s.kv_heads);
}

// CTAs of the scores' kernel that the device holds.
template <int HD>
constexpr int kScoreSmem = HD / 16 * 2 * 512 + kScores * 4;
template <int HD, int R, bool FAR = false>
cudaError_t resident(int* blocks) {
  return persistent_blocks(reinterpret_cast<const void*>(&score_kernel<HD, R, FAR>), kScoreThreads<R>, kScoreSmem<HD>,
                           int64_t{1} << 30, blocks);
}

template <int HD, int R, bool FAR = false>
cudaError_t launch_score(ScoreArgs score, cudaStream_t stream) {
  int blocks = 0;
  cudaError_t err = resident<HD, R, FAR>(&blocks);
  if (err != cudaSuccess) return err;
  // query blocks of a CTA: 16, or fewer where all CTAs run at once all the same
  const int64_t rows = (score.sums.rows[0] * score.s.kv_heads + blocks - 1) / blocks;
  score.rows = static_cast<int>(rows < 1 ? 1 : rows > kRows ? kRows : rows);
  int64_t grid = (score.sums.rows[0] + score.rows - 1) / score.rows * score.s.kv_heads;
  if (FAR && grid > kFarRows) grid = kFarRows;
  cudaLaunchConfig_t config{};
  config.gridDim = dim3(static_cast<unsigned>(grid));
  config.blockDim = dim3(kScoreThreads<R>);
  config.dynamicSmemBytes = kScoreSmem<HD>;
  config.stream = stream;
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  config.attrs = &early;
  config.numAttrs = 1;
  return cudaLaunchKernelEx(&config, score_kernel<HD, R, FAR>, score);
}

template <int HD>
cudaError_t launch(const PoolArgs& pool, const ScoreArgs& score, cudaStream_t stream) {
  const int64_t warps = (pool.sums.rows[0] + pool.sums.rows[1]) * pool.kv_heads;
  const int64_t pool_blocks = (warps + kPoolThreads / 32 - 1) / (kPoolThreads / 32);
  int single = 0;
  cudaError_t err = resident<HD, 32>(&single);
  if (err != cudaSuccess) return err;
  pool_kernel<HD><<<static_cast<unsigned>(pool_blocks), kPoolThreads, 0, stream>>>(pool);
  if ((err = cudaGetLastError()) != cudaSuccess) return err;
  // Many lists: three CTAs an SM, whose warps hold 512 scores, which is enough where sequences have so many key
  // blocks on average (65,280 tokens 425 us, with the other instance 485).  Else one of twice the threads, whose warps
  // hold 1,024 and ask for operands ahead (16 single tokens 40.5 us, with the first 43.2; 4 chunks 51.5 and 51.7).
  const int64_t longest = (score.s.rows_k + score.s.block_k - 1) / score.s.block_k;
  const bool many = score.sums.rows[0] * score.s.kv_heads >= int64_t{2} * single * kRows;
  if (score.sums.far != nullptr) return launch_score<HD, 32, true>(score, stream);
  return many && longest <= 512 * static_cast<int64_t>(score.s.batch) ? launch_score<HD, 16>(score, stream)
                                                               : launch_score<HD, 32>(score, stream);
}

}  // namespace

cudaError_t launch_select_blocks(const BlockShape& s, const uint16_t* q, int64_t ld_q, const uint16_t* k, int64_t ld_k,
                                 int first, int32_t* blocks, float* scores, uint8_t* workspace, cudaStream_t stream) {
  PoolArgs pool{};
  pool.x[0] = q;
  pool.x[1] = k;
  pool.ld[0] = ld_q;
  pool.ld[1] = ld_k;
  pool.cu[0] = s.cu_q;
  pool.cu[1] = s.cu_k;
  pool.total[0] = s.rows_q;
  pool.total[1] = s.rows_k;
  pool.shift[0] = log2_of(s.block_q);
  pool.shift[1] = log2_of(s.block_k);
  pool.group[0] = s.heads / s.kv_heads;
  pool.group[1] = 1;
  pool.batch = s.batch;
  pool.kv_heads = s.kv_heads;
  pool.sums = carve(s, workspace);
  ScoreArgs score{};
  score.s = s;
  score.sums = pool.sums;
  score.shift_q = pool.shift[0];
  score.shift_k = pool.shift[1];
  score.first = first;
  score.blocks = blocks;
  score.scores = scores;
  return s.head_dim == 64 ? launch<64>(pool, score, stream) : launch<128>(pool, score, stream);
}

}  // namespace h3q
