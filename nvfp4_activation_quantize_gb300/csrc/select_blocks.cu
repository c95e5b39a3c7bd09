// select_blocks.cu -- the blocks of keys that each block of queries attends to.
//
// Score of query block i and key block j of a key head: (sum of the block's query rows, over the
// heads of the group) . (sum of the block's keys) / (keys of the block).  The `top` highest
// are kept; of equal ones those with the lowest numbers.
//
// Two kernels.
//   pool    sums the rows of each block of q and of k: every input byte is read once, which is
//           the bound (DRAM).  A sum is kept as hi + lo, two fp32 that hold 48 bits of it (D. E.
//           Knuth's two-sum, The Art of Computer Programming vol. 2, 4.2.2: the rounding error of
//           an fp32 addition is itself an fp32): seven packed additions a pair of values, half of what
//           the loads leave time for.
//   score   16 query blocks a CTA against all key blocks of their sequence: products of the hi
//           parts in fp32 (the lo parts are below their rounding), 8 x 4 scores a thread
//           from tiles in shared memory, then a warp per query block finds the top-th
//           highest score by bisection.
//
// What fp32 cannot tell apart is told apart in 64 bits: a score is off by at most
// delta = 2^-18 * sum|q_i| * max|k_i| (parts hi: 2 * 2^-24; chains of 16 fused products, and 8 sums of
// them: 24 * 2^-24; the mean: 2^-23; less than 64 * 2^-24 in all).  Where the top-th score is more
// than 2 delta above the next, the choice is the exact one.  Where it is not (one list in a hundred
// for unrelated blocks), the scores within 2 delta of it are formed again from hi + lo in fp64, and
// the places that are left go to the highest of those.
#include <cfloat>

#include "h3q_async.cuh"
#include "h3q_blocks.cuh"
#include "h3q_device.cuh"
#include "h3q_internal.h"

namespace h3q {
namespace {

// ---------------------------------------------------------------------------- pool

constexpr int kPoolThreads = 256;

// The workspace: hi and lo parts [kv_heads][block rows][head_dim] of q and of k, then for each block sum |q|
// and max |mean k|.
struct Sums {
  float* hi[2];
  float* lo[2];
  float* size[2];
  int64_t rows[2];   // block rows
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
  for (int t = 0; t < 2; ++t) {
    w.size[t] = at;
    at += w.rows[t] * s.kv_heads;
  }
  return w;
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

// (hi, lo) += x: hi + error = hi + x without rounding.
__device__ __forceinline__ void add_to(float2& hi, float2& lo, float2 x) {
  const float2 s = add2(hi, x);
  const float2 y = sub2(s, hi);
  lo = add2(lo, add2(sub2(hi, sub2(s, y)), sub2(x, y)));
  hi = s;
}

template <int HD>
__global__ void __launch_bounds__(kPoolThreads) pool_kernel(const __grid_constant__ PoolArgs a) {
  constexpr int kLanes8 = HD / 8;           // lanes of a row of a head, 8 values each
  constexpr int kRows = 32 / kLanes8;       // rows of a head that a load of the warp takes
  constexpr int kUnroll = 8;
  const int lane = threadIdx.x & 31;
  const int c = lane % kLanes8;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * (kPoolThreads / 32) + (threadIdx.x >> 5);
  int64_t r = unit / a.kv_heads;
  const int head = static_cast<int>(unit - r * a.kv_heads);
  if (r >= a.sums.rows[0] + a.sums.rows[1]) return;
  const int t = r >= a.sums.rows[0];
  if (t) r -= a.sums.rows[0];
  const BlockPlace p = block_at(a.cu[t], a.batch, a.total[t], a.shift[t], r);
  if (p.rows == 0) return;   // (never read)
  const int group = a.group[t], items = p.rows * group;   // rows of single heads
  const int64_t ld = a.ld[t];
  const uint16_t* const x = a.x[t] + p.row0 * ld + static_cast<int64_t>(head) * group * HD + c * 8;
  float2 hi[4], lo[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) hi[i] = lo[i] = make_float2(0.0f, 0.0f);
  for (int i0 = lane / kLanes8; i0 < items; i0 += kRows * kUnroll) {
    uint4 w[kUnroll];
#pragma unroll
    for (int n = 0; n < kUnroll; ++n) {
      const int i = i0 + n * kRows;
      w[n] = make_uint4(0u, 0u, 0u, 0u);
      if (i < items) {
        const int row = i / group;
        w[n] = load16_stream(x + row * ld + (i - row * group) * HD);
      }
    }
#pragma unroll
    for (int n = 0; n < kUnroll; ++n) {
      add_to(hi[0], lo[0], bf16x2_to_float2(w[n].x));
      add_to(hi[1], lo[1], bf16x2_to_float2(w[n].y));
      add_to(hi[2], lo[2], bf16x2_to_float2(w[n].z));
      add_to(hi[3], lo[3], bf16x2_to_float2(w[n].w));
    }
  }
  // the other rows' lanes
#pragma unroll
  for (int o = kLanes8; o < 32; o <<= 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 h = make_float2(__shfl_xor_sync(0xffffffffu, hi[i].x, o), __shfl_xor_sync(0xffffffffu, hi[i].y, o));
      const float2 l = make_float2(__shfl_xor_sync(0xffffffffu, lo[i].x, o), __shfl_xor_sync(0xffffffffu, lo[i].y, o));
      add_to(hi[i], lo[i], h);
      lo[i] = add2(lo[i], l);
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
    size = t ? fmaxf(size, fabsf(h[i])) : __fadd_rn(size, fabsf(h[i]));
  }
  if (t && !(size <= FLT_MAX)) size = 0.0f;   // (its scores are no numbers, or infinite, whatever fp32 makes of them)
#pragma unroll
  for (int o = 1; o < kLanes8; o <<= 1) {
    const float other = __shfl_xor_sync(0xffffffffu, size, o);
    size = t ? fmaxf(size, other) : __fadd_rn(size, other);
  }
  const int64_t at = static_cast<int64_t>(head) * a.sums.rows[t] + r;
  if (lane == 0) a.sums.size[t][at] = t ? __fdiv_rn(size, static_cast<float>(p.rows)) : size;
  if (lane < kLanes8) {
    float4* const hd = reinterpret_cast<float4*>(a.sums.hi[t] + at * HD + c * 8);
    float4* const ld4 = reinterpret_cast<float4*>(a.sums.lo[t] + at * HD + c * 8);
    hd[0] = make_float4(h[0], h[1], h[2], h[3]);
    hd[1] = make_float4(h[4], h[5], h[6], h[7]);
    ld4[0] = make_float4(l[0], l[1], l[2], l[3]);
    ld4[1] = make_float4(l[4], l[5], l[6], l[7]);
  }
}

// ---------------------------------------------------------------------------- score

constexpr int kThreads = 128;
constexpr int kRows = 16;         // query blocks of a CTA at most
constexpr int kTile = 256;        // key blocks of a tile,
constexpr int kDims = 16;         // and its dimensions
constexpr int kStride = kDims + 4;   // floats between a tile's rows: eight rows' 16 bytes meet in no bank
constexpr int kTileBytes = kTile * kStride * 4;
// Scores that a CTA holds: 16 query blocks against 256, 512 or 1,024 key blocks, or fewer against more (one
// against 16,384, see kMaxBlocks).
constexpr int kMostScores = kRows * 1024;

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
__device__ __forceinline__ uint32_t order_of(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(__fadd_rn(x, 0.0f));   // (-0 counts as 0)
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t order) {
  return __uint_as_float(order & 0x80000000u ? order & 0x7fffffffu : ~order);
}

// The n-th highest of the orders that `get` gives for 0 .. count - 1 (1 <= n <= the count of those above 0 or
// any), by bisection of the 32 bits; `above`: how many are higher.  Whole warp.
template <typename Get>
__device__ __forceinline__ uint32_t nth_highest(int count, int n, Get get, int& above) {
  const int lane = threadIdx.x & 31;
  uint32_t lowest = 0xffffffffu, highest = 0u;
  for (int i = lane; i < count; i += 32) {
    const uint32_t x = get(i);
    lowest = min(lowest, x);
    highest = max(highest, x);
  }
  uint32_t lo = __reduce_min_sync(0xffffffffu, lowest), hi = __reduce_max_sync(0xffffffffu, highest);
  // at least n are >= lo; fewer than n are > hi
  while (lo < hi) {
    const uint32_t mid = lo + (hi - lo) / 2 + 1;
    int mine = 0;
    for (int i = lane; i < count; i += 32) mine += get(i) >= mid;
    const int got = __reduce_add_sync(0xffffffffu, mine);
    if (got >= n) {
      lo = mid;
      if (got == n) {   // exactly these: the lowest of them
        uint32_t least = 0xffffffffu;
        for (int i = lane; i < count; i += 32) {
          const uint32_t x = get(i);
          if (x >= mid) least = min(least, x);
        }
        lo = __reduce_min_sync(0xffffffffu, least);
        break;
      }
    } else {
      hi = mid - 1;
    }
  }
  int mine = 0;
  for (int i = lane; i < count; i += 32) mine += get(i) > lo;
  above = __reduce_add_sync(0xffffffffu, mine);
  return lo;
}

struct RowPlace {
  BlockPlace block;
  int candidates;    // key blocks that may be chosen: the first of them
  int own;           // those from here on are (causal)
  float delta;       // how far a score may be off
};

template <int HD, int CAPACITY>
__global__ void __launch_bounds__(kThreads) score_kernel(const __grid_constant__ ScoreArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  float* const tiles = reinterpret_cast<float*>(smem);                        // two
  float* const q = reinterpret_cast<float*>(smem + 2 * kTileBytes);           // [kRows][HD]
  float* const scores = q + kRows * HD;                                       // [rows of a pass][width]
  uint32_t* const near_flags = reinterpret_cast<uint32_t*>(scores + CAPACITY);   // [rows of a pass][width / 32]
  __shared__ RowPlace places[kRows];
  __shared__ float most_k;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t lists = a.sums.rows[0], kb_rows = a.sums.rows[1];
  const int64_t chunks = (lists + a.rows - 1) / a.rows;
  const int head = static_cast<int>(blockIdx.x / chunks);
  const int64_t r0 = (blockIdx.x - head * chunks) * a.rows;
  const int rows = static_cast<int>(lists - r0 < a.rows ? lists - r0 : a.rows);

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
  __syncthreads();

  for (int seg = 0; seg < rows;) {
    // rows of one sequence, as many as the scores have room for
    const RowPlace head_place = places[seg];
    int most = head_place.candidates, n = 1;
    const int width_of_one = (most + kTile - 1) / kTile * kTile;
    int width = width_of_one;
    while (seg + n < rows && places[seg + n].block.rows > 0 && head_place.block.rows > 0 &&
           places[seg + n].block.sequence == head_place.block.sequence) {
      const int other = places[seg + n].candidates > most ? places[seg + n].candidates : most;
      const int w = (other + kTile - 1) / kTile * kTile;
      if ((n + 1) * w > CAPACITY) break;
      most = other;
      width = w;
      ++n;
    }
    if (most > 0) {
      const int b = head_place.block.sequence;
      const int64_t kb0 = (a.s.cu_k[b] >> a.shift_k) + static_cast<int64_t>(b);   // the sequence's key block rows
      const int64_t len = rows_of(a.s.cu_k, b, a.s.rows_k);
      const float* const k_hi = a.sums.hi[1] + (static_cast<int64_t>(head) * kb_rows + kb0) * HD;
      const float* const k_size = a.sums.size[1] + static_cast<int64_t>(head) * kb_rows + kb0;
      const float* const q_hi = a.sums.hi[0] + (static_cast<int64_t>(head) * lists + r0 + seg) * HD;
      const float* const q_size = a.sums.size[0] + static_cast<int64_t>(head) * lists + r0 + seg;
      if (threadIdx.x == 0) most_k = 0.0f;
      for (int i = threadIdx.x; i < kRows * HD / 4; i += kThreads) {
        const bool there = i / (HD / 4) < n;
        reinterpret_cast<float4*>(q)[i] =
            there ? reinterpret_cast<const float4*>(q_hi)[i] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      }
      __syncthreads();
      {
        float m = 0.0f;
        for (int i = threadIdx.x; i < most; i += kThreads) m = fmaxf(m, k_size[i]);
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (lane == 0) atomicMax(reinterpret_cast<int*>(&most_k), __float_as_int(m));   // (none is negative)
      }

      // ---- scores: 16 query blocks by tiles of 256 key blocks, 16 dimensions at a time
      constexpr int kSteps = HD / kDims;
      const int steps = width / kTile * kSteps;
      auto fetch = [&](int step) {
        const int j0 = step / kSteps * kTile, d0 = step % kSteps * kDims;
        float* const to = tiles + (step & 1) * (kTileBytes / 4);
#pragma unroll
        for (int i = 0; i < kTile * kDims / 4 / kThreads; ++i) {
          const int piece = threadIdx.x + i * kThreads;
          const int j = piece / (kDims / 4), d = piece % (kDims / 4) * 4;
          const int from = j0 + j < most ? j0 + j : most - 1;   // (past the last: any)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to + j * kStride + d)),
                       "l"(k_hi + static_cast<int64_t>(from) * HD + d0 + d)
                       : "memory");
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      };
      // A thread's scores: query blocks 8 (warp / 2) .. + 7, key blocks (warp % 2) * 128 + lane + 32 x.
      const int q_first = warp / 2 * 8, k_first = warp % 2 * 128 + lane;
      float2 total[8][2];   // key blocks x = 0, 1 and 2, 3
      fetch(0);
      for (int step = 0; step < steps; ++step) {
        if (step + 1 < steps) {
          fetch(step + 1);
          asm volatile("cp.async.wait_group 1;" ::: "memory");
        } else {
          asm volatile("cp.async.wait_group 0;" ::: "memory");
        }
        __syncthreads();
        const float* const k = tiles + (step & 1) * (kTileBytes / 4) + k_first * kStride;
        const float* const qd = q + q_first * HD + step % kSteps * kDims;
        float2 part[8][2];
#pragma unroll
        for (int d = 0; d < kDims; d += 4) {
          float4 kv[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) kv[x] = *reinterpret_cast<const float4*>(k + 32 * x * kStride + d);
#pragma unroll
          for (int y = 0; y < 8; ++y) {
            const float4 qv = *reinterpret_cast<const float4*>(qd + y * HD + d);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const float4 k0 = kv[2 * x], k1 = kv[2 * x + 1];
              float2 p = d == 0 ? mul2(make_float2(qv.x, qv.x), make_float2(k0.x, k1.x))
                                : fma2(make_float2(qv.x, qv.x), make_float2(k0.x, k1.x), part[y][x]);
              p = fma2(make_float2(qv.y, qv.y), make_float2(k0.y, k1.y), p);
              p = fma2(make_float2(qv.z, qv.z), make_float2(k0.z, k1.z), p);
              part[y][x] = fma2(make_float2(qv.w, qv.w), make_float2(k0.w, k1.w), p);
            }
          }
        }
        const bool begins = step % kSteps == 0;
#pragma unroll
        for (int y = 0; y < 8; ++y)
#pragma unroll
          for (int x = 0; x < 2; ++x) total[y][x] = begins ? part[y][x] : add2(total[y][x], part[y][x]);
        if (step % kSteps == kSteps - 1) {
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int j = step / kSteps * kTile + k_first + 32 * x;
            const int64_t left = len - (static_cast<int64_t>(j) << a.shift_k);
            const int keys = left < 1 ? 1 : left < a.s.block_k ? static_cast<int>(left) : a.s.block_k;
            const float per_key = __fdiv_rn(1.0f, static_cast<float>(keys));
#pragma unroll
            for (int y = 0; y < 8; ++y)
              if (q_first + y < n) {
                const float2 z = total[y][x / 2];
                scores[(q_first + y) * width + j] = __fmul_rn(x & 1 ? z.y : z.x, per_key);
              }
          }
        }
        __syncthreads();   // the tile may be filled again
      }
      if (threadIdx.x < n) places[seg + threadIdx.x].delta =
          fmaxf(__fmul_rn(__fmul_rn(q_size[threadIdx.x], most_k), 0x1p-18f), 0x1p-140f);
      __syncthreads();
    }

    // ---- the choice: a warp for each query block
    for (int y = warp; y < n; y += kThreads / 32) {
      const RowPlace p = places[seg + y];
      const int64_t list = (static_cast<int64_t>(head) * lists + r0 + seg + y) * a.s.top;
      float* const row = scores + y * width;
      uint32_t* const near = near_flags + y * (width / 32);
      const int m = p.block.rows > 0 ? p.candidates : 0, top = a.s.top;
      auto kept = [&](int j) { return j < a.first || j >= p.own; };
      auto order = [&](int j) { return kept(j) ? 0xffffffffu : order_of(row[j]); };
      uint32_t border = 0u;   // all above it are chosen, and the first `ties` of those at it
      int ties = m;
      bool again = false;     // those near the border are chosen by their exact scores
      if (m > top) {
        int above;
        border = nth_highest(m, top, order, above);
        ties = top - above;
        uint32_t next = 0u;   // the highest that would not be chosen
        int at_border = 0;
        for (int j = lane; j < m; j += 32) {
          const uint32_t x = order(j);
          at_border += x == border;
          if (x < border) next = max(next, x);
        }
        next = __reduce_add_sync(0xffffffffu, at_border) > ties ? border : __reduce_max_sync(0xffffffffu, next);
        const float t = value_of(border), below = next == 0u ? -INFINITY : value_of(next);
        const float reach = __fmul_rn(p.delta, 2.0f);
        again = border != 0xffffffffu && border != 0u && reach <= FLT_MAX && __fsub_rn(t, below) <= reach;
        if (again) {
          // The candidates within reach: their scores from hi + lo in 64 bits, less t (so that fp32 holds them
          // to 2^-24 of delta); they compete for the places that those above leave.
          const int b = p.block.sequence;
          const int64_t len = rows_of(a.s.cu_k, b, a.s.rows_k);
          const int64_t q_at = (static_cast<int64_t>(head) * lists + r0 + seg + y) * HD;
          const int64_t k_at = (static_cast<int64_t>(head) * kb_rows + (a.s.cu_k[b] >> a.shift_k) + b) * HD;
          constexpr int kEach = HD / 32;
          double qd[kEach];
#pragma unroll
          for (int i = 0; i < kEach; ++i)
            qd[i] = static_cast<double>(a.sums.hi[0][q_at + lane + 32 * i]) +
                    static_cast<double>(a.sums.lo[0][q_at + lane + 32 * i]);
          int higher = 0;
          for (int j0 = 0; j0 < m; j0 += 32) {
            const int j = j0 + lane;
            const float x = j < m ? row[j] : 0.0f;
            const bool over = j < m && (kept(j) || __fsub_rn(x, t) > reach);
            const bool close = j < m && !over && fabsf(__fsub_rn(x, t)) <= reach;
            higher += __popc(__ballot_sync(0xffffffffu, over));
            uint32_t todo = __ballot_sync(0xffffffffu, close);
            if (lane == 0) near[j0 / 32] = todo;
            while (todo) {
              const int i = __ffs(todo) - 1;
              todo &= todo - 1;
              const int64_t k_row = k_at + static_cast<int64_t>(j0 + i) * HD + lane;
              double sum = 0.0;
#pragma unroll
              for (int z = 0; z < kEach; ++z)
                sum = fma(qd[z], static_cast<double>(a.sums.hi[1][k_row + 32 * z]) +
                                     static_cast<double>(a.sums.lo[1][k_row + 32 * z]), sum);
#pragma unroll
              for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
              const int64_t left = len - (static_cast<int64_t>(j0 + i) << a.shift_k);
              sum = sum / static_cast<double>(left < a.s.block_k ? left : a.s.block_k) - static_cast<double>(t);
              if (lane == i) row[j] = static_cast<float>(sum);
            }
          }
          __syncwarp();
          const int places_left = top - higher;   // >= 1; those at t or above are either higher or among the near
          auto exact = [&](int j) { return near[j / 32] >> (j % 32) & 1u ? order_of(row[j]) : 0u; };
          int above_exact;
          const uint32_t line = nth_highest(m, places_left, exact, above_exact);
          int left_over = places_left - above_exact, written = 0;
          const float rows_f = static_cast<float>(p.block.rows) * static_cast<float>(a.s.heads / a.s.kv_heads);
          for (int j0 = 0; j0 < m; j0 += 32) {
            const int j = j0 + lane;
            const bool is_near = j < m && (near[j0 / 32] >> lane & 1u);
            const float x = j < m ? row[j] : 0.0f;
            const uint32_t e = is_near ? order_of(x) : 0u;
            const uint32_t at_line = __ballot_sync(0xffffffffu, is_near && e == line);
            const bool in = is_near ? e > line || (e == line && __popc(at_line & ((1u << lane) - 1u)) < left_over)
                                    : j < m && (kept(j) || __fsub_rn(x, t) > reach);
            left_over -= __popc(at_line);
            left_over = left_over < 0 ? 0 : left_over;
            const uint32_t chosen = __ballot_sync(0xffffffffu, in);
            const int place = written + __popc(chosen & ((1u << lane) - 1u));
            if (in && place < top) {
              a.blocks[list + place] = j;
              if (a.scores) a.scores[list + place] = __fdiv_rn(is_near ? __fadd_rn(t, x) : x, rows_f);
            }
            written += __popc(chosen);
          }
          continue;   // (top of them)
        }
      }
      int written = 0, tied = 0;
      const float rows_f = static_cast<float>(p.block.rows) * static_cast<float>(a.s.heads / a.s.kv_heads);
      for (int j0 = 0; j0 < m; j0 += 32) {
        const int j = j0 + lane;
        const uint32_t x = j < m ? order(j) : 0u;
        const uint32_t at = __ballot_sync(0xffffffffu, j < m && x == border);
        const bool in = j < m && (m <= top || x > border || (x == border && tied + __popc(at & ((1u << lane) - 1u)) < ties));
        tied += __popc(at);
        const uint32_t chosen = __ballot_sync(0xffffffffu, in);
        const int place = written + __popc(chosen & ((1u << lane) - 1u));
        if (in && place < top) {
          a.blocks[list + place] = j;
          if (a.scores) a.scores[list + place] = __fdiv_rn(row[j], rows_f);
        }
        written += __popc(chosen);
      }
      for (int place = written + lane; place < top; place += 32) {
        a.blocks[list + place] = -1;
        if (a.scores) a.scores[list + place] = -INFINITY;
      }
    }
    seg += n;
    __syncthreads();   // the scores, and places' deltas, are overwritten
  }
}

template <int HD, int CAPACITY>
cudaError_t launch_score(ScoreArgs score, cudaStream_t stream) {
  const int smem = 2 * kTileBytes + kRows * HD * 4 + CAPACITY * 4 + CAPACITY / 8;
  int blocks = 0;
  const void* kernel = reinterpret_cast<const void*>(&score_kernel<HD, CAPACITY>);
  cudaError_t err = persistent_blocks(kernel, kThreads, smem, int64_t{1} << 30, &blocks);
  if (err != cudaSuccess) return err;
  // query blocks of a CTA: 16, or fewer where the CTAs would not fill the GPU
  const int64_t rows = score.sums.rows[0] * score.s.kv_heads / blocks;
  score.rows = static_cast<int>(rows < 1 ? 1 : rows > kRows ? kRows : rows);
  const int64_t chunks = (score.sums.rows[0] + score.rows - 1) / score.rows;
  score_kernel<HD, CAPACITY><<<static_cast<unsigned>(chunks * score.s.kv_heads), kThreads, smem, stream>>>(score);
  return cudaGetLastError();
}

template <int HD>
cudaError_t launch(const PoolArgs& pool, const ScoreArgs& score, cudaStream_t stream) {
  const int64_t warps = (pool.sums.rows[0] + pool.sums.rows[1]) * pool.kv_heads;
  const int64_t pool_blocks = (warps + kPoolThreads / 32 - 1) / (kPoolThreads / 32);
  pool_kernel<HD><<<static_cast<unsigned>(pool_blocks), kPoolThreads, 0, stream>>>(pool);
  cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess) return err;
  // room for the longest sequence that there can be
  const int64_t longest = (score.s.rows_k + score.s.block_k - 1) / score.s.block_k;
  if (longest <= 256) return launch_score<HD, kRows * 256>(score, stream);
  if (longest <= 512) return launch_score<HD, kRows * 512>(score, stream);
  return launch_score<HD, kMostScores>(score, stream);
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
