// attention_cache_wide.cu -- attention over the paged NVFP4 cache where many rows share a
// key head: trees of drafted tokens, or large groups of query heads.
//
// The mathematics is attention_cache.cu's; there the products are mma.sync's, 1,024 a clock and
// SM, which 32 rows use up at the rate the cache arrives.  Here up to 128 rows are one tile of
// the fifth-generation tensor cores (4,096 a clock), and the values of the cache are
// laid out for them: exact fp16 in shared memory.
//
// Bound: the cache's bytes (18.4 KB a tile of 128 keys at head_dim 128: 787 clocks of an SM's
// share of the copy rate), closely followed by the way from codes to fp16 (32,768 elements a
// tile: about 750 clocks of four warps) and by the powers (128 rows: 512).  The products are
// 1,024 clocks of M = 128 whether or not its rows are used; they run beside everything else.
//
//   warps 0..3, 4..7  softmax of the even and of the odd tiles: a thread owns one row of S in
//                     TMEM and writes its weights, 2^6 e^(x - reference) in fp16, over it in two
//                     halves; the reference follows the row's maximum when that has grown by
//                     more than 2^8 (weights stay below 2^14).  Two streams with outputs of their
//                     own, so that the tensor cores work on one while the other has its
//                     softmax; joined at the end of a (sequence, head).
//   warps 8..11       codes and scales -> fp16 tiles, 128-byte swizzle, keys and values alike (a
//                     value tile's rows are the reduction of its product)
//   warp 12           copies pages of codes and scales into a raw ring, a lane each
//   warp 13           the products
// Work is dealt out and joined as in attention_cache.cu, in tiles of 128 keys, one CTA per SM.
// Where no sequence has more than 64 rows a key head (FEW) they fill both halves of the 128, so that two
// threads share a row's softmax, the keys of the tile's lower and of its upper half: each has zeros for
// weights of the other's keys, and an output of its own, joined as the streams' are.
//
// Measured, 32 query heads over 8 key heads of 128: 16 trees of 9 to 16 tokens (36 to 64 rows a
// key head) over 1,000 to 8,000 positions in 67 us (3 more with one thread a row), where the bytes take 13.  A
// tile of 128 keys takes about 2,530 clocks; 1,530 of them shared memory is busy (queries, keys and values
// read by the products 96 KB, fp16 tiles written 64 KB, codes in and out 36 KB, at 128 bytes a clock), and 17 us
// are launch, plan, queries, first tile, outputs and the joining kernel.  Without the conversions it was 65 us
// of 72, without the products 68, without the copies 69.  (Keys converted a tile ahead of values, fewer rows
// for the converting warps beside the softmax: no faster, and 85 us.)
// Every wait is bounded: one that runs out sets a device flag and tells the other roles to stop.
#include "attention_cache.cuh"
#include "h3q_ring.h"
#include "h3q_tcgen05.cuh"

namespace h3q {
namespace {

using namespace cached;

constexpr int kThreads = 512;
constexpr int kConvertWarp0 = 8;
constexpr int kCopyWarp = 12;
constexpr int kMmaWarp = 13;
constexpr int kRows = 128;             // rows per tile
constexpr int kKeys = 128;             // keys per tile
constexpr int kMaxCtas = 152;          // the workspace holds the parts of so many (608 of 32 rows)
constexpr int kGroupCost = 6;          // the time of a group's start and end, in tiles
constexpr int kFewRegs0 = 160, kFewRegs1 = 104, kFewRegs2 = 88;
constexpr float kInShift = 6.0f;       // weights are held as 2^6 e^(x - reference)
constexpr float kSlack = 8.0f;         // how far (log2) a row's maximum may pass its reference

__device__ int g_wide_fault;

template <int HD, bool FEW>
struct Shape {
  static constexpr int kTileRows = FEW ? 64 : kRows;          // rows that are different
  static constexpr int kCols = FEW ? kKeys / 2 : kKeys;       // keys of a thread's row
  static constexpr int kTileBytes = kKeys * HD * 2;           // a tile of keys or values in fp16
  static constexpr int kCodeBytes = kKeys * HD / 2;
  static constexpr int kRawBytes = kCodeBytes + kKeys * HD / 16;
  static constexpr int kSlots = 4;                            // fp16 tiles: K0 V0 K1 V1 ...
  static constexpr int kRaw = 4;                              // raw tiles, in the same order
  static constexpr int kOffTiles = kRows * HD * 2;            // after Q
  static constexpr int kOffRaw = kOffTiles + kSlots * kTileBytes;
  static constexpr int kOffJoin = kOffRaw + kRaw * kRawBytes; // 32 columns of 128 rows, fp32
  static constexpr int kOffMl = kOffJoin + 32 * kRows * 4;
  static constexpr int kOffFactor = kOffMl + kRows * 8;
  static constexpr int kOffBar = kOffFactor + kRows * 4;
  static constexpr int kBars = 2 * kSlots + 2 * kRaw + 1 + 8 + 1;
  static constexpr int kOffMisc = kOffBar + 8 * kBars;
  static constexpr int kSmem = kOffMisc + 16 + 1024;
  // TMEM: two S buffers (weights over them), then two outputs
  static constexpr uint32_t kO = 256;
  // Instruction descriptors (kind::f16): fp32 result (bit 4), fp16 operands (0), N >> 3 at bits
  // 17-22, M >> 4 at 24-28; V is transposed (bit 16).
  static constexpr uint32_t kIdescS = (1u << 4) | (uint32_t(kKeys >> 3) << 17) | (8u << 24);
  static constexpr uint32_t kIdescO = (1u << 4) | (1u << 16) | (uint32_t(HD >> 3) << 17) | (8u << 24);
};

__device__ __forceinline__ uint64_t ones(int64_t n) {
  return n <= 0 ? 0 : n >= 64 ? ~uint64_t{0} : (uint64_t{1} << n) - 1;
}

// 16 scores -> weights 2^(s * c + base), packed to fp16, and their sum added.
__device__ __forceinline__ void weights16(const uint32_t* s, float2 c2, float2 b2, float2& sum, uint32_t* w) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float2 p = fma2(make_float2(__uint_as_float(s[2 * j]), __uint_as_float(s[2 * j + 1])), c2, b2);
    p.x = ex2(p.x);
    p.y = ex2(p.y);
    sum = add2(sum, p);
    w[j] = half2_of(p.x, p.y);
  }
}

template <int HD, bool FEW>
__global__ void __launch_bounds__(kThreads, 1) cache_attention_wide_kernel(const Args a) {
  using S = Shape<HD, FEW>;
  constexpr int kTileRows = S::kTileRows;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t{1023});
  __shared__ PlanScratch<kThreads / 32> scratch;
  const uint32_t base = smem_u32(smem);
  const uint32_t bar_full = base + S::kOffBar;              // + 8 * slot
  const uint32_t bar_empty = bar_full + 8 * S::kSlots;
  const uint32_t bar_raw = bar_empty + 8 * S::kSlots;       // + 8 * raw slot
  const uint32_t bar_used = bar_raw + 8 * S::kRaw;
  const uint32_t bar_q = bar_used + 8 * S::kRaw;
  const uint32_t bar_s = bar_q + 8;                         // + 8 * stream
  const uint32_t bar_p = bar_s + 16;
  const uint32_t bar_p2 = bar_p + 16;
  const uint32_t bar_o = bar_p2 + 16;
  const uint32_t bar_drain = bar_o + 16;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::kOffMisc);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + S::kOffMisc + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kSlots; ++i) {
      mbar_init(bar_full + 8 * i, 128);
      mbar_init(bar_empty + 8 * i, 1);
    }
    for (int i = 0; i < S::kRaw; ++i) {
      mbar_init(bar_raw + 8 * i, 1);
      mbar_init(bar_used + 8 * i, 4);
    }
    mbar_init(bar_q, 256);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar_s + 8 * i, 1);
      mbar_init(bar_p + 8 * i, 128);
      mbar_init(bar_p2 + 8 * i, 128);
      mbar_init(bar_o + 8 * i, 1);
    }
    mbar_init(bar_drain, 1);
    *abort = 0;
    mbar_init_fence();
  }
  after_stream();
  Range w;
  if (!plan<kThreads / 32, kGroupCost>(a, kTileRows, kKeys, scratch, w)) return;

  auto wait = [&](uint32_t bar, uint32_t parity) {   // the whole warp: one decision
    return static_cast<bool>(__all_sync(0xffffffffu, wait_or_abort(bar, parity, abort, &g_wide_fault)));
  };

  // Registers: 8 softmax warps 200, 4 converting warps 72, the other four 40 (512 x 128 in all); with 168,
  // 96 and 80 a thread's 128 scores did not fit, 80 us for 16 trees, not 72.  Half the scores: 160, 104 and 88 (69
  // us; 144, 112, 112: 74, and 200, 72, 40: 73).
  if (warp < kConvertWarp0) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(FEW ? kFewRegs0 : 200));
    // ---- softmax of one stream
    const int x = warp >> 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;   // the TMEM of all 512 columns begins at 0
    const uint32_t col0 = FEW ? row / 64 * 64 : 0;   // of the thread's keys
    const uint32_t taddr = lane_base + x * kKeys, taddr_o = lane_base + S::kO + x * HD;
    float* join = reinterpret_cast<float*>(smem + S::kOffJoin) + row;          // [column][row]
    float2* join_ml = reinterpret_cast<float2*>(smem + S::kOffMl) + row;
    float* factors = reinterpret_cast<float*>(smem + S::kOffFactor);
    const float k_factor = __fmul_rn(__fdiv_rn(__fmul_rn(a.scale, kLog2e), *a.k_gsf), 256.0f);
    auto sync_both = [] { asm volatile("bar.sync 1, 256;" ::: "memory"); };
    bool first_segment = true, ok = true;
    uint32_t s_count = 0, o_count = 0;
    while (w.count > 0) {
      const int count = w.here();
      const bool whole = w.tile == 0 && count == w.s.tiles;
      const int kv_head = w.kv_head(), row_tile = w.group - kv_head * w.s.row_tiles;
      const int rho = row_tile * kTileRows + row % kTileRows;
      const bool valid = rho < w.s.n * a.group;
      const bool rows = rho - lane < w.s.n * a.group;   // any of the warp's
      {
        // the rows' queries, scaled, in fp16: rows of 128 bytes, their 16-byte pieces swizzled; a
        // row's lanes are side by side
        constexpr int kLanes = HD / 8, kStep = 32 / kLanes;   // lanes a row, rows a step of a warp
        constexpr int kSteps = 16 / kStep;
        const int col = lane % kLanes, r0 = warp * 16 + lane / kLanes;
        uint4 q[kSteps];
        uint32_t m[kSteps];
        {
          const int first = row_tile * kTileRows + r0 % kTileRows;   // (16 rows of a warp: no end of a tile inside)
          int t = first / a.group;
          int h = first - t * a.group;
#pragma unroll
          for (int i = 0; i < kSteps; ++i) {
            q[i] = make_uint4(0, 0, 0, 0);
            if (t < w.s.n)
              q[i] = load16_fresh(a.q + (w.s.row0 + t) * a.ld_q + static_cast<int64_t>(kv_head * a.group + h) * HD + col * 8);
            for (h += kStep; h >= a.group; h -= a.group) ++t;
          }
        }
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          const uint32_t words[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
          m[i] = magnitude_bits(words);
        }
#pragma unroll
        for (int o = kLanes / 2; o >= 1; o >>= 1)
#pragma unroll
          for (int i = 0; i < kSteps; ++i) m[i] = max(m[i], __shfl_xor_sync(0xffffffffu, m[i], o));
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          const uint32_t words[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
          const int r = r0 + i * kStep;
          const float f = query_factor(m[i]);
          if (col == 0) factors[r] = inverse_power(f);
          uint32_t h[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 v = bf16x2_to_float2(words[k]);
            h[k] = half2_of(__fmul_rn(v.x, f), __fmul_rn(v.y, f));
          }
          *reinterpret_cast<uint4*>(smem + (col / 8) * (kRows * 128) + r * 128 + (((col % 8) ^ (r & 7)) << 4)) =
              make_uint4(h[0], h[1], h[2], h[3]);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // the products read them
        mbar_arrive(bar_q);
      }
      sync_both();
      const float c = fmaxf(__fmul_rn(k_factor, factors[row]), 0x1p-126f);   // never 0: a hidden key's -inf stays one
      float m_ref = -INFINITY, m_seen = -INFINITY, l = 0.0f;
      // Move the reference to the maximum seen, where that has grown: scale the sum and O.
      auto rescale = [&](bool any_o) {
        float alpha = 1.0f;
        if (__fmul_rn(__fadd_rn(m_seen, -m_ref), c) > kSlack) {
          alpha = ex2(__fmul_rn(__fadd_rn(m_ref, -m_seen), c));
          m_ref = m_seen;
          l = __fmul_rn(l, alpha);
        }
        if (!any_o) return;
#pragma unroll 1
        for (int i = 0; i < HD; i += 32) {
          uint32_t o[32];
          tc_load32(taddr_o + i, o);
          tc_wait_load(o);
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__fmul_rn(__uint_as_float(o[k]), alpha));
          tc_store32(taddr_o + i, o);
        }
        tc_wait_store();
      };
      const uint32_t seen_by_all = w.s.ctx < 0 ? 0 : min(w.s.ctx, w.s.len);
      for (int i = x; i < count && ok; i += 2) {
        if (!(ok = wait(bar_s + 8 * x, s_count & 1))) break;
        ++s_count;
        if (!rows) {   // no row of this warp exists: its weights are nobody's
          mbar_arrive(bar_p + 8 * x);
          mbar_arrive(bar_p2 + 8 * x);
          continue;
        }
        tc_fence_after();   // S was issued after the product before it of this stream: O is at rest
        const uint32_t key0 = static_cast<uint32_t>(w.tile + i) * kKeys;
        const bool masked = key0 + kKeys > seen_by_all;
        uint32_t see[4] = {~0u, ~0u, ~0u, ~0u};
        if (masked) {   // which of the tile's keys the row sees
          const int64_t d = w.s.ctx - static_cast<int64_t>(key0);
          const int tok = rho / a.group;
          const uint64_t mask = !valid ? 0 : a.mask != nullptr ? static_cast<uint64_t>(a.mask[w.s.row0 + tok])
                                                               : ~uint64_t{0} >> (63 - tok);
          uint64_t lo = ones(d), hi = ones(d - 64);
          if (d >= 64 && d < 128) {
            hi |= mask << (d - 64);
          } else if (d > 0 && d < 64) {
            lo |= mask << d;
            hi |= mask >> (64 - d);
          } else if (d <= 0 && d > -64) {
            lo |= mask >> -d;
          }
          lo &= ones(w.s.len - static_cast<int64_t>(key0));
          hi &= ones(w.s.len - static_cast<int64_t>(key0) - 64);
          see[0] = static_cast<uint32_t>(lo), see[1] = static_cast<uint32_t>(lo >> 32);
          see[2] = static_cast<uint32_t>(hi), see[3] = static_cast<uint32_t>(hi >> 32);
          if (FEW && col0 != 0) see[0] = see[2], see[1] = see[3];
        }
        const float2 c2 = make_float2(c, c);
        uint32_t s[S::kCols / 32][32];
        uint32_t wt[32];
        float2 sum;
        bool fresh = i < 2;   // no reference yet: only the maximum is formed
        for (;;) {
#pragma unroll
          for (int k = 0; k < S::kCols / 32; ++k) tc_load32(taddr + col0 + 32 * k, s[k]);
          tc_wait_load(s[0]);
#pragma unroll
          for (int k = 1; k < S::kCols / 32; ++k) tc_loaded(s[k]);
          if (masked) {
#pragma unroll
            for (int k = 0; k < S::kCols; ++k)
              if (!(see[k / 32] >> (k % 32) & 1)) s[k / 32][k % 32] = 0xff800000u;
          }
          float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int k = 0; k < S::kCols; k += 8)
#pragma unroll
            for (int h = 0; h < 4; ++h)
              m[h] = max3(m[h], __uint_as_float(s[k / 32][k % 32 + 2 * h]), __uint_as_float(s[k / 32][k % 32 + 2 * h + 1]));
          if (fresh) {
            fresh = false;
            m_seen = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
            rescale(false);
            continue;
          }
          const float shift = m_ref == -INFINITY ? kInShift : __fadd_rn(kInShift, -__fmul_rn(m_ref, c));
          const float2 b2 = make_float2(shift, shift);
          sum = make_float2(0.0f, 0.0f);
#pragma unroll
          for (int k = 0; k < 64; k += 16) weights16(s[k / 32] + k % 32, c2, b2, sum, wt + k / 2);
          m_seen = fmaxf(max3(m_seen, m[0], m[1]), fmaxf(m[2], m[3]));
          // (a difference of two -inf is no number, and not above)
          if (!__any_sync(0xffffffffu, __fmul_rn(__fadd_rn(m_seen, -m_ref), c) > kSlack)) break;
          rescale(i >= 2);
        }
        const float shift = m_ref == -INFINITY ? kInShift : __fadd_rn(kInShift, -__fmul_rn(m_ref, c));
        const float2 b2 = make_float2(shift, shift);
        if constexpr (FEW) {   // the weights of this thread's half, and none of the other's
          store_weights<32>(taddr + col0 / 2, wt);
          uint32_t none[32] = {};
          store_weights<32>(taddr + (32 - col0 / 2), none);
          l = __fadd_rn(l, __fadd_rn(sum.x, sum.y));
          tc_wait_store();
          tc_fence_before();
          mbar_arrive(bar_p + 8 * x);
        } else {
          store_weights<32>(taddr, wt);
          tc_wait_store();
          tc_fence_before();
          mbar_arrive(bar_p + 8 * x);
#pragma unroll
          for (int k = 0; k < 64; k += 16) weights16(s[S::kCols / 64 + k / 32] + k % 32, c2, b2, sum, wt + k / 2);
          store_weights<32>(taddr + 32, wt);
          l = __fadd_rn(l, __fadd_rn(sum.x, sum.y));
          tc_wait_store();
          tc_fence_before();
        }
        mbar_arrive(bar_p2 + 8 * x);
      }
      if (ok && x < count) {
        ok = wait(bar_o + 8 * x, o_count & 1);
        ++o_count;
        tc_fence_after();
      }
      if (raised(abort)) ok = false;
      // ---- join the streams, 32 columns at a time; write the outputs or leave the part
      const float m_mine = m_ref == -INFINITY ? -INFINITY : __fmul_rn(m_ref, c);
      if (x == 1) *join_ml = make_float2(m_mine, l);
      sync_both();
      const bool two = count > 1;
      float f0 = 0.0f, f1 = 0.0f, m = m_mine;
      if (x == 0) {
        const float2 other = *join_ml;
        if (two) m = fmaxf(m, other.x);
        const float use = m == -INFINITY ? 0.0f : m;
        f0 = ex2(__fadd_rn(m_mine, -use));
        f1 = two ? ex2(__fadd_rn(other.x, -use)) : 0.0f;
        l = __fmul_rn(l, f0);
        if (two) l = __fmaf_rn(other.y, f1, l);
      }
      float g0 = 1.0f, g1 = 0.0f;   // the lower and the upper keys' share
      if constexpr (FEW) {
        sync_both();
        if (x == 0 && col0 != 0) *join_ml = make_float2(m, l);
        sync_both();
        if (x == 0 && col0 == 0) {
          const float2 other = join_ml[64];
          const float top = fmaxf(m, other.x), use = top == -INFINITY ? 0.0f : top;
          g0 = ex2(__fadd_rn(m, -use));
          g1 = ex2(__fadd_rn(other.x, -use));
          l = __fmaf_rn(other.y, g1, __fmul_rn(l, g0));
          m = top;
        }
      }
      // outputs are divided by the sum here, and scaled as they are stored: both at once may be too small for fp32
      const float inv = !whole ? 1.0f : l == 0.0f ? 0.0f : __fdiv_rn(1.0f, l);
      if constexpr (FEW) {
        g0 = __fmul_rn(g0, inv);
        g1 = __fmul_rn(g1, inv);
      } else {
        f0 = __fmul_rn(f0, inv);
        f1 = __fmul_rn(f1, inv);
      }
      const float v_factor = __fdiv_rn(256.0f, *a.v_gsf);
      int rho_out = rho;
      asm volatile("" : "+r"(rho_out));   // (where it goes is formed here, not kept over the tiles)
      const int tok = rho_out / a.group, head = kv_head * a.group + rho_out - tok * a.group;
      const int64_t out_row = w.s.row0 + tok;
      const int64_t part = (static_cast<int64_t>(blockIdx.x) * 2 + (first_segment ? 0 : 1)) * kTileRows + row % kTileRows;
#pragma unroll 1
      for (int i = 0; i < HD; i += 32) {
        uint32_t o[32];
        __syncwarp();
        if (ok && rows && (x == 0 || two)) {   // (given up: the TMEM may not even be this CTA's yet)
          tc_load32(taddr_o + i, o);
          tc_wait_load(o);
        }
        if (rows && x == 1 && two) {
#pragma unroll
          for (int k = 0; k < 32; ++k) join[k * kRows] = __uint_as_float(o[k]);
        }
        if (two) sync_both();
        float v[32];
        if (x == 0 && rows) {
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            v[k] = __fmul_rn(__uint_as_float(o[k]), f0);
            if (two) v[k] = __fmaf_rn(join[k * kRows], f1, v[k]);
          }
        }
        if constexpr (FEW) {
          if (x == 0 && rows && col0 != 0) {   // (its own places, which it has just read)
#pragma unroll
            for (int k = 0; k < 32; ++k) join[k * kRows] = v[k];
          }
          sync_both();
          if (x == 0 && rows && col0 == 0) {
#pragma unroll
            for (int k = 0; k < 32; ++k) v[k] = __fmaf_rn(join[k * kRows + 64], g1, __fmul_rn(v[k], g0));
          }
        }
        if (x == 0 && col0 == 0 && valid && ok) {
          if (whole) {
            uint16_t* dst = a.o + (out_row * a.heads + head) * HD + i;
#pragma unroll
            for (int k = 0; k < 32; k += 8) {
              uint32_t p[4];
#pragma unroll
              for (int h = 0; h < 4; ++h)
                p[h] = l == 0.0f ? 0u
                                 : float2_to_bf16x2(make_float2(__fmul_rn(v[k + 2 * h], v_factor),
                                                                __fmul_rn(v[k + 2 * h + 1], v_factor)));
              store16(dst + k, make_uint4(p[0], p[1], p[2], p[3]));
            }
          } else {
            constexpr float kUp = 256.0f;   // parts hold 2^14 e^(x - m): 2^(kPShift - kInShift) times more
            float* dst = a.part + part * HD + i;
#pragma unroll
            for (int k = 0; k < 32; k += 4)
              *reinterpret_cast<float4*>(dst + k) = make_float4(__fmul_rn(v[k], kUp), __fmul_rn(v[k + 1], kUp),
                                                                __fmul_rn(v[k + 2], kUp), __fmul_rn(v[k + 3], kUp));
          }
        }
        if (two || FEW) sync_both();
      }
      if (x == 0 && col0 == 0 && valid && ok) {
        if (!whole)
          reinterpret_cast<float2*>(a.part_ml)[part] = make_float2(m, __fmul_rn(l, 256.0f));
        else if (a.lse != nullptr)
          a.lse[head * a.rows + out_row] =
              l == 0.0f ? -INFINITY : __fmul_rn(__fadd_rn(m, __fadd_rn(log2f(l), -kInShift)), kLn2);
      }
      tc_fence_before();   // O has been read before the next segment's first weights are announced
      first_segment = false;
      w.advance(a, count, kTileRows, kKeys);
    }
  } else if (warp < kCopyWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(FEW ? kFewRegs1 : 72));
    // ---- codes and scales -> fp16.  A lane takes 32 codes of a row (16 bytes), a row's lanes
    // side by side; it writes four 16-byte pieces.  Lanes of the upper 64 columns take theirs in
    // another order, so that eight lanes' pieces fall into eight banks.
    constexpr int kRowLanes = HD / 32;
    constexpr int kStepRows = 32 / kRowLanes;
    const int part = lane % kRowLanes, row_in = lane / kRowLanes;
    const int half = part >> 1;
    uint32_t n = 0;
    for (int left = w.count; left > 0; --left) {
      bool ok = true;
#pragma unroll 1
      for (int v = 0; v < 2; ++v, ++n) {
        const uint32_t slot = n % S::kSlots, raw = n % S::kRaw;
        if (!(ok = wait(bar_raw + 8 * raw, (n / S::kRaw) & 1) && wait(bar_empty + 8 * slot, ((n / S::kSlots) & 1) ^ 1u)))
          break;
        const uint8_t* codes = smem + S::kOffRaw + raw * S::kRawBytes;
        const uint8_t* scales = codes + S::kCodeBytes;
        uint8_t* tile = smem + S::kOffTiles + slot * S::kTileBytes + half * (kKeys * 128);
        const int row0 = (warp - kConvertWarp0) * 32 + row_in;
        uint4 c4[kRowLanes];
        uint32_t sc[kRowLanes];
#pragma unroll
        for (int i = 0; i < kRowLanes; ++i) {   // all loads before the first store
          const int row = row0 + i * kStepRows;
          c4[i] = *reinterpret_cast<const uint4*>(codes + row * (HD / 2) + part * 16);
          sc[i] = *reinterpret_cast<const uint16_t*>(scales + row * (HD / 16) + part * 2);
        }
#pragma unroll
        for (int i = 0; i < kRowLanes; ++i) {
          const int row = row0 + i * kStepRows;
          uint32_t cw[4] = {c4[i].x, c4[i].y, c4[i].z, c4[i].w};
          uint32_t f[2] = {scale_half(sc[i]) * 0x10001u, scale_half(sc[i] >> 8) * 0x10001u};
          const int flip = half * 2;
          if (half) {
            cw[0] = c4[i].z, cw[1] = c4[i].w, cw[2] = c4[i].x, cw[3] = c4[i].y;
            const uint32_t f0 = f[0];
            f[0] = f[1], f[1] = f0;
          }
          uint8_t* dst = tile + row * 128;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t h[4];
            codes_to_half(cw[k], h);
#pragma unroll
            for (int e = 0; e < 4; ++e) h[e] = hmul2(h[e], f[k >> 1]);
            const int piece = (part & 1) * 4 + (k ^ flip);
            *reinterpret_cast<uint4*>(dst + ((piece ^ (row & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_used + 8 * raw);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // the products read it
        mbar_arrive(bar_full + 8 * slot);
      }
      if (!ok) break;
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(FEW ? kFewRegs2 : 40));
    if (warp == kCopyWarp) {
      // ---- copies: lane 2 i has the codes of page i of the tile, lane 2 i + 1 its scales
      const int page_shift = a.cache.page_shift;
      const int piece_keys = 1 << page_shift;   // at most a tile's 128
      const int pieces = kKeys >> page_shift;
      const int piece = lane >> 1, what = lane & 1;
      const int per = what ? HD / 16 : HD / 2;   // bytes a key
      const uint32_t dst = base + S::kOffRaw + (what ? S::kCodeBytes : 0) + piece * piece_keys * per;
      auto page_number = [&]() -> int {   // of this lane's piece of the tile, -1 for none
        const int64_t pos = static_cast<int64_t>(w.tile) * kKeys + piece * piece_keys;
        if (piece >= pieces || pos >= w.s.len) return -1;
        const int64_t p = a.at.table[w.b * a.at.max_pages + (pos >> page_shift)];
        return p < 0 || p >= a.cache.num_pages ? 0 : static_cast<int>(p);  // any page, so that the read is of the cache
      };
      int page = page_number();
      uint32_t n = 0;
      bool ok = true;
      while (w.count > 0 && ok) {
        const int64_t row = (static_cast<int64_t>(page) * a.cache.kv_heads + w.kv_head()) << page_shift;
        const uint32_t live = __ballot_sync(0xffffffffu, page >= 0);
        const bool mine = page >= 0;
        w.advance(a, 1, kTileRows, kKeys);   // the next tile's pages, before this one's slots are waited for
        if (w.count > 0) page = page_number();
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          const uint32_t raw = fill_slot(n, S::kRaw), bar = bar_raw + 8 * raw;
          if (!(ok = wait(bar_used + 8 * raw, fill_parity(n, S::kRaw) ^ 1u))) break;
          if (lane == 0) mbar_expect_tx(bar, __popc(live) / 2 * piece_keys * (HD / 2 + HD / 16));
          __syncwarp();
          if (mine)
            bulk_load(dst + raw * S::kRawBytes, (what ? a.cache.scales[v] : a.cache.codes[v]) + row * per,
                      piece_keys * per, bar);
          ++n;
        }
      }
      // converting warps that give up do not wait for the copies: they have landed before the CTA goes
      for (uint32_t k = first_fill_under_way(n, S::kRaw); k < n; ++k)
        (void)wait_bounded(bar_raw + 8 * fill_slot(k, S::kRaw), fill_parity(k, S::kRaw));
    } else if (warp == kMmaWarp) {
      // ---- products.  The whole warp allocates the CTA's TMEM: all 512 columns, so they begin at 0.
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                   "r"(512)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
      const uint32_t q_low = desc_low(base, 16);
      const uint32_t k_low = desc_low(base + S::kOffTiles, 16);
      const uint32_t v_low = desc_low(base + S::kOffTiles, kKeys * 128);   // 64 columns of V, then the next 64
      uint32_t n0 = 0;                   // slot number of the segment's first K tile
      uint32_t p_count[2] = {0, 0}, segments = 0;
      bool ok = true;
      // Each lane waits for a barrier of its own (0: none), the warp for all of them.
      auto wait_lanes = [&](uint32_t bar, uint32_t parity) {
        bool done = bar == 0 || mbar_try_wait(bar, parity);
        if (__all_sync(0xffffffffu, done)) return true;
        const uint64_t start = now_ns();
        for (uint32_t i = 1;; ++i) {
          if (!done) done = mbar_try_wait(bar, parity);
          if (__all_sync(0xffffffffu, done)) return true;
          if ((i & (kPolls - 1)) == 0) {
            const bool late = now_ns() - start >= kWaitNs;
            if (late && lane == 0) {
              *abort = 1;
              atomicExch(&g_wide_fault, 1);
            }
            if (__any_sync(0xffffffffu, late || raised_here(abort))) return false;
          }
        }
      };
      auto slot_of = [&](int i) { return (n0 + i) % S::kSlots; };
      auto full = [&](int i) { return bar_full + 8 * slot_of(i); };
      auto full_parity = [&](int i) { return ((n0 + i) / S::kSlots) & 1u; };
      auto release = [&](int i) { commit_elected(bar_empty + 8 * slot_of(i)); };
      auto s_product = [&](int x, int i) {   // S[x] = Q K[i]^T
        const uint32_t k = k_low + slot_of(2 * i) * (S::kTileBytes >> 4);
        tc_fence_after();
#pragma unroll
        for (int d = 0; d < HD / 16; ++d)
          mma_ss(x * kKeys, q_low + (((d / 4) * (kRows * 128) + (d % 4) * 32) >> 4),
                 k + (((d / 4) * (kKeys * 128) + (d % 4) * 32) >> 4), S::kIdescS, d > 0);
        commit_elected(bar_s + 8 * x);
        release(2 * i);
      };
      auto o_half = [&](int x, int i, int half) {   // half of O[x] += P[x] V[i]
        const uint32_t v = v_low + slot_of(2 * i + 1) * (S::kTileBytes >> 4);
        tc_fence_after();
#pragma unroll
        for (int d = half * 4; d < half * 4 + 4; ++d)
          mma_ts(S::kO + x * HD, x * kKeys + 8 * d, v + (d * 2048 >> 4), S::kIdescO, i > 1 || d > 0);
      };
      while (w.count > 0 && ok) {
        const int count = uniform(w.here());
        ok = wait_lanes(lane == 0 ? bar_q : lane == 1 ? full(0) : lane == 2 && count > 1 ? full(2) : 0u,
                        lane == 0 ? segments & 1 : lane == 1 ? full_parity(0) : full_parity(2));
        ++segments;
        if (ok) {
          s_product(0, 0);
          if (count > 1) s_product(1, 1);
        }
        for (int i0 = 0; i0 < count && ok; i0 += 2) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int i = i0 + x;
            if (!ok || i >= count) continue;
            const bool more = i + 2 < count;
            const uint32_t parity = p_count[x]++ & 1;
            if (!(ok = wait_lanes(lane == 0 ? bar_p + 8 * x : lane == 1 ? full(2 * i + 1) : 0u,
                                  lane == 0 ? parity : full_parity(2 * i + 1))))
              continue;
            o_half(x, i, 0);
            if (!(ok = wait_lanes(lane == 0 ? bar_p2 + 8 * x : 0u, parity))) continue;
            o_half(x, i, 1);
            release(2 * i + 1);   // (its successor is converted before K[i + 2]'s)
            if (more) {
              if (!(ok = wait_lanes(lane == 0 ? full(2 * i + 4) : 0u, full_parity(2 * i + 4)))) continue;
              s_product(x, i + 2);
            } else {
              commit_elected(bar_o + 8 * x);
            }
          }
        }
        n0 += 2 * count;
        w.advance(a, count, kTileRows, kKeys);
      }
      // what is issued finishes before the TMEM is freed, whoever gave up and when
      commit_elected(bar_drain);
      (void)wait_bounded(bar_drain, 0);
      __syncwarp();
      // the commits to the empty barriers arrive before the CTA goes
      for (uint32_t k = n0 < S::kSlots ? 0 : n0 - S::kSlots; ok && k < n0; ++k)
        ok = wait(bar_empty + 8 * (k % S::kSlots), (k / S::kSlots) & 1);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(*tmem_slot), "r"(512) : "memory");
  }
}

template <int HD, bool FEW>
cudaError_t launch(Args a, uint8_t* workspace, cudaStream_t stream) {
  using S = Shape<HD, FEW>;
  static_assert(S::kSmem <= 227 * 1024, "shared memory");
  static_assert(256 * kFewRegs0 + 128 * kFewRegs1 + 128 * kFewRegs2 <= 65536, "registers");
  int blocks = 0;
  cudaError_t err = persistent_blocks(reinterpret_cast<const void*>(&cache_attention_wide_kernel<HD, FEW>), kThreads,
                                      S::kSmem, kMaxCtas, &blocks);
  if (err != cudaSuccess) return err;
  place_workspace(a, workspace, kMaxCtas, S::kTileRows);
  a.whole = whole_groups(a, blocks, S::kTileRows, kKeys);
  err = launch_early(&cache_attention_wide_kernel<HD, FEW>, blocks, kThreads, S::kSmem, stream, a);
  if (err != cudaSuccess || blocks < 2 || a.whole) return err;
  return launch_join<HD, S::kTileRows, kKeys>(a, blocks, stream);
}

template <int HD>
cudaError_t dispatch(const Args& a, uint8_t* workspace, cudaStream_t stream) {
  return static_cast<int64_t>(a.max_rows) * a.group <= 64 ? launch<HD, true>(a, workspace, stream)
                                                           : launch<HD, false>(a, workspace, stream);
}

}  // namespace

cudaError_t launch_cache_attention_wide(const cached::Args& a, uint8_t* workspace, cudaStream_t stream) {
  return a.cache.head_dim == 64 ? dispatch<64>(a, workspace, stream) : dispatch<128>(a, workspace, stream);
}

cudaError_t cache_attention_wide_error_flag(int* flag) {
  int zero = 0;
  cudaError_t err = cudaMemcpyFromSymbol(flag, g_wide_fault, sizeof(int));
  if (err == cudaSuccess) err = cudaMemcpyToSymbol(g_wide_fault, &zero, sizeof(int));
  return err;
}

}  // namespace h3q
