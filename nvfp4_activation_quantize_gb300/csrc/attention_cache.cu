// attention_cache.cu -- attention of one or a few new tokens a sequence over the paged
// NVFP4 cache that holds their context and, at its end, the tokens themselves.
//
// Per row (a token and one of its heads): x_j = scale * q . k_j over the keys it sees,
// o = sum_j e^(x_j - m) v_j / sum_j e^(x_j - m), m = max_j x_j, in one pass with the
// running maximum and sum.  Keys before the new tokens are seen by all of them; a new
// token sees the new tokens of its mask (64 bits; without one, itself and those before).
//
// What bounds it is the cache: 2 x 72 bytes a position and head at head_dim 128.
// The rows that share a key head (a token's group of query heads, all tokens of the
// sequence) are taken together, so the cache is read once for up to 8 * NT rows.
//
// Arithmetic.  A value of the cache is E2M1 * E4M3 / gsf.  The product has at most six
// significant bits, so it is exact in fp16 (scaled by 2^-8: 2^-18 .. 10.5), and 1 / gsf
// goes into the softmax scale and into the output: keys and values enter the tensor
// cores without a rounding.  A query row is scaled by the power of two that brings its
// largest magnitude into [2^14, 2^15), where every bf16 value down to 2^-29 of it is
// exact in fp16.  Weights are held as 2^6 e^(x - reference), below 2^14, and rounded to fp16
// once (11 bits), their sum is formed in fp32 from the unrounded ones; all accumulators are fp32.
//
// Products with mma.sync m16n8k16 (16 keys or 16 value columns by 8 rows): a
// decoding step has 8 to 32 rows where a tcgen05 tile has 128.  S^T = K Q^T takes the
// keys as the left operand, so a lane's codes (32 consecutive elements of a key) are the
// operand as they lie in memory, one conversion instruction per two codes; O^T = V^T P^T
// pairs the codes of two keys by two byte-wise selections per 8 + 8 codes first, and P^T
// is the transposed accumulator (movmatrix).  Measured on this GPU: the conversion with the scaling
// runs at 77 elements a clock and SM (the copy rate needs 42), bit-field arithmetic
// instead at 44; mma.sync at 1,024 products a clock and SM, a third of it used at NT 1.
//
// Work: tiles of 256 keys (128 at head_dim 256) of one (sequence, key head, row tile), in that
// order, dealt out in contiguous ranges to the CTAs of one wave, equal in tiles and one more for
// each group (without it the CTAs of short sequences came last: 78 us for 64 tokens, not 72).
// In a CTA one warp copies: the tile's keys, then its values, into a ring of such slots, a
// copy a lane (a page's codes, its scales), the page numbers looked up a tile ahead.
// Four warps take 64 keys of each tile, each with its own running maximum, sum and output,
// and are joined through shared memory at the end of a (sequence, head).  One that a
// range's end cuts leaves its parts in the workspace, which the second kernel joins in order of
// the ranges: no atomics, the same result every time.  (With a ring of 32-key tiles to each
// warp, four copies of 256 bytes and 2 KB a tile: 103 us for 64 tokens over 4,503 positions
// each, 68 of them in the copies alone.)
//
// A row's weights are taken against a reference, a power of two, that follows its maximum only where that
// has grown by more than 2^8, so most tiles need one vote and no exchange between lanes.
//
// Measured, 32 query heads over 8 key heads of 128: 64 tokens over 500 to 8,191 positions each in
// 68 us (49 is the bytes' time at the copy rate), two tokens over 120,000 to 131,071 in 61 us (44).
// Longer contexts cost the copy rate's time, 6.7 TB/s; 11 us are launch, plan, first tiles and join.  At 70
// us it was 63 with the copies alone and 64 with the arithmetic alone.
#include <cmath>

#include "attention_cache.cuh"
#include "h3q_ring.h"

namespace h3q {
namespace {

using namespace cached;

constexpr int kWarps = 4;                        // that compute; one more copies
constexpr int kGroupCost = 1;                    // the time of a group's start and end, in tiles
constexpr float kInShift = 6.0f;                 // weights are held as 2^6 e^(x - reference)
constexpr float kSlack = 8.0f;                   // how far (log2) a maximum may pass its reference

__device__ int g_cache_attention_fault;

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

template <int BYTES>
__device__ __forceinline__ void lds(const uint8_t* p, uint32_t (&w)[BYTES / 4]) {
  if constexpr (BYTES == 4) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (BYTES == 8) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x, w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < BYTES / 16; ++i) {
      const uint4 v = *reinterpret_cast<const uint4*>(p + 16 * i);
      w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
    }
  }
}

template <int HD, int NT>
struct Shape {
  static constexpr int kRows = 8 * NT;                 // rows per tile
  static constexpr int kWarpKeys = HD == 256 || NT == 3 || (NT == 4 && HD == 128) ? 32 : 64;   // keys of a tile per warp
  static constexpr int kKeys = kWarps * kWarpKeys;     // keys per tile
  static constexpr int kMt = NT == 1 ? kWarpKeys / 16 : 2;   // 16-key products whose scores are held at once
  static constexpr int kCodeBytes = kKeys * HD / 2;    // a slot: a tile's codes of keys or values, then their scales
  static constexpr int kSlotBytes = kCodeBytes + kKeys * HD / 16;
  static constexpr int kSlots = HD == 64 || kKeys == 128 ? 4 : 3;
  // Many rows need more registers than an even split leaves: there the copying warp has three
  // idle ones beside it, and the four hand theirs over (256 x 128 = 128 x 200 + 128 x 56), two CTAs
  // an SM, not three.  (64 sequences of 4,503 positions, split and even: 16 rows a key head at
  // head_dim 128 106 and 128 us; at 64, 16 rows 78 and 66, 24 rows 109 and 92, 32 rows 115 and 153.)
  static constexpr bool kSplit = HD == 256 || (NT > 1 && HD == 128) || NT == 4;
  static constexpr int kThreads = (kWarps + (kSplit ? 4 : 1)) * 32;
  static constexpr int kCtas = kSplit ? 2 : 3;         // per SM
  static constexpr int kSteps = HD / 16;               // products of 16 along the head
  static constexpr bool kQShared = NT > 2 || (NT == 2 && HD == 64);   // query fragments in shared memory
  static constexpr int kPitch = HD + 4;                // floats per row of the joining buffer
  static constexpr int kOffJoin = kSlots * kSlotBytes;
  static constexpr int kOffMl = kOffJoin + kWarps * 8 * kPitch * 4;
  static constexpr int kOffQ = kOffMl + kWarps * 8 * 8;
  static constexpr int kOffMask = kOffQ + (kQShared ? NT * kSteps * 32 * 8 : 0);
  static constexpr int kOffFactor = kOffMask + kRows * 8;
  static constexpr int kOffBar = kOffFactor + kRows * 4;
  static constexpr int kSmem = kOffBar + 2 * kSlots * 8 + 8;
};

// 2^e for e <= 0 (0 below 2^-126).
__device__ __forceinline__ float power(int e) { return e < -126 ? 0.0f : __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

// The computing warps' barrier (the copying warp runs ahead).
__device__ __forceinline__ void sync_compute() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

template <int HD, int NT>
__global__ void __launch_bounds__(Shape<HD, NT>::kThreads, Shape<HD, NT>::kCtas) cache_attention_kernel(const Args a) {
  using S = Shape<HD, NT>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ PlanScratch<S::kThreads / 32> scratch;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t bar_full = smem_u32(smem + S::kOffBar);   // + 8 * slot
  const uint32_t bar_empty = bar_full + 8 * S::kSlots;
  volatile int* abort = reinterpret_cast<volatile int*>(smem + S::kOffBar + 16 * S::kSlots);

  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kSlots; ++i) {
      mbar_init(bar_full + 8 * i, 1);
      mbar_init(bar_empty + 8 * i, kWarps);
    }
    *abort = 0;
    mbar_init_fence();
  }
  after_stream();
  Range r;
  if (!plan<S::kThreads / 32, kGroupCost>(a, S::kRows, S::kKeys, scratch, r)) return;

  if (warp >= kWarps) {
    if constexpr (S::kSplit) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
      if (warp > kWarps) return;
    }
    // ---- copies.  A lane has one page of the tile (`per` lanes more than one page's codes and
    // scales at the smaller pages): lane 2 i its codes, lane 2 i + 1 its scales.
    const int page_shift = a.cache.page_shift;
    const int page_keys = 1 << page_shift;
    const int piece_keys = page_keys < S::kKeys ? page_keys : S::kKeys;
    const int pieces = S::kKeys / piece_keys;
    const int piece = lane >> 1, what = lane & 1;
    const int per = what ? HD / 16 : HD / 2;   // bytes a key
    const uint32_t dst_off = (what ? S::kCodeBytes : 0) + piece * piece_keys * per;
    const uint32_t slots = smem_u32(smem);
    auto page_number = [&]() -> int {   // of this lane's piece of the tile, -1 for none
      const int64_t pos = static_cast<int64_t>(r.tile) * S::kKeys + piece * piece_keys;
      if (piece >= pieces || pos >= r.s.len) return -1;
      const int64_t p = a.at.table[r.b * a.at.max_pages + (pos >> page_shift)];
      return p < 0 || p >= a.cache.num_pages ? 0 : static_cast<int>(p);  // any page, so that the read is of the cache
    };
    int page = page_number();
    uint32_t n = 0;   // slots filled
    bool ok = true;
    while (r.count > 0 && ok) {
      const int64_t in_page = (static_cast<int64_t>(r.tile) * S::kKeys + piece * piece_keys) & (page_keys - 1);
      const int64_t row = ((static_cast<int64_t>(page) * a.cache.kv_heads + r.kv_head()) << page_shift) + in_page;
      const uint32_t live = __ballot_sync(0xffffffffu, page >= 0);
      const bool mine = page >= 0;
      // the next tile's pages, before this one's slots are waited for
      r.advance(a, 1, S::kRows, S::kKeys);
      if (r.count > 0) page = page_number();
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const uint32_t slot = fill_slot(n, S::kSlots), bar = bar_full + 8 * slot;
        ok = __all_sync(0xffffffffu, wait_or_abort(bar_empty + 8 * slot, fill_parity(n, S::kSlots) ^ 1u, abort,
                                                   &g_cache_attention_fault));
        if (!ok) break;
        if (lane == 0) mbar_expect_tx(bar, __popc(live) / 2 * piece_keys * (HD / 2 + HD / 16));
        __syncwarp();
        if (mine)
          bulk_load(slots + slot * S::kSlotBytes + dst_off, (what ? a.cache.scales[v] : a.cache.codes[v]) + row * per,
                    piece_keys * per, bar);
        ++n;
      }
    }
    // computing warps that give up do not wait for the copies: they have landed before the CTA goes
    for (uint32_t k = first_fill_under_way(n, S::kSlots); k < n; ++k)
      (void)wait_bounded(bar_full + 8 * fill_slot(k, S::kSlots), fill_parity(k, S::kSlots));
    return;
  }

  // ---- the computing warps
  if constexpr (S::kSplit) asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
  const int g = lane >> 2, t = lane & 3;
  float* join = reinterpret_cast<float*>(smem + S::kOffJoin);
  float2* join_ml = reinterpret_cast<float2*>(smem + S::kOffMl);
  uint2* q_shared = reinterpret_cast<uint2*>(smem + S::kOffQ);
  uint64_t* row_mask = reinterpret_cast<uint64_t*>(smem + S::kOffMask);
  float* row_factor = reinterpret_cast<float*>(smem + S::kOffFactor);
  const float k_factor = __fmul_rn(__fdiv_rn(__fmul_rn(a.scale, kLog2e), *a.k_gsf), 256.0f);
  const float v_factor = __fdiv_rn(256.0f, *a.v_gsf);
  uint32_t slot = 0, parity = 0;   // of the slot that is taken next
  bool alive = true;     // false: a wait ran out; no further tile is computed, and no output stored
  auto take = [&]() {    // the slot, once it is full
    const uint32_t bar = bar_full + 8 * slot;
    if (!__all_sync(0xffffffffu, mbar_try_wait(bar, parity)) && alive)
      alive = __all_sync(0xffffffffu, wait_or_abort(bar, parity, abort, &g_cache_attention_fault));
    return smem + slot * S::kSlotBytes;
  };
  auto give = [&]() {    // every lane has read it; a warp that gave up keeps it, its copy may be under way
    __syncwarp();
    if (lane < static_cast<int>(alive)) mbar_arrive(bar_empty + 8 * slot);
    if (++slot == S::kSlots) slot = 0, parity ^= 1u;
  };

  // the segments of the range: the part of each group that lies in it
  bool first_segment = true;
  while (r.count > 0) {
    const Seq& s = r.s;
    const int count = r.here(), seg_end = r.tile + count;
    const bool whole = r.tile == 0 && count == s.tiles;
    const int kv_head = r.kv_head();
    const int row_tile = r.group - kv_head * s.row_tiles;
    const int tile_row0 = row_tile * S::kRows;
    const int live_rows = s.n * a.group - tile_row0;   // rows of the tile that exist (may be more than it holds)

    // query fragments: lane (g, t) holds elements t * HD/4 .. of row g of each 8-row tile
    uint32_t qf[S::kQShared ? 1 : NT][S::kQShared ? 1 : S::kSteps][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if (S::kQShared && nt != warp) continue;  // the warps share the work
      const int rho = nt * 8 + g;
      const int tok = (tile_row0 + rho) / a.group;
      uint32_t w[HD / 8];
      if (rho < live_rows) {
        const int head = kv_head * a.group + (tile_row0 + rho) - tok * a.group;
        const uint16_t* src = a.q + (s.row0 + tok) * a.ld_q + static_cast<int64_t>(head) * HD + t * (HD / 4);
#pragma unroll
        for (int i = 0; i < HD / 32; ++i) {
          const uint4 v = load16_fresh(src + 8 * i);
          w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < HD / 8; ++i) w[i] = 0;
      }
      uint32_t m = magnitude_bits(w);
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
      const float f = query_factor(m);
#pragma unroll
      for (int i = 0; i < HD / 8; ++i) {
        const float2 v = bf16x2_to_float2(w[i]);
        const uint32_t h = half2_of(__fmul_rn(v.x, f), __fmul_rn(v.y, f));
        if constexpr (S::kQShared) {
          reinterpret_cast<uint32_t*>(q_shared)[((nt * S::kSteps + i / 2) * 32 + lane) * 2 + (i & 1)] = h;
        } else {
          qf[nt][i / 2][i & 1] = h;
        }
      }
      if (t == 0) {   // (several warps may write the same values)
        row_factor[rho] = inverse_power(f);
        row_mask[rho] = rho >= live_rows    ? 0
                        : a.mask != nullptr ? static_cast<uint64_t>(a.mask[s.row0 + tok])
                                            : ~uint64_t{0} >> (63 - tok);
      }
    }
    if constexpr (S::kQShared) sync_compute(); else __syncwarp();

    float cf[NT][2];    // x = cf * S of the lane's columns (rows 2t, 2t + 1 of each tile), in units of
                        // log2; never 0, so that a hidden key's -inf stays one
    float m_run[NT][2], l_run[NT][2];
    float acc[NT][S::kSteps][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        cf[nt][i] = fmaxf(__fmul_rn(k_factor, row_factor[nt * 8 + 2 * t + i]), 0x1p-126f);
        m_run[nt][i] = -INFINITY;
        l_run[nt][i] = 0.0f;
      }
#pragma unroll
      for (int i = 0; i < S::kSteps; ++i) acc[nt][i][0] = acc[nt][i][1] = acc[nt][i][2] = acc[nt][i][3] = 0.0f;
    }

    const uint32_t seen_by_all = s.ctx < 0 ? 0 : min(s.ctx, s.len);
    for (int tile = r.tile; alive && tile < seg_end; ++tile) {
      // this warp's keys of the tile; -1: none of them is in the sequence
      const uint32_t first_key = static_cast<uint32_t>(tile) * S::kKeys + warp * S::kWarpKeys;
      const bool work = first_key < static_cast<uint32_t>(s.len);
      // Scores and weights of all the warp's keys (kept as the right operand of the second
      // product), 16 * kMt keys at a time.
      uint32_t pf[S::kWarpKeys / 16][NT][2];
      const uint8_t* kc = take();
      if (work) {
        const uint8_t* ks = kc + S::kCodeBytes + warp * S::kWarpKeys * (HD / 16);
        kc += warp * S::kWarpKeys * (HD / 2);
#pragma unroll
        for (int sub = 0; sub < S::kWarpKeys / 16; sub += S::kMt) {
          const uint32_t key0 = first_key + 16 * sub;
          // S^T: rows of the left operand are keys 4 (g / 2) + g % 2 and that + 2, so that the
          // values' operand below finds its four keys 4t .. 4t + 3 side by side
          float sc[S::kMt][NT][4];
#pragma unroll
          for (int mt = 0; mt < S::kMt; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) sc[mt][nt][0] = sc[mt][nt][1] = sc[mt][nt][2] = sc[mt][nt][3] = 0.0f;
#pragma unroll
          for (int mt = 0; mt < S::kMt; ++mt) {
            const int r0 = (sub + mt) * 16 + 4 * (g >> 1) + (g & 1);
            uint32_t w0[HD / 32], w1[HD / 32];
            lds<HD / 8>(kc + r0 * (HD / 2) + t * (HD / 8), w0);
            lds<HD / 8>(kc + (r0 + 2) * (HD / 2) + t * (HD / 8), w1);
            uint32_t b0, b1;    // the lane's HD / 64 scale bytes of both keys
            if constexpr (HD == 64) {
              b0 = ks[r0 * 4 + t];
              b1 = ks[(r0 + 2) * 4 + t];
            } else if constexpr (HD == 128) {
              b0 = *reinterpret_cast<const uint16_t*>(ks + r0 * 8 + t * 2);
              b1 = *reinterpret_cast<const uint16_t*>(ks + (r0 + 2) * 8 + t * 2);
            } else {
              b0 = *reinterpret_cast<const uint32_t*>(ks + r0 * 16 + t * 4);
              b1 = *reinterpret_cast<const uint32_t*>(ks + (r0 + 2) * 16 + t * 4);
            }
#pragma unroll
            for (int w = 0; w < HD / 32; ++w) {   // a word: 8 codes, two steps of 4; 16 codes share a scale
              const uint32_t f0 = scale_half(b0 >> (8 * (w >> 1))) * 0x10001u;
              const uint32_t f1 = scale_half(b1 >> (8 * (w >> 1))) * 0x10001u;
              uint32_t h0[4], h1[4];
              codes_to_half(w0[w], h0);
              codes_to_half(w1[w], h1);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                h0[i] = hmul2(h0[i], f0);
                h1[i] = hmul2(h1[i], f1);
              }
#pragma unroll
              for (int half = 0; half < 2; ++half)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  uint32_t qb0, qb1;
                  if constexpr (S::kQShared) {
                    const uint2 v = q_shared[(nt * S::kSteps + 2 * w + half) * 32 + lane];
                    qb0 = v.x, qb1 = v.y;
                  } else {
                    qb0 = qf[nt][2 * w + half][0], qb1 = qf[nt][2 * w + half][1];
                  }
                  mma(sc[mt][nt], h0[2 * half], h1[2 * half], h0[2 * half + 1], h1[2 * half + 1], qb0, qb1);
                }
            }
          }

          // keys that a row does not see
          if (key0 + 16 * S::kMt > seen_by_all) {
#pragma unroll
            for (int mt = 0; mt < S::kMt; ++mt)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const int64_t key = static_cast<int64_t>(key0) + mt * 16 + 4 * (g >> 1) + (g & 1) + (i & 2);
                  const int64_t draft = key - s.ctx;
                  const uint64_t bits = row_mask[nt * 8 + 2 * t + (i & 1)];
                  const bool seen = key < s.len && (draft < 0 || (draft < 64 && ((bits >> draft) & 1)));
                  if (!seen) sc[mt][nt][i] = -INFINITY;
                }
          }

          // running maximum and sum, and the weights
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float top[2];   // of the lane's keys, in units of log2
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float m = fmaxf(sc[0][nt][i], sc[0][nt][i + 2]);
#pragma unroll
              for (int mt = 1; mt < S::kMt; ++mt) m = max3(m, sc[mt][nt][i], sc[mt][nt][i + 2]);
              top[i] = __fmul_rn(m, cf[nt][i]);
            }
            if (__any_sync(0xffffffffu, top[0] > m_run[nt][0] + kSlack || top[1] > m_run[nt][1] + kSlack)) {
              // The reference is a whole number (in units of log2), so what is taken to a new one is multiplied
              // by a power of two: weights that are fp16 already are not rounded again.
              float alpha[2];
              int down[2];   // log2 of alpha, as far as it matters
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                float m = top[i];
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
                m = fmaxf(m_run[nt][i], ceilf(m));
                down[i] = max(__float2int_rz(__fadd_rn(m_run[nt][i], m == -INFINITY ? 0.0f : -m)), -127);
                alpha[i] = power(down[i]);
                l_run[nt][i] = __fmul_rn(l_run[nt][i], alpha[i]);
                m_run[nt][i] = m;
              }
              if constexpr (S::kMt * 16 < S::kWarpKeys) {   // weights of this tile that were formed before
                // row g's factor as two that fp16 holds (below 2^-48 it leaves nothing of a weight)
                const int of0 = __shfl_sync(0xffffffffu, down[0], g >> 1), of1 = __shfl_sync(0xffffffffu, down[1], g >> 1);
                const int e = max(g & 1 ? of1 : of0, -48), half = e / 2;
                const uint32_t a0 = half2_of(power(half), power(half)), a1 = half2_of(power(e - half), power(e - half));
#pragma unroll
                for (int mt = 0; mt < sub; ++mt) {
                  pf[mt][nt][0] = hmul2(hmul2(pf[mt][nt][0], a0), a1);
                  pf[mt][nt][1] = hmul2(hmul2(pf[mt][nt][1], a0), a1);
                }
              }
#pragma unroll
              for (int i = 0; i < S::kSteps; ++i) {
                acc[nt][i][0] = __fmul_rn(acc[nt][i][0], alpha[0]);
                acc[nt][i][1] = __fmul_rn(acc[nt][i][1], alpha[1]);
                acc[nt][i][2] = __fmul_rn(acc[nt][i][2], alpha[0]);
                acc[nt][i][3] = __fmul_rn(acc[nt][i][3], alpha[1]);
              }
            }
            const float2 c2 = make_float2(cf[nt][0], cf[nt][1]);
            const float2 b2 = make_float2(__fadd_rn(kInShift, m_run[nt][0] == -INFINITY ? 0.0f : -m_run[nt][0]),
                                          __fadd_rn(kInShift, m_run[nt][1] == -INFINITY ? 0.0f : -m_run[nt][1]));
            float2 add = make_float2(l_run[nt][0], l_run[nt][1]);
#pragma unroll
            for (int mt = 0; mt < S::kMt; ++mt) {
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                float2 p = fma2(make_float2(sc[mt][nt][2 * i], sc[mt][nt][2 * i + 1]), c2, b2);
                p.x = ex2(p.x);
                p.y = ex2(p.y);
                add = add2(add, p);
                pf[sub + mt][nt][i] = transpose8x8(half2_of(p.x, p.y));
              }
            }
            l_run[nt][0] = add.x;
            l_run[nt][1] = add.y;
          }
        }
      }
      give();

      // O^T: lane (g, t) holds columns g * HD/8 .. of keys 4t .. 4t + 3
      const uint8_t* vc = take();
      if (work) {
        const uint8_t* vs = vc + S::kCodeBytes + warp * S::kWarpKeys * (HD / 16);
        vc += warp * S::kWarpKeys * (HD / 2);
#pragma unroll
        for (int mt = 0; mt < S::kWarpKeys / 16; ++mt) {
          uint32_t w[4][HD / 64];
          uint32_t f[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int key = mt * 16 + 4 * t + k;
            lds<HD / 16>(vc + key * (HD / 2) + g * (HD / 16), w[k]);
            if constexpr (HD == 64)
              f[k] = vs[key * 4 + (g >> 1)];
            else if constexpr (HD == 128)
              f[k] = vs[key * 8 + g];
            else
              f[k] = *reinterpret_cast<const uint16_t*>(vs + key * 16 + g * 2);
          }
#pragma unroll
          for (int j = 0; j < HD / 64; ++j) {   // a word: 8 columns of each key
            const int sh = HD == 256 ? 8 * (j >> 1) : 0;
            const uint32_t f01 = scale_half(f[0] >> sh) | scale_half(f[1] >> sh) << 16;
            const uint32_t f23 = scale_half(f[2] >> sh) | scale_half(f[3] >> sh) << 16;
            // bytes of (first key's, second key's) codes of the even and of the odd columns
            const uint32_t e01 = (w[0][j] & 0x0f0f0f0fu) | ((w[1][j] << 4) & 0xf0f0f0f0u);
            const uint32_t o01 = ((w[0][j] >> 4) & 0x0f0f0f0fu) | (w[1][j] & 0xf0f0f0f0u);
            const uint32_t e23 = (w[2][j] & 0x0f0f0f0fu) | ((w[3][j] << 4) & 0xf0f0f0f0u);
            const uint32_t o23 = ((w[2][j] >> 4) & 0x0f0f0f0fu) | (w[3][j] & 0xf0f0f0f0u);
            uint32_t a0[4], a1[4], a2[4], a3[4];
            codes_to_half(e01, a0);
            codes_to_half(o01, a1);
            codes_to_half(e23, a2);
            codes_to_half(o23, a3);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              a0[i] = hmul2(a0[i], f01);
              a1[i] = hmul2(a1[i], f01);
              a2[i] = hmul2(a2[i], f23);
              a3[i] = hmul2(a3[i], f23);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma(acc[nt][4 * j + i], a0[i], a1[i], a2[i], a3[i], pf[mt][nt][0], pf[mt][nt][1]);
            }
          }
        }
      }
      give();
    }

    // ---- join the warps, eight rows at a time; write the outputs or leave the part
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float l = l_run[nt][i];
        l = __fadd_rn(l, __shfl_xor_sync(0xffffffffu, l, 4));
        l = __fadd_rn(l, __shfl_xor_sync(0xffffffffu, l, 8));
        l = __fadd_rn(l, __shfl_xor_sync(0xffffffffu, l, 16));
        if (g == 0) join_ml[warp * 8 + 2 * t + i] = make_float2(m_run[nt][i], l);
      }
      {
        float* dst = join + warp * 8 * S::kPitch + g * (HD / 8);
#pragma unroll
        for (int i = 0; i < S::kSteps; ++i) {
          *reinterpret_cast<float2*>(dst + (2 * t) * S::kPitch + 2 * i) = make_float2(acc[nt][i][0], acc[nt][i][2]);
          *reinterpret_cast<float2*>(dst + (2 * t + 1) * S::kPitch + 2 * i) =
              make_float2(acc[nt][i][1], acc[nt][i][3]);
        }
      }
      sync_compute();
      {
        constexpr int kPer = HD / 16;        // columns per thread, 16 threads a row
        const int row = threadIdx.x >> 4, c0 = (threadIdx.x & 15) * kPer;
        const int rho = nt * 8 + row;
        if (rho < live_rows && !raised_here(abort)) {   // (a warp that has given up raised it before the barrier above)
          float m = -INFINITY;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) m = fmaxf(m, join_ml[w * 8 + row].x);
          const float use = m == -INFINITY ? 0.0f : m;
          float l = 0.0f, v[kPer];
#pragma unroll
          for (int i = 0; i < kPer; ++i) v[i] = 0.0f;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float2 ml = join_ml[w * 8 + row];
            const float f = ex2(__fadd_rn(__fadd_rn(ml.x, -use), kPShift - kInShift));
            l = __fmaf_rn(ml.y, f, l);
#pragma unroll
            for (int i = 0; i < kPer; i += 4) {
              const float4 x = *reinterpret_cast<const float4*>(join + (w * 8 + row) * S::kPitch + c0 + i);
              v[i] = __fmaf_rn(x.x, f, v[i]);
              v[i + 1] = __fmaf_rn(x.y, f, v[i + 1]);
              v[i + 2] = __fmaf_rn(x.z, f, v[i + 2]);
              v[i + 3] = __fmaf_rn(x.w, f, v[i + 3]);
            }
          }
          const int tok = (tile_row0 + rho) / a.group;
          const int head = kv_head * a.group + (tile_row0 + rho) - tok * a.group;
          const int64_t out_row = s.row0 + tok;
          if (whole) {
            const float f = l == 0.0f ? 0.0f : __fdiv_rn(1.0f, l);   // (v_factor / l may be too small for fp32)
            uint32_t w[kPer / 2];
#pragma unroll
            for (int i = 0; i < kPer / 2; ++i)
              w[i] = float2_to_bf16x2(make_float2(__fmul_rn(__fmul_rn(v[2 * i], f), v_factor),
                                                  __fmul_rn(__fmul_rn(v[2 * i + 1], f), v_factor)));
            uint16_t* dst = a.o + (out_row * a.heads + head) * HD + c0;
            if constexpr (kPer == 4) {
              *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
            } else {
#pragma unroll
              for (int i = 0; i < kPer / 8; ++i)
                store16(dst + 8 * i, make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]));
            }
            if (a.lse != nullptr && c0 == 0)
              a.lse[head * a.rows + out_row] =
                  l == 0.0f ? -INFINITY : __fmul_rn(__fadd_rn(m, __fadd_rn(log2f(l), -kPShift)), kLn2);
          } else {
            const int64_t slot = static_cast<int64_t>(blockIdx.x) * 2 + (first_segment ? 0 : 1);
            float* dst = a.part + (slot * S::kRows + rho) * HD + c0;
#pragma unroll
            for (int i = 0; i < kPer; i += 4)
              *reinterpret_cast<float4*>(dst + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
            if (c0 == 0) reinterpret_cast<float2*>(a.part_ml)[slot * S::kRows + rho] = make_float2(m, l);
          }
        }
      }
      sync_compute();
    }
    first_segment = false;
    r.advance(a, count, S::kRows, S::kKeys);
  }
}

template <int HD, int NT>
cudaError_t launch(Args a, uint8_t* workspace, cudaStream_t stream) {
  using S = Shape<HD, NT>;
  static_assert(S::kSmem <= 227 * 1024, "shared memory");
  static_assert(!S::kQShared || NT <= kWarps, "a warp loads at most one 8-row tile of queries");
  int blocks = 0;
  cudaError_t err = persistent_blocks(reinterpret_cast<const void*>(&cache_attention_kernel<HD, NT>), S::kThreads,
                                      S::kSmem, kCacheAttentionMaxCtas, &blocks);
  if (err != cudaSuccess) return err;
  place_workspace(a, workspace, kCacheAttentionMaxCtas, S::kRows);
  a.whole = whole_groups(a, blocks, S::kRows, S::kKeys);
  err = launch_early(&cache_attention_kernel<HD, NT>, blocks, S::kThreads, S::kSmem, stream, a);
  if (err != cudaSuccess || blocks < 2 || a.whole) return err;
  return launch_join<HD, S::kRows, S::kKeys>(a, blocks, stream);
}

// Rows that share a key head are taken 8, 16, 24 or 32 at a time: the fewest that hold them
// all, so the cache is read once for up to 32 rows (16 at head_dim 256, where the
// outputs of 32 would not fit the registers).  64 sequences of 4,503 positions at head_dim 128: 66, 104,
// 141 and 213 us (20 rows as 32: 192).  More than kWideRows go to the tcgen05 kernel, which takes 201 and 200 us
// for 28 and for 32 of them where this one takes 196 and 213 (148 and 141 against 113 at head_dim 64).
constexpr int kWideRows = 32;
template <int HD>
cudaError_t dispatch(const Args& a, uint8_t* workspace, cudaStream_t stream) {
  const int64_t rows = static_cast<int64_t>(a.max_rows) * a.group;
  if (rows <= 8) return launch<HD, 1>(a, workspace, stream);
  if constexpr (HD == 256) return launch<HD, 2>(a, workspace, stream);
  else
    return rows <= 16          ? launch<HD, 2>(a, workspace, stream)
           : rows <= 24        ? launch<HD, 3>(a, workspace, stream)
           : rows <= kWideRows ? launch<HD, 4>(a, workspace, stream)
                               : launch_cache_attention_wide(a, workspace, stream);
}

}  // namespace

cudaError_t launch_cache_attention(const PagedCache& cache, const PagedRows& at, const uint16_t* q, int64_t ld_q,
                                   int64_t rows, int heads, int max_rows, const int64_t* mask, const float* k_gsf,
                                   const float* v_gsf, float scale, uint16_t* o, float* lse, uint8_t* workspace,
                                   cudaStream_t stream) {
  Args a{};
  a.cache = cache;
  a.at = at;
  a.q = q;
  a.ld_q = ld_q;
  a.rows = rows;
  a.heads = heads;
  a.group = heads / cache.kv_heads;
  a.max_rows = max_rows;
  a.mask = mask;
  a.k_gsf = k_gsf;
  a.v_gsf = v_gsf;
  a.scale = scale;
  a.o = o;
  a.lse = lse;
  switch (cache.head_dim) {
    case 64: return dispatch<64>(a, workspace, stream);
    case 128: return dispatch<128>(a, workspace, stream);
    default: return dispatch<256>(a, workspace, stream);
  }
}

cudaError_t cache_attention_error_flag(int* flag) {
  int zero = 0, wide = 0;
  cudaError_t err = cudaMemcpyFromSymbol(flag, g_cache_attention_fault, sizeof(int));
  if (err == cudaSuccess) err = cudaMemcpyToSymbol(g_cache_attention_fault, &zero, sizeof(int));
  if (err == cudaSuccess) err = cache_attention_wide_error_flag(&wide);
  *flag |= wide;
  return err;
}

}  // namespace h3q
