// attention.cu -- softmax attention over whole packed sequences (prompts, chunks of
// prompts over their prefixes, the tokens of video frames) on the fifth-generation tensor
// cores.
//
// Per row (a query token and one of its heads): x_j = scale * q . k_j over the keys that
// it sees, o = sum_j e^(x_j - m) v_j / sum_j e^(x_j - m).  One pass over the keys
// with the running maximum and sum; x and the weights never leave the SM.
//
// Bound: the tensor cores, 4 * head_dim operations per row and key seen.  A
// clock of an SM holds 4,096 multiply-adds, 32 powers of two (sm_103a: the special
// function units do twice sm_100's) and 128 lanes of everything else, so 256 rows by
// 128 keys at head_dim 128 are 2,048 clocks of products, 1,024 of powers and about
// 900 of the rest: the products set the pace if everything else runs beside them.
//
// A CTA takes two tiles of up to 128 rows (one at head_dim 256) of one group
// of query heads that share a key head: a row tile is `tokens` tokens x `heads_per_tile`
// heads, so a key tile serves the whole group, a short sequence of grouped heads fills
// its tiles, and the masked corner of a causal tile is `tokens` wide, not 128.
// While the softmax of one tile runs, the tensor cores work on the other.
//
//   warps 0..3, 4..7  softmax of tile 0, 1: a thread owns one row of S in TMEM.  It
//                     reads the row, takes the weights against a reference that follows the
//                     row's maximum only when that has grown by more than 2^8 (the
//                     output is rescaled rarely, and the powers do not wait for the
//                     maximum), writes them as bf16 over S in two halves, and sums
//                     them in fp32 unrounded.  A weight's rounding to
//                     bf16 (at most 2^-8 of it, the type of V that it is multiplied with) is
//                     the format's; maxima, sums and outputs are fp32.  At the end
//                     it scales its row of O and stores it.
//   warp 8, one lane  TMA: Q once, then K and V tiles in a ring
//   warp 9            the products: S = Q K^T (operands in shared memory), O += P V (P in
//                     TMEM, V as it lies in memory: its rows are the reduction)
//   warp 10           only where an output came out as no number: 0 * NaN in the tiles of V that
//                     some row does not see whole (keys to come, rows of the next sequence) can
//                     have done that, so the unit is taken again with those tiles cleaned first.
//                     Rows past the sequence's end become zero, and so do values that are no
//                     numbers; the epilogue adds these back for the rows that see them.
//                     (Every such tile looked at, the products waited 1 to 3 us a unit.)
//   warp 11           the plan: which unit is next.  The CTA's own block first, then those of
//                     blocks that have not started, which it takes over from the launch
//
// Measured: four frames of 2,040 tokens, 56 heads of 128, 1.26 ms (1.52 PFLOP/s at the power
// limit, where the library's products alone reach 1.70); 16 packed causal prompts, 32 heads over
// 8, 0.218 ms; four chunks over their prefixes 0.203 ms (2.6 units a CTA, so a third of it is
// the last ones' time).  A pair of tiles takes about 2,750 clocks: 1,235 from S to the weights,
// the products' own, and the two warps' notices to each other.
//
// Every wait is bounded: one that runs out sets a device flag and tells the other roles
// to stop; the CTA drains what it has in flight, frees its TMEM and returns.
#include <cmath>

#include "h3q_async.cuh"
#include "h3q_device.cuh"
#include "h3q_internal.h"
#include "h3q_roles.cuh"
#include "h3q_softmax.cuh"
#include "h3q_tcgen05.cuh"
#include "h3q_units.h"

namespace h3q {
namespace {

constexpr int kThreads = 384;
constexpr int kTmaWarp = 8;
constexpr int kMmaWarp = 9;
constexpr int kCheckWarp = 10;
constexpr int kSlots = 3;        // units known ahead
constexpr int kTileRows = 128;
constexpr float kSlack = 8.0f;  // a row's reference moves when its maximum has passed it by 2^8,
constexpr float kJump = 16.0f;  // at once when a tile passes it by 2^16: over 2^25 keys the sums of weights stay
                                // below 2^41, those of weights and values finite for values up to 2^86

__device__ int g_attention_fault;

struct Args {
  const int32_t* cu_q;
  const int32_t* cu_k;
  int batch;
  int64_t rows_q, rows_k;
  int heads, group;          // query heads, and per key head
  int heads_per_tile, tokens, tile_groups;  // a row tile: tokens x heads_per_tile; tile_groups of heads
  int head_chunk;            // tile groups that are swept together (their keys and values stay in L2)
  int causal;
  float scale;
  const uint16_t* v;         // for the values that are no numbers
  int64_t ld_v;
  uint16_t* o;
  float* lse;                // or nullptr
};

template <int HD>
struct Shape {
  static constexpr int kTiles = HD == 256 ? 1 : 2;      // row tiles per CTA
  static constexpr int kKeys = HD == 256 ? 64 : 128;    // keys per tile
  static constexpr int kHalves = HD / 64;               // 64-element (128-byte) column blocks of a row
  static constexpr int kQBytes = kTileRows * HD * 2;
  static constexpr int kKvBytes = kKeys * HD * 2;
  static constexpr int kStages = 4;                     // K and V tiles in the ring (even: V tiles take every other)
  static constexpr int kOffKv = kTiles * kQBytes;
  static constexpr int kOffOut = kOffKv + kStages * kKvBytes;   // 32 rows x 64 columns of output per softmax warp
  static constexpr int kOffBar = kOffOut + kTiles * 4 * 4096;
  static constexpr int kBars = 4 * kStages + 12 + 2 * kSlots + 4;   // named in the kernel
  static constexpr int kOffMisc = kOffBar + 8 * kBars;    // TMEM address, abort; a taken block's id (16-byte aligned)
  static constexpr int kOffSlots = kOffMisc + 32;
  static constexpr int kSmem = kOffSlots + kSlots * 96 + 1024;
  static_assert(kOffMisc % 16 == 0, "alignment");
  // TMEM: two S buffers (P over them), then O
  static constexpr uint32_t kS = kKeys;                 // columns of an S buffer
  static constexpr uint32_t kO = 256;
  // Instruction descriptors (kind::f16): fp32 result (bit 4), bf16 operands (1 at bits 7-9
  // and 10-12), N >> 3 at bits 17-22, M >> 4 at 24-28; V is transposed (bit 16): its rows
  // run along the reduction.
  static constexpr uint32_t kIdescS = (1u << 4) | (1u << 7) | (1u << 10) | (uint32_t(kKeys >> 3) << 17) | (8u << 24);
  static constexpr uint32_t kIdescO =
      (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | (uint32_t(HD >> 3) << 17) | (8u << 24);
};

__device__ __forceinline__ bool wait_or_abort(uint32_t bar, uint32_t parity, volatile int* abort) {
  return h3q::wait_or_abort(bar, parity, abort, &g_attention_fault);
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// A unit of work: one sequence's pair of row tiles of one group of heads, as the planning
// warp hands it to the others.
struct Unit {
  int64_t q0, k0;        // first packed rows of the sequence
  int n, len;            // its queries and keys; n < 0: no more units
  int head0;             // first head of the tile
  int tok[2];            // first token of each row tile
  int tiles[2];          // key tiles that each reads (0: none, or no rows)
  int partial[2];        // first of them that some row of the tile does not see whole
  int least;             // keys that every row of the unit sees
  int checked;           // the second time round: partial V tiles go through the check warp
  int redo;              // an output was no number
  int bad;               // which V tiles (from the unit's first partial one) held values that are no numbers
};

// Key tiles of the unit, and the first that some row does not see whole (a causal tile 0
// sees less than tile 1).
__device__ __forceinline__ int tiles_of(const Unit& u) { return u.tiles[0] > u.tiles[1] ? u.tiles[0] : u.tiles[1]; }
__device__ __forceinline__ int partial_of(const Unit& u) { return u.tiles[0] == 0 ? u.partial[1] : u.partial[0]; }

__device__ __forceinline__ int clamp_keys(int64_t x, int len) {
  return x < 0 ? 0 : x > len ? len : static_cast<int>(x);
}

template <int HD>
__device__ __forceinline__ void write_unit(const Args& a, int b, int64_t rank, Unit& u) {
  using S = Shape<HD>;
  const int64_t q0 = a.cu_q[b], k0 = a.cu_k[b];
  int64_t n = static_cast<int64_t>(a.cu_q[b + 1]) - q0, len = static_cast<int64_t>(a.cu_k[b + 1]) - k0;
  // (n is in range where it is counted; lists of keys that point past the rows hold none)
  if (n > a.rows_q - q0) n = a.rows_q - q0;
  if (k0 < 0 || len < 0) len = 0;
  if (len > a.rows_k - k0) len = a.rows_k - k0 < 0 ? 0 : a.rows_k - k0;
  u.q0 = q0;
  u.k0 = k0;
  u.n = static_cast<int>(n);
  u.len = static_cast<int>(len);
  const int span = a.tokens * S::kTiles;
  const int64_t q_tiles = (u.n + span - 1) / span;
  const int64_t chunk = rank / (a.head_chunk * q_tiles);
  const int64_t rest = rank - chunk * a.head_chunk * q_tiles;
  const int h0 = static_cast<int>(chunk) * a.head_chunk;
  const int here = a.tile_groups - h0 < a.head_chunk ? a.tile_groups - h0 : a.head_chunk;
  const int qt = static_cast<int>(q_tiles - 1 - rest / here);   // the longest rows first
  u.head0 = (h0 + static_cast<int>(rest % here)) * a.heads_per_tile;
  const int64_t shift = static_cast<int64_t>(u.len) - u.n + 1;  // token t sees keys below t + shift
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int tok = qt * span + x * a.tokens;
    const bool any = x < S::kTiles && tok < u.n;
    const int last = tok + a.tokens < u.n ? tok + a.tokens - 1 : u.n - 1;
    const int most = !any ? 0 : a.causal ? clamp_keys(last + shift, u.len) : u.len;
    const int least = a.causal ? clamp_keys(tok + shift, u.len) : u.len;
    u.tok[x] = tok;
    u.tiles[x] = (most + S::kKeys - 1) / S::kKeys;
    u.partial[x] = least / S::kKeys;
    if (x == 0 || u.tiles[0] == 0) u.least = least;
  }
  u.checked = u.redo = u.bad = 0;
}

__device__ __forceinline__ int64_t units_of(const Args& a, int b, int span) {
  const int64_t q0 = a.cu_q[b];
  int64_t n = static_cast<int64_t>(a.cu_q[b + 1]) - q0;
  if (n > a.rows_q - q0) n = a.rows_q - q0;
  if (q0 < 0 || n < 0) n = 0;
  return (n + span - 1) / span * a.tile_groups;
}

// 16 scores -> weights 2^(s * c + base), packed to bf16, and their sum added.
__device__ __forceinline__ void weights16(const uint32_t* s, float2 c2, float2 b2, float2& sum, uint32_t* w) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float2 p = fma2(make_float2(__uint_as_float(s[2 * j]), __uint_as_float(s[2 * j + 1])), c2, b2);
    p.x = ex2(p.x);
    p.y = ex2(p.y);
    sum = add2(sum, p);
    w[j] = float2_to_bf16x2(p);
  }
}

template <int HD>
__global__ void __launch_bounds__(kThreads, 1)
attention_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                 const __grid_constant__ CUtensorMap map_v, const Args a) {
  using S = Shape<HD>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t{1023});
  const uint32_t base = smem_u32(smem);
  const uint32_t bar_full = base + S::kOffBar;             // + 8 * stage
  const uint32_t bar_empty = bar_full + 8 * S::kStages;
  const uint32_t bar_vraw = bar_empty + 8 * S::kStages;    // a V tile that the check warp looks at first ...
  const uint32_t bar_vok = bar_vraw + 8 * S::kStages;      // ... and has passed on
  const uint32_t bar_q = bar_vok + 8 * S::kStages;         // + 8 * row tile: Q has landed,
  const uint32_t bar_qfree = bar_q + 16;                   // is no longer read
  const uint32_t bar_s = bar_qfree + 16;                   // + 8 * S buffer
  const uint32_t bar_p = bar_s + 16;
  const uint32_t bar_p2 = bar_p + 16;                      // the weights of the second half of a tile's keys
  const uint32_t bar_o = bar_p2 + 16;                      // + 8 * row tile
  const uint32_t bar_unit = bar_o + 16;                    // + 8 * slot: a unit is there,
  const uint32_t bar_slot = bar_unit + 8 * kSlots;         // all have read it
  const uint32_t bar_next = bar_slot + 8 * kSlots;         // a waiting block was taken over, or none was left
  const uint32_t bar_want = bar_next + 8;                  // the loads of a unit are about to end
  const uint32_t bar_drain = bar_want + 8;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::kOffMisc);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + S::kOffMisc + 4);
  const uint32_t next_block_at = base + S::kOffMisc + 16;
  Unit* units = reinterpret_cast<Unit*>(smem + S::kOffSlots);
  static_assert(sizeof(Unit) <= 96, "slots");
  constexpr int kReaders = 4 * S::kTiles + 3;   // warps that read a slot: softmax, TMA, products, check
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(bar_full + 8 * i, 1);
      mbar_init(bar_empty + 8 * i, 1);
      mbar_init(bar_vraw + 8 * i, 1);
      mbar_init(bar_vok + 8 * i, 32);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar_q + 8 * i, 1);
      mbar_init(bar_qfree + 8 * i, 1);
      mbar_init(bar_s + 8 * i, 1);
      mbar_init(bar_p + 8 * i, kTileRows);
      mbar_init(bar_p2 + 8 * i, kTileRows);
      mbar_init(bar_o + 8 * i, 1);
    }
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(bar_unit + 8 * i, 1);
      mbar_init(bar_slot + 8 * i, kReaders);
    }
    mbar_init(bar_next, 1);
    mbar_init(bar_want, 1);
    mbar_init(bar_drain, 1);
    *abort = 0;
    mbar_init_fence();
  }
  __syncthreads();

  // The unit number `it` of this CTA, or nullptr after the last (or an abort).  Whole warp.
  auto unit_at = [&](int it) -> Unit* {
    const int slot = it % kSlots;
    if (!__all_sync(0xffffffffu, wait_or_abort(bar_unit + 8 * slot, (it / kSlots) & 1, abort))) return nullptr;
    return units[slot].n < 0 ? nullptr : units + slot;
  };
  auto leave_unit = [&](int it) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar_slot + 8 * (it % kSlots));
  };

  // (384 threads have 168 registers each.  A split by setmaxnreg, 208 for the softmax warps and
  // 88 for the others, was no faster: 1.32 ms both ways at 8,160 x 56 heads.)
  if (warp < kTmaWarp) {
    if (warp < 4 * S::kTiles) {
      // ---- softmax and epilogue of one row tile
      const int x = warp >> 2;
      const int row = (warp & 3) * 32 + lane;
      const int row_tok = row / a.heads_per_tile, row_head = row % a.heads_per_tile;
      const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;   // the TMEM of all 512 columns begins at 0
      const uint32_t taddr_o = lane_base + S::kO + x * HD;
      const float c = fmaxf(__fmul_rn(a.scale, kLog2e), 0x1p-126f);   // never 0: a hidden key's -inf stays one
      uint8_t* staged = smem + S::kOffOut + warp * 4096;
      uint32_t s_count = 0, o_count = 0;   // S tiles and outputs waited for
      bool ok = true;
      Unit* u;
      for (int it = 0; ok && (u = unit_at(it)) != nullptr; ++it) {
        const int tok = u->tok[x] + row_tok;
        const bool valid = row < a.tokens * a.heads_per_tile && tok < u->n;
        const int len = u->len;
        const int sees = !valid ? 0 : a.causal ? clamp_keys(static_cast<int64_t>(tok) + len - u->n + 1, len) : len;
        const int n = u->tiles[x], partial = u->partial[x];
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
        for (int j = 0; j < n; ++j) {
          const int buf = S::kTiles == 2 ? x : s_count & 1;
          const uint32_t parity = S::kTiles == 2 ? s_count & 1 : (s_count >> 1) & 1;
          if (!(ok = __all_sync(0xffffffffu, wait_or_abort(bar_s + 8 * buf, parity, abort)))) break;
          ++s_count;
          // O is at rest: with two tiles S[j] was issued after P[j-1] V[j-1]; with one it was
          // issued before, so that product is waited for (each in turn: a phase that is two
          // behind looks like one to come).
          if constexpr (S::kTiles == 1) {
            if (j > 0) {
              if (!(ok = __all_sync(0xffffffffu, wait_or_abort(bar_o, o_count & 1, abort)))) break;
              ++o_count;
            }
          }
          tc_fence_after();
          const uint32_t taddr = lane_base + buf * S::kS;
          if (j > 0 && __any_sync(0xffffffffu, __fmul_rn(__fadd_rn(m_seen, -m_ref), c) > kSlack)) rescale(true);
          constexpr int kHalf = S::kKeys / 2;
          const int seen = sees - j * S::kKeys;
          const bool masked = j >= partial;
          const float2 c2 = make_float2(c, c);
          uint32_t s[S::kKeys / 32][32];
          uint32_t w[kHalf / 2];
          float2 sum;
          // The weights of this tile are taken against the reference as it is, while the tile's
          // maximum is still being formed; only where a row passes it by 2^kJump is the reference
          // moved at once and the tile read again.
          bool fresh = j == 0;   // no reference yet: only the maximum is formed
          for (;;) {
#pragma unroll
            for (int i = 0; i < S::kKeys / 32; ++i) tc_load32(taddr + 32 * i, s[i]);
            tc_wait_load(s[0]);
#pragma unroll
            for (int i = 1; i < S::kKeys / 32; ++i) tc_loaded(s[i]);
            if (masked) {
#pragma unroll
              for (int i = 0; i < S::kKeys; ++i)
                if (i >= seen) s[i / 32][i % 32] = 0xff800000u;
            }
            float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int i = 0; i < S::kKeys; i += 8)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                m[k] = max3(m[k], __uint_as_float(s[i / 32][i % 32 + 2 * k]), __uint_as_float(s[i / 32][i % 32 + 2 * k + 1]));
            if (fresh) {
              fresh = false;
              m_seen = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
              rescale(false);
              continue;
            }
            const float base = m_ref == -INFINITY ? 0.0f : -__fmul_rn(m_ref, c);
            const float2 b2 = make_float2(base, base);
            sum = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < kHalf; i += 16) weights16(s[i / 32] + i % 32, c2, b2, sum, w + i / 2);
            m_seen = fmaxf(max3(m_seen, m[0], m[1]), fmaxf(m[2], m[3]));
            // (a difference of two -inf is no number, and not above)
            if (!__any_sync(0xffffffffu, __fmul_rn(__fadd_rn(m_seen, -m_ref), c) > kJump)) break;
            rescale(j > 0);
          }
          const float base = m_ref == -INFINITY ? 0.0f : -__fmul_rn(m_ref, c);
          const float2 b2 = make_float2(base, base);
          store_weights<kHalf / 2>(taddr, w);
          tc_wait_store();
          tc_fence_before();
          mbar_arrive(bar_p + 8 * buf);            // the products of the first half of the keys may start
#pragma unroll
          for (int i = 0; i < kHalf; i += 16)
            weights16(s[(kHalf + i) / 32] + i % 32, c2, b2, sum, w + i / 2);
          store_weights<kHalf / 2>(taddr + kHalf / 2, w);
          l = __fadd_rn(l, __fadd_rn(sum.x, sum.y));
          tc_wait_store();
          tc_fence_before();
          mbar_arrive(bar_p2 + 8 * buf);
        }
        if (n > 0 && ok) {
          ok = __all_sync(0xffffffffu, wait_or_abort(bar_o + 8 * x, o_count & 1, abort));
          ++o_count;
          tc_fence_after();
        }
        if (ok) {
          // The row of O, scaled, through shared memory (the 16-byte pieces of a row in the order of
          // their number's exclusive or with the row's, so that no two rows' meet in a bank), 128
          // bytes of a row at a time, and out eight lanes a row.  (A thread that stores its own row
          // takes a transaction per 16 bytes: 2.8 us a unit, against 0.7.)
          const float inv = l == 0.0f ? 0.0f : __fdiv_rn(1.0f, l);
          const int64_t out_row = u->q0 + tok;
          const int head = u->head0 + row_head;
          const int bad = *static_cast<volatile int*>(&u->bad);
          const unsigned long long dst =
              valid ? reinterpret_cast<unsigned long long>(a.o + (out_row * a.heads + head) * HD) : 0ull;
          float2 odd = make_float2(0.0f, 0.0f);   // no number if an output is none
#pragma unroll 1
          for (int i = 0; i < HD; i += 64) {
            uint32_t o[2][32];
            if (n > 0) {
              __syncwarp();
              tc_load32(taddr_o + i, o[0]);
              tc_load32(taddr_o + i + 32, o[1]);
              tc_wait_load(o[0]);
              tc_loaded(o[1]);
            } else {
#pragma unroll
              for (int k = 0; k < 64; ++k) o[k / 32][k % 32] = 0;
            }
            if (bad != 0 && valid) {   // values that are no numbers, of keys that this row sees
              const int first = partial_of(*u), from = u->least, kv_head = u->head0 / a.group;
              for (int j = first; j < n; ++j) {
                if (!(bad >> (j - first) & 1)) continue;
                const int end = sees < (j + 1) * S::kKeys ? sees : (j + 1) * S::kKeys;
                for (int key = j * S::kKeys > from ? j * S::kKeys : from; key < end; ++key) {
                  const uint16_t* src = a.v + (u->k0 + key) * a.ld_v + static_cast<int64_t>(kv_head) * HD + i;
#pragma unroll
                  for (int k = 0; k < 64; ++k) {
                    const uint32_t w = src[k];
                    if ((w & 0x7f80u) == 0x7f80u)
                      o[k / 32][k % 32] =
                          __float_as_uint(__fadd_rn(__uint_as_float(o[k / 32][k % 32]), __uint_as_float(w << 16)));
                  }
                }
              }
            }
#pragma unroll
            for (int piece = 0; piece < 8; ++piece) {
              uint32_t w[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint32_t* pair = o[piece / 4] + piece % 4 * 8 + 2 * k;
                const float2 y = make_float2(__uint_as_float(pair[0]), __uint_as_float(pair[1]));
                odd = fma2(y, make_float2(0.0f, 0.0f), odd);
                w[k] = l == 0.0f ? 0u : float2_to_bf16x2(mul2(y, make_float2(inv, inv)));
              }
              *reinterpret_cast<uint4*>(staged + lane * 128 + ((piece ^ (lane & 7)) << 4)) =
                  make_uint4(w[0], w[1], w[2], w[3]);
            }
            __syncwarp();
            uint4 v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const int r = 4 * k + (lane >> 3), piece = lane & 7;
              v[k] = *reinterpret_cast<const uint4*>(staged + r * 128 + ((piece ^ (r & 7)) << 4));
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const unsigned long long to = __shfl_sync(0xffffffffu, dst, 4 * k + (lane >> 3));
              if (to != 0) store16(reinterpret_cast<uint16_t*>(to) + i + 8 * (lane & 7), v[k]);
            }
            __syncwarp();
          }
          const float odd_sum = __fadd_rn(odd.x, odd.y);
          if (valid && odd_sum != odd_sum && u->checked == 0 && partial_of(*u) < tiles_of(*u))
            *static_cast<volatile int*>(&u->redo) = 1;
          if (valid && a.lse != nullptr)
            a.lse[head * a.rows_q + out_row] =
                l == 0.0f ? -INFINITY : __fmul_rn(__fadd_rn(__fmul_rn(m_ref, c), log2f(l)), kLn2);
          tc_fence_before();   // O has been read before the next unit's first weights are announced
        }
        leave_unit(it);
      }
    }
  } else if (warp == kTmaWarp) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_q)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_k)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_v)) : "memory");
    const int rows = a.tokens * a.heads_per_tile;
    bool ok = true;
    uint32_t pos = 0;                            // tiles issued: K0 V0 K1 V1 ..., unit after unit
    uint32_t q_count[2] = {0, 0};                // Q tiles issued
    uint32_t full_phase = 0, raw_phase = 0;      // per stage: the phases of its full and v_raw barriers
    uint32_t last_raw = 0;                       // per stage: its last tile went to the check warp
    Unit* u;
    for (int it = 0; ok && (u = unit_at(it)) != nullptr; ++it) {
      const int tiles = tiles_of(*u), partial = partial_of(*u), kv_head = u->head0 / a.group;
      const int row_q0 = static_cast<int>(u->q0), row_k0 = static_cast<int>(u->k0), head0 = u->head0;
      const int tok[2] = {u->tok[0], u->tok[1]};
      const bool any[2] = {u->tiles[0] > 0, u->tiles[1] > 0}, checked = u->checked != 0;
      leave_unit(it);
      if (lane == 0) {
        auto load_q = [&](int x) {
          if (!any[x]) return true;
          if (!wait_or_abort(bar_qfree + 8 * x, (q_count[x] & 1) ^ 1u, abort)) return false;
          ++q_count[x];
          mbar_expect_tx(bar_q + 8 * x, rows * HD * 2);
          for (int h = 0; h < S::kHalves; ++h)
            tma_load_3d(base + x * S::kQBytes + h * (kTileRows * 128), &map_q, 64 * h, head0, row_q0 + tok[x],
                        bar_q + 8 * x);
          return true;
        };
        if (tiles == 0) mbar_arrive(bar_want);
        ok = load_q(0);
        for (int i = 0; i < 2 * tiles && ok; ++i) {
          if (i == 2 * tiles - 2) mbar_arrive(bar_want);
          const uint32_t stage = pos % S::kStages;
          if (!(ok = wait_or_abort(bar_empty + 8 * stage, ((pos / S::kStages) & 1) ^ 1u, abort))) break;
          const bool raw = checked && (i & 1) && (i >> 1) >= partial;
          const uint32_t bar = (raw ? bar_vraw : bar_full) + 8 * stage;
          last_raw = (last_raw & ~(1u << stage)) | static_cast<uint32_t>(raw) << stage;
          (raw ? raw_phase : full_phase) ^= 1u << stage;
          mbar_expect_tx(bar, S::kKvBytes);
          for (int h = 0; h < S::kHalves; ++h)
            tma_load_3d(base + S::kOffKv + stage * S::kKvBytes + h * (S::kKeys * 128), i & 1 ? &map_v : &map_k, 64 * h,
                        kv_head, row_k0 + (i >> 1) * S::kKeys, bar);
          ++pos;
          if (i == 0 && S::kTiles == 2) ok = load_q(1);
        }
      }
      ok = __shfl_sync(0xffffffffu, static_cast<int>(ok), 0);
    }
    // Before the CTA goes: every stage's last tile is released (the products' commits arrive
    // here); after an abort, every copy issued has landed.
    if (lane == 0) {
      const uint32_t first = pos < S::kStages ? 0 : pos - S::kStages;
      for (uint32_t i = first; i < pos && !raised_here(abort); ++i)
        (void)wait_or_abort(bar_empty + 8 * (i % S::kStages), (i / S::kStages) & 1, abort);
      if (raised_here(abort)) {
        for (uint32_t i = first; i < pos; ++i) {
          const uint32_t stage = i % S::kStages;
          const bool raw = last_raw >> stage & 1;
          (void)wait_bounded((raw ? bar_vraw : bar_full) + 8 * stage, ((raw ? raw_phase : full_phase) >> stage & 1) ^ 1u);
        }
        for (int x = 0; x < S::kTiles; ++x)
          if (q_count[x] > 0) (void)wait_bounded(bar_q + 8 * x, (q_count[x] - 1) & 1);
      }
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // The whole warp allocates the CTA's TMEM (one CTA per SM): all 512 columns, so they begin at 0.
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    // One warp issues both tiles' products, a tile's O and next S after the other's: that
    // order keeps the tiles half a step apart, one in its softmax while the other has the
    // tensor cores.  (A warp for each tile lets them fall into step: both in their softmax,
    // then both waiting for the tensor cores; 8,160 x 56 heads took 1.676 ms against 1.392.)
    const uint32_t q_low = desc_low(base, 16);
    const uint32_t k_low = desc_low(base + S::kOffKv, 16);
    const uint32_t v_low = desc_low(base + S::kOffKv, S::kKeys * 128);   // 64 columns of V, then the next 64
    uint32_t pos0 = 0;                      // ring position of the unit's first K tile
    uint32_t full_phase = 0, ok_phase = 0;  // per stage: phases of the full and v_ok barriers
    uint32_t p_count[2] = {0, 0}, q_count[2] = {0, 0};
    bool ok = true;
    // Each lane waits for a barrier of its own (0: none), the warp for all of them: a wait that
    // is met at once still takes a hundred clocks or more, so what a turn needs is one wait.
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
            atomicExch(&g_attention_fault, 1);
          }
          if (__any_sync(0xffffffffu, late || raised_here(abort))) return false;
        }
      }
    };
    auto wait = [&](uint32_t bar, uint32_t parity) { return wait_lanes(lane == 0 ? bar : 0u, parity); };
    auto stage_of = [&](int i) { return (pos0 + i) % S::kStages; };
    // The barrier of ring tile i and its parity, each tile once.
    auto tile_bar = [&](int i, bool checked, uint32_t& parity) {
      const uint32_t stage = stage_of(i);
      parity = (checked ? ok_phase : full_phase) >> stage & 1;
      (checked ? ok_phase : full_phase) ^= 1u << stage;
      return (checked ? bar_vok : bar_full) + 8 * stage;
    };
    auto wait_tile = [&](int i, bool checked) {
      uint32_t parity;
      const uint32_t bar = tile_bar(i, checked, parity);
      return wait(bar, parity);
    };
    auto s_product = [&](int x, int buf, int j) {   // S[buf] = Q[x] K[j]^T
      const uint32_t q = q_low + x * (S::kQBytes >> 4), k = k_low + stage_of(2 * j) * (S::kKvBytes >> 4);
#pragma unroll
      for (int i = 0; i < HD / 16; ++i)
        mma_ss(buf * S::kS, q + (((i / 4) * (kTileRows * 128) + (i % 4) * 32) >> 4),
               k + (((i / 4) * (S::kKeys * 128) + (i % 4) * 32) >> 4), S::kIdescS, i > 0);
      commit_elected(bar_s + 8 * buf);
    };
    // half of O[x] += P[buf] V[j]
    auto o_half = [&](int x, int buf, int j, int half) {
      const uint32_t v = v_low + stage_of(2 * j + 1) * (S::kKvBytes >> 4);
      tc_fence_after();
#pragma unroll
      for (int i = half * S::kKeys / 32; i < (half + 1) * S::kKeys / 32; ++i)
        // rows of V 16 i ..: two 8-row groups of 1,024 bytes
        mma_ts(S::kO + x * HD, buf * S::kS + 8 * i, v + (i * 2048 >> 4), S::kIdescO, j > 0 || i > 0);
    };
    // each half of the keys as its weights are there
    auto o_product = [&](int x, int buf, int j) {
      const uint32_t parity = p_count[buf]++ & 1;
      if (!wait(bar_p + 8 * buf, parity)) return false;
      o_half(x, buf, j, 0);
      if (!wait(bar_p2 + 8 * buf, parity)) return false;
      o_half(x, buf, j, 1);
      return true;
    };
    auto release = [&](int i) { commit_elected(bar_empty + 8 * stage_of(i)); };
    auto wait_q = [&](int x) { return wait(bar_q + 8 * x, q_count[x]++ & 1); };
    uint32_t s_next = 0;   // (one tile: S buffers in turn)
    Unit* u;
    for (int it = 0; ok && (u = unit_at(it)) != nullptr; ++it) {
      const int tiles = uniform(tiles_of(*u));
      const int partial = uniform(u->checked ? partial_of(*u) : tiles);   // V tiles from here on are checked
      const int n0 = uniform(u->tiles[0]), n1 = uniform(u->tiles[1]);
      leave_unit(it);
      if (tiles == 0) continue;
      if constexpr (S::kTiles == 2) {
        ok = wait_tile(0, false);
        if (ok && n0 > 0 && (ok = wait_q(0))) {
          tc_fence_after();
          s_product(0, 0, 0);
          if (n0 == 1) commit_elected(bar_qfree);
        }
        if (ok && n1 > 0 && (ok = wait_q(1))) {
          tc_fence_after();
          s_product(1, 1, 0);
          if (n1 == 1) commit_elected(bar_qfree + 8);
        }
        if (ok) release(0);
        int held = -1;   // a K tile and the V tile before it whose release waits for the next turn
        auto release_held = [&]() {
          if (held < 0) return;
          release(held - 1);
          if (held < 2 * tiles) release(held);
          held = -1;
        };
        for (int j = 0; j < tiles && ok; ++j) {
          uint32_t v_parity, k_parity = 0;
          const uint32_t v_bar = tile_bar(2 * j + 1, j >= partial, v_parity);
          const uint32_t k_bar = j + 1 < tiles ? tile_bar(2 * j + 2, false, k_parity) : 0u;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int n = x == 0 ? n0 : n1, other = x == 0 ? n1 : n0;
            if (!ok || j >= n) continue;
            // V[j], K[j + 1] and the first half of the weights, all at once
            const uint32_t parity = p_count[x]++ & 1;
            const uint32_t bar = lane == 0 ? bar_p + 8 * x : lane == 1 ? v_bar : lane == 2 ? k_bar : 0u;
            if (!(ok = wait_lanes(bar, lane == 0 ? parity : lane == 1 ? v_parity : k_parity))) continue;
            // Commits go in where the queue of products is short (behind a full one they would
            // keep the warp until it has run), so the turn before left its stages to this one.
            release_held();
            o_half(x, x, j, 0);
            if (!(ok = wait(bar_p2 + 8 * x, parity))) continue;
            o_half(x, x, j, 1);
            if (j + 1 < n) {
              s_product(x, x, j + 1);
              if (j + 2 == n) commit_elected(bar_qfree + 8 * x);
            } else {
              commit_elected(bar_o + 8 * x);
            }
            if (x == 1 || j >= other) held = 2 * j + 2;   // the last of the tiles that read V[j]
          }
        }
        if (ok) release_held();
      } else {
        ok = wait_tile(0, false) && wait_q(0);
        if (ok) {
          tc_fence_after();
          s_product(0, s_next & 1, 0);
          if (tiles == 1) commit_elected(bar_qfree);
          release(0);
        }
        for (int j = 0; j < tiles && ok; ++j) {
          if (j + 1 < tiles) {   // the next S goes into the other buffer while this one's softmax runs
            if (!(ok = wait_tile(2 * j + 2, false))) break;
            tc_fence_after();
            s_product(0, (s_next + 1) & 1, j + 1);
            if (j + 2 == tiles) commit_elected(bar_qfree);
            release(2 * j + 2);
          }
          if (!(ok = wait_tile(2 * j + 1, j >= partial) && (s_next & 1 ? o_product(0, 1, j) : o_product(0, 0, j)))) break;
          ++s_next;
          release(2 * j + 1);
          commit_elected(bar_o);
        }
      }
      pos0 += 2 * tiles;
    }
    // what is issued finishes before the TMEM is freed, whoever gave up and when
    commit_elected(bar_drain);
    (void)wait_bounded(bar_drain, 0);
    __syncwarp();
  } else if (warp == kCheckWarp) {
    uint32_t pos0 = 0, raw_phase = 0;
    bool ok = true;
    Unit* u;
    for (int it = 0; ok && (u = unit_at(it)) != nullptr; ++it) {
      const int tiles = tiles_of(*u), partial = u->checked ? partial_of(*u) : tiles;
      const int from = a.causal ? u->least : u->len;   // only rows that some row of the unit does not see matter
      for (int j = partial; j < tiles; ++j) {
        const uint32_t stage = (pos0 + 2 * j + 1) % S::kStages;
        if (!(ok = __all_sync(0xffffffffu, wait_or_abort(bar_vraw + 8 * stage, raw_phase >> stage & 1, abort)))) break;
        raw_phase ^= 1u << stage;
        uint8_t* v = smem + S::kOffKv + stage * S::kKvBytes;
        const int live = u->len - j * S::kKeys;       // rows of the sequence in this tile
        const int row0 = from - j * S::kKeys > 0 ? from - j * S::kKeys : 0;
        bool bad = false;
#pragma unroll 1
        for (int h = 0; h < S::kHalves; ++h) {
          uint4* col = reinterpret_cast<uint4*>(v + h * (S::kKeys * 128));
#pragma unroll 4
          for (int i = row0 * 8 + lane; i < S::kKeys * 8; i += 32) {   // 128 bytes of a row: 8 pieces in some order
            uint4 w = col[i];
            // a half whose exponent is all ones carries into its top bit
            auto odd = [](uint32_t y) { return ((y & 0x7f807f80u) + 0x00800080u) & 0x80008000u; };
            if ((i >> 3) >= live) {
              col[i] = make_uint4(0, 0, 0, 0);
            } else if (odd(w.x) | odd(w.y) | odd(w.z) | odd(w.w)) {
              auto clean = [&](uint32_t y) {
                const uint32_t z = odd(y);
                return y & ~((z & 0x8000u ? 0xffffu : 0u) | (z & 0x80000000u ? 0xffff0000u : 0u));
              };
              col[i] = make_uint4(clean(w.x), clean(w.y), clean(w.z), clean(w.w));
              bad = true;
            }
          }
        }
        if (bad) atomicOr(&u->bad, 1 << (j - partial));
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // the products read what was written here
        mbar_arrive(bar_vok + 8 * stage);
      }
      pos0 += 2 * tiles;
      leave_unit(it);
    }
  } else {
    // ---- the plan: this block's unit, then those of blocks that have not started, which the CTA
    // takes over one after the other: no launch, allocation or empty pipeline between units, and
    // whichever CTA is free takes the next
    int64_t block = blockIdx.x;
    uint32_t asked = 0;   // blocks asked for
    auto done = [&](int it) {   // unit `it` has been left by all
      return static_cast<bool>(
          __all_sync(0xffffffffu, wait_or_abort(bar_slot + 8 * (it % kSlots), (it / kSlots) & 1, abort)));
    };
    for (int it = 0;; ++it) {
      // The next unit is looked for when the loads of the one before are at its last tile: two
      // or three tiles before its end, which is when it is needed.  (Taken as early as there was a
      // slot, a CTA held two units while others had none: the last of 16 packed prompts' CTAs
      // ended 49 us after the first.)
      if (it > 0 && !__all_sync(0xffffffffu, wait_or_abort(bar_want, (it - 1) & 1, abort))) break;
      if (it >= kSlots && !done(it - kSlots)) break;
      Unit& slot = units[it % kSlots];
      int from = -1;   // a finished unit's slot that has to be taken again
      if (it >= kSlots && slot.redo != 0) from = it % kSlots;
      int found = -1;
      int64_t rank = 0;
      // (a block past the last unit has none, but the one that the CTA is given in its place may)
      bool asking = true;
      while (from < 0 && block >= 0 && found < 0 && asking) {
        __syncwarp();
        if (lane == 0) {   // ask for the next while this one is looked up
          mbar_expect_tx(bar_next, 16);
          asm volatile(
              "fence.proxy.async.shared::cta;\n\t"
              "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                  next_block_at),
              "r"(bar_next)
              : "memory");
        }
        // the sequences' units are counted 32 at a time
        const int span = a.tokens * S::kTiles;
        int64_t before = 0;
        for (int b0 = 0; b0 < a.batch && found < 0; b0 += 32) {
          const int b = b0 + lane;
          const int64_t mine = b < a.batch ? units_of(a, b, span) : 0;
          int64_t upto = mine;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += y;
          }
          const int64_t r = block - before;
          const uint32_t hit = __ballot_sync(0xffffffffu, r >= upto - mine && r < upto);
          if (hit) {
            found = b0 + __ffs(hit) - 1;
            rank = __shfl_sync(0xffffffffu, r - (upto - mine), __ffs(hit) - 1);
          }
          before += __shfl_sync(0xffffffffu, upto, 31);
        }
        if (found >= 0 && lane == 0) {
          write_unit<HD>(a, found, rank, slot);
          mbar_arrive(bar_unit + 8 * (it % kSlots));
        }
        asking = __all_sync(0xffffffffu, wait_or_abort(bar_next, asked & 1, abort));
        if (!asking) {
          (void)wait_bounded(bar_next, asked & 1);
          break;
        }
        ++asked;
        uint32_t taken, x;
        asm volatile(
            "{\n\t.reg .b128 r;\n\t.reg .pred p;\n\t.reg .b32 y, z, w;\n\t"
            "ld.shared.b128 r, [%2];\n\t"
            "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
            "selp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
            "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, y, z, w}, r;\n\t}"
            : "=r"(taken), "=r"(x)
            : "r"(next_block_at)
            : "memory");
        block = next_block(taken != 0, static_cast<int64_t>(x), found >= 0, before);
      }
      if (!asking) break;
      if (found >= 0) continue;
      // No block left: the units under way may still have to be taken again.
      bool ok = true;
      for (int k = it - 1; from < 0 && ok && k >= 0 && k > it - kSlots; --k) {
        ok = done(k);
        if (ok && units[k % kSlots].redo != 0) from = k % kSlots;
      }
      if (!ok) break;
      __syncwarp();
      if (lane == 0) {
        if (from >= 0) {
          if (from != it % kSlots) slot = units[from];
          units[from].redo = 0;
          slot.checked = 1;
          slot.redo = slot.bad = 0;
        } else {
          slot.n = -1;
        }
        mbar_arrive(bar_unit + 8 * (it % kSlots));
      }
      __syncwarp();
      if (from < 0) break;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(*tmem_slot), "r"(512) : "memory");
  }
}

// bf16 [rows, heads, head_dim] in boxes of 64 elements x box_heads x box_rows, 128-byte swizzle; rows past
// the end read as zero.
cudaError_t head_map(CUtensorMap* map, const void* p, int64_t rows, int64_t heads, int64_t head_dim, int64_t ld,
                     uint32_t box_heads, uint32_t box_rows) {
  EncodeTiled enc = encode_tiled();
  if (enc == nullptr) return cudaErrorNotSupported;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(head_dim), static_cast<cuuint64_t>(heads),
                              static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(head_dim) * 2, static_cast<cuuint64_t>(ld) * 2};
  const cuuint32_t box[3] = {64, box_heads, box_rows};
  const cuuint32_t elem[3] = {1, 1, 1};
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p), dims, strides, box, elem,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int HD>
cudaError_t launch(const uint16_t* q, int64_t ld_q, const uint16_t* k, int64_t ld_k, Args a, cudaStream_t stream) {
  using S = Shape<HD>;
  static_assert(S::kSmem <= 227 * 1024, "shared memory");
  CUtensorMap map_q, map_k, map_v;
  cudaError_t err = head_map(&map_q, q, a.rows_q, a.heads, HD, ld_q, a.heads_per_tile, a.tokens);
  // a tensor of no keys has no map: any valid one, it is not read
  const bool keys = a.rows_k > 0;
  if (err == cudaSuccess)
    err = keys ? head_map(&map_k, k, a.rows_k, a.heads / a.group, HD, ld_k, 1, S::kKeys)
               : head_map(&map_k, q, a.rows_q, a.heads, HD, ld_q, 1, S::kKeys);
  if (err == cudaSuccess)
    err = keys ? head_map(&map_v, a.v, a.rows_k, a.heads / a.group, HD, a.ld_v, 1, S::kKeys)
               : head_map(&map_v, q, a.rows_q, a.heads, HD, ld_q, 1, S::kKeys);
  if (err != cudaSuccess) return err;
  int one = 0;
  err = persistent_blocks(reinterpret_cast<const void*>(&attention_kernel<HD>), kThreads, S::kSmem, 1, &one);
  if (err != cudaSuccess) return err;
  const int64_t span = static_cast<int64_t>(a.tokens) * S::kTiles;
  // at most this many pairs of row tiles, however the rows fall into sequences (each has a row)
  const int64_t most = (a.rows_q + a.batch * (span - 1)) / span;
  const int64_t pairs = most < a.rows_q ? most : a.rows_q;
  const int64_t blocks = pairs * a.tile_groups;
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  attention_kernel<HD><<<static_cast<unsigned>(blocks), kThreads, S::kSmem, stream>>>(map_q, map_k, map_v, a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attention(const uint16_t* q, int64_t ld_q, const uint16_t* k, int64_t ld_k, const uint16_t* v,
                             int64_t ld_v, const int32_t* cu_q, const int32_t* cu_k, int batch, int64_t rows_q,
                             int64_t rows_k, int heads, int kv_heads, int head_dim, int causal, float scale,
                             uint16_t* o, float* lse, cudaStream_t stream) {
  Args a{};
  a.cu_q = cu_q;
  a.cu_k = cu_k;
  a.batch = batch;
  a.rows_q = rows_q;
  a.rows_k = rows_k;
  a.heads = heads;
  a.group = heads / kv_heads;
  // heads of a row tile: the divisor of the group that fills the most of 128 rows, the
  // largest of those
  int best = 0;
  for (int d = 1; d <= a.group && d <= kTileRows; ++d)
    if (a.group % d == 0 && kTileRows / d * d >= best) {
      best = kTileRows / d * d;
      a.heads_per_tile = d;
    }
  a.tokens = kTileRows / a.heads_per_tile;
  a.tile_groups = heads / a.heads_per_tile;
  // heads whose keys and values are swept together: as many as stay in half of the L2
  const int64_t kv_bytes = rows_k * head_dim * 4;
  int64_t kv_chunk = kv_bytes > 0 ? (int64_t{64} << 20) / kv_bytes : kv_heads;
  kv_chunk = kv_chunk < 1 ? 1 : kv_chunk > kv_heads ? kv_heads : kv_chunk;
  a.head_chunk = static_cast<int>(kv_chunk * (a.group / a.heads_per_tile));
  a.causal = causal;
  a.scale = scale;
  a.v = v;
  a.ld_v = ld_v;
  a.o = o;
  a.lse = lse;
  switch (head_dim) {
    case 64: return launch<64>(q, ld_q, k, ld_k, a, stream);
    case 128: return launch<128>(q, ld_q, k, ld_k, a, stream);
    default: return launch<256>(q, ld_q, k, ld_k, a, stream);
  }
}

cudaError_t attention_error_flag(int* flag) {
  int zero = 0;
  cudaError_t err = cudaMemcpyFromSymbol(flag, g_attention_fault, sizeof(int));
  if (err == cudaSuccess) err = cudaMemcpyToSymbol(g_attention_fault, &zero, sizeof(int));
  return err;
}

}  // namespace h3q
