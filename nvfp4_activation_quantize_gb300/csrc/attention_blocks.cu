// attention_blocks.cu -- softmax attention over listed blocks of keys (video, prompts, single new
// tokens) on the fifth-generation tensor cores.
//
// Per row (a query token and one of its heads), over the keys of the blocks that the list of its
// query block and key head names, and that it sees: x_j = scale * q . k_j, o = sum_j e^(x_j - m) v_j /
// sum_j e^(x_j - m), in one pass with the running maximum and sum, as attention.cu does it.
//
// Bound: the tensor cores, 4 * head_dim operations per row and listed key.  A CTA takes two row tiles of up
// to 128 rows (tokens x heads of one group), so that one has its softmax while the other has the
// tensor cores.  A tile of 128 keys is two runs of 64, each anywhere in the sequence: a block of 64,
// or half of a larger one's part.
//   Where a query block fills both tiles (grouped heads, 256 tokens), they share every key tile.
//   Where it fills one (128 tokens of a head of its own), the tiles are neighbouring query blocks
//   with a list each, and every key tile is loaded for one row tile.  That is 64 KB from L2 for 1,024 clocks
//   of products, 64 bytes a clock of an SM, where copies of 32 KB alone get 80 (23 TB/s) and those in
//   runs of 64 keys 60.
// 32,640 tokens, 56 heads of 128, 32 blocks of 128 keys a list: 3.1 to 3.3 ms, 1.16 to 1.24 PFLOP/s, with a list for
// each 128 tokens (tensor cores busy 47% of the time).  Of the ring's five tiles two are held, whole, by the products
// under way, so about three are in flight, and the loads' latency is the bound: 11 TB/s.  2.5 to 2.65 ms, 1.45 to
// 1.51 PFLOP/s, with a list for 256 tokens (61%), near what the power limit allows.
//
//   warps 0..3, 4..7  softmax of tile 0, 1: a thread owns one row of S in TMEM, takes the weights against
//                     a reference that follows the row's maximum when that has grown by more than
//                     2^8, writes them as bf16 over S in two halves and sums them in fp32 unrounded.
//                     (A weight's rounding, at most 2^-8 of it, is the type of V that it is
//                     multiplied with; maxima, sums and outputs are fp32.)  At the end it scales its
//                     row of O and stores it.
//   warp 8            the lists, 32 entries at a time, and TMA: Q once, then K and V tiles
//   warp 9            the products: S = Q K^T (operands in shared memory), O += P V (P in TMEM)
//   warp 10           looks at the tiles of V that some row does not see whole: rows past the sequence's end
//                     become zero, and so do values that are no numbers (0 * NaN would reach rows that do
//                     not see them); the epilogue adds these back for the rows that do.  One to three tiles
//                     a unit, checked while the softmax of their S runs.
//   warp 11           the plan: which unit is next, how many key tiles its lists come to.  The CTA's own
//                     block first, then those of blocks that have not started, which it takes over
//
// Every wait is bounded: one that runs out sets a device flag and tells the other roles
// to stop; the CTA drains what it has in flight, frees its TMEM and returns.
#include <cmath>

#include "h3q_async.cuh"
#include "h3q_blocks.cuh"
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
constexpr int kKeys = 128;       // of a tile: two runs of 64
constexpr int kRun = 64;
constexpr int kTellRing = 16;    // key tiles whose first keys are told ahead (those in the ring, and two more unread)
constexpr int kMostPartial = 4;  // tiles that some row does not see whole: runs that begin among 64 + 255 keys
constexpr float kSlack = 8.0f;   // a row's reference moves when its maximum has passed it by 2^8,
constexpr float kJump = 16.0f;   // at once when a tile passes it by 2^16 (sums stay finite, see attention.cu)

__device__ int g_blocks_fault;

struct Args {
  const int32_t* cu_q;
  const int32_t* cu_k;
  int batch;
  int64_t rows_q, rows_k;
  int heads, group;          // query heads, and per key head
  int heads_per_tile, tokens, tile_groups;  // a row tile: tokens x heads_per_tile; tile_groups of heads
  int head_chunk;            // tile groups that are swept together (their keys and values stay in L2)
  int shift_q, shift_k;      // log2 of the blocks' sizes
  int split_sms;             // the last units are split where they leave half of so many CTAs idle; 0: never
  int block_pairs;           // pairs of row tiles of a query block; 0: a block is one tile, two blocks a pair
  const int32_t* lists;      // [kv_heads][list_rows][top]
  int64_t list_rows;
  int top;
  int causal;
  float scale;
  const uint16_t* v;         // for the values that are no numbers
  int64_t ld_v;
  uint16_t* o;
  float* lse;                // or nullptr
};

template <int HD>
struct Shape {
  static constexpr int kHalves = HD / 64;               // 64-element (128-byte) column blocks of a row
  static constexpr int kQBytes = kTileRows * HD * 2;
  static constexpr int kKvBytes = kKeys * HD * 2;
  static constexpr int kStages = 5 * 128 / HD;          // K and V tiles in the ring, in the order of their products
  static constexpr int kOffKv = 2 * kQBytes;
  static constexpr int kOffBar = kOffKv + kStages * kKvBytes;
  static constexpr int kBars = 4 * kStages + 12 + 2 * kSlots + 4;   // named in the kernel
  static constexpr int kOffMisc = kOffBar + 8 * kBars;    // TMEM address, abort; a taken block's id (16-byte aligned)
  static constexpr int kOffTell = kOffMisc + 32;          // [row tile][kTellRing] first keys of a tile's runs
  static constexpr int kOffSlots = kOffTell + 2 * kTellRing * 8;
  static constexpr int kSlotBytes = 192;
  static constexpr int kSmem = kOffSlots + kSlots * kSlotBytes + 1024;
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
  return h3q::wait_or_abort(bar, parity, abort, &g_blocks_fault);
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// A unit of work: a pair of row tiles of one sequence and group of heads, as the planning warp
// hands it to the others.
struct Unit {
  int64_t q0, k0;        // first packed rows of the sequence
  const int32_t* list[2];
  int n, len;            // its queries and keys; n < 0: no more units
  int head0;             // first head of the tile
  int shared;            // both tiles have list[0]
  int tok[2], toks[2];   // first token of each row tile, and how many
  int most[2];           // keys that some row of the tile (shared: of either) sees
  int least[2];          // keys that every row of it sees
  int tiles[2];          // key tiles that each reads
  int partial[2];        // first of them that some row does not see whole
  int bad[2];            // which of the partial V tiles held values that are no numbers (shared: [0]),
  int2 bad_at[2][kMostPartial];   // and their runs
};

__device__ __forceinline__ int clamp_keys(int64_t x, int len) {
  return x < 0 ? 0 : x > len ? len : static_cast<int>(x);
}

// Pairs of row tiles of a sequence of n queries.
__device__ __forceinline__ int64_t pairs_of(const Args& a, int64_t n) {
  const int64_t size = int64_t{1} << a.shift_q;
  if (a.block_pairs == 0) return ((n + size - 1) / size + 1) / 2;
  const int64_t rest = n & (size - 1);
  return (n >> a.shift_q) * a.block_pairs + ((rest + a.tokens - 1) / a.tokens + 1) / 2;
}

__device__ __forceinline__ int64_t units_of(const Args& a, int b) {
  return pairs_of(a, rows_of(a.cu_q, b, a.rows_q)) * a.tile_groups;
}

// Which of 32 entries of a list count (an entry for each lane; -1 past its end): the numbers of blocks, above
// all before them that count.  `above`: the last that did, before and after.  Whole warp.
__device__ __forceinline__ bool entry_counts(int v, int blocks, int& above) {
  const int lane = threadIdx.x & 31;
  const int w = v >= 0 && v < blocks ? v : -1;
  int upto = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto = max(upto, y);
  }
  int before = __shfl_up_sync(0xffffffffu, upto, 1);
  before = lane == 0 ? above : max(before, above);
  above = max(above, __shfl_sync(0xffffffffu, upto, 31));
  return w > before;
}

// Fills in unit number `rank` of sequence b, or its row tile number `half` alone: every lane the same.  Whole warp.
template <int HD>
__device__ __forceinline__ void write_unit(const Args& a, int b, int64_t rank, int half, Unit& u) {
  const int lane = threadIdx.x & 31;
  const int64_t q0 = a.cu_q[b];
  const int64_t n = rows_of(a.cu_q, b, a.rows_q);
  const int len = static_cast<int>(rows_of(a.cu_k, b, a.rows_k));
  const int64_t pairs = pairs_of(a, n);
  const int64_t chunk = rank / (a.head_chunk * pairs);
  const int64_t rest = rank - chunk * a.head_chunk * pairs;
  const int h0 = static_cast<int>(chunk) * a.head_chunk;
  const int here = a.tile_groups - h0 < a.head_chunk ? a.tile_groups - h0 : a.head_chunk;
  const int64_t pair = pairs - 1 - rest / here;   // the longest rows first
  const int head0 = (h0 + static_cast<int>(rest % here)) * a.heads_per_tile;
  const int64_t shift = static_cast<int64_t>(len) - n + 1;  // token t sees keys below t + shift
  const bool shared = a.block_pairs > 0;
  const int64_t first_list = (a.cu_q[b] >> a.shift_q) + static_cast<int64_t>(b);
  int tok[2], toks[2], most[2], least[2], tiles[2] = {0, 0}, partial[2] = {0, 0};
  const int32_t* list[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int tile = half < 0 ? x : half;
    const int64_t block = shared ? pair / a.block_pairs : 2 * pair + tile;
    const int64_t from = (block << a.shift_q) + (shared ? (2 * (pair % a.block_pairs) + tile) * a.tokens : 0);
    int64_t end = (block + 1) << a.shift_q;   // of the block's tokens
    if (end > n) end = n;
    const int64_t count = end - from < a.tokens ? end - from : a.tokens;
    toks[x] = count < 0 || (half >= 0 && x == 1) ? 0 : static_cast<int>(count);
    tok[x] = toks[x] > 0 ? static_cast<int>(from) : 0;
    least[x] = a.causal ? clamp_keys(tok[x] + shift, len) : len;
    most[x] = toks[x] == 0 ? 0 : a.causal ? clamp_keys(tok[x] + toks[x] - 1 + shift, len) : len;
    list[x] = a.lists + (static_cast<int64_t>(head0 / a.group) * a.list_rows + first_list + (toks[x] > 0 ? block : 0)) * a.top;
  }
  if (shared) {   // one plan for both (the first has rows, or neither)
    most[0] = most[1] = max(most[0], most[1]);
    least[1] = least[0];
  }
  const int blocks = (len + (1 << a.shift_k) - 1) >> a.shift_k;
  const int runs_each = 1 << (a.shift_k - 6);
#pragma unroll 1
  for (int x = 0; x < (shared ? 1 : 2); ++x) {
    int above = -1, runs = 0, whole = 0;
    for (int i0 = 0; i0 < a.top && (static_cast<int64_t>(above + 1) << a.shift_k) < most[x]; i0 += 32) {
      const int v = i0 + lane < a.top ? list[x][i0 + lane] : -1;
      if (entry_counts(v, blocks, above)) {
        const int from = v << a.shift_k;
        runs += min(max((most[x] - from + kRun - 1) >> 6, 0), runs_each);
        whole += min(max((least[x] - from) >> 6, 0), runs_each);
      }
    }
    runs = __reduce_add_sync(0xffffffffu, runs);
    whole = __reduce_add_sync(0xffffffffu, whole);
    tiles[x] = (runs + 1) / 2;
    partial[x] = whole / 2;
  }
  if (shared) {
    tiles[1] = toks[1] > 0 ? tiles[0] : 0;
    partial[1] = partial[0];
  }
  if (lane == 0) {
    u.q0 = q0;
    u.k0 = len > 0 ? a.cu_k[b] : 0;
    u.n = static_cast<int>(n);
    u.len = len;
    u.head0 = head0;
    u.shared = shared;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      u.list[x] = list[x];
      u.tok[x] = tok[x];
      u.toks[x] = toks[x];
      u.most[x] = most[x];
      u.least[x] = least[x];
      u.tiles[x] = tiles[x];
      u.partial[x] = partial[x];
      u.bad[x] = 0;
    }
  }
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
attention_blocks_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                        const __grid_constant__ CUtensorMap map_v, const Args a) {
  using S = Shape<HD>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t{1023});
  const uint32_t base = smem_u32(smem);
  const uint32_t bar_full = base + S::kOffBar;             // + 8 * stage
  const uint32_t bar_empty = bar_full + 8 * S::kStages;
  const uint32_t bar_vraw = bar_empty + 8 * S::kStages;       // a V tile that the check warp looks at first ...
  const uint32_t bar_vok = bar_vraw + 8 * S::kStages;         // ... and has passed on
  const uint32_t bar_q = bar_vok + 8 * S::kStages;            // + 8 * row tile: Q has landed,
  const uint32_t bar_qfree = bar_q + 16;                   // is no longer read
  const uint32_t bar_s = bar_qfree + 16;                   // + 8 * row tile
  const uint32_t bar_p = bar_s + 16;
  const uint32_t bar_p2 = bar_p + 16;                      // the weights of the second half of a tile's keys
  const uint32_t bar_o = bar_p2 + 16;
  const uint32_t bar_unit = bar_o + 16;                    // + 8 * slot: a unit is there,
  const uint32_t bar_slot = bar_unit + 8 * kSlots;         // all have read it
  const uint32_t bar_next = bar_slot + 8 * kSlots;         // a waiting block was taken over, or none was left
  const uint32_t bar_want = bar_next + 8;                  // the loads of a unit are about to end
  const uint32_t bar_drain = bar_want + 8;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::kOffMisc);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + S::kOffMisc + 4);
  const uint32_t next_block_at = base + S::kOffMisc + 16;
  volatile int2* tell = reinterpret_cast<volatile int2*>(smem + S::kOffTell);   // [row tile * kTellRing + count % kTellRing]
  static_assert(sizeof(Unit) <= S::kSlotBytes, "slots");
  auto unit_slot = [&](int it) { return reinterpret_cast<Unit*>(smem + S::kOffSlots + it % kSlots * S::kSlotBytes); };
  constexpr int kReaders = 8 + 3;   // warps that read a slot: softmax, TMA, products, check
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
    if (!__all_sync(0xffffffffu, wait_or_abort(bar_unit + 8 * (it % kSlots), (it / kSlots) & 1, abort))) return nullptr;
    Unit* u = unit_slot(it);
    return u->n < 0 ? nullptr : u;
  };
  auto leave_unit = [&](int it) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar_slot + 8 * (it % kSlots));
  };

  if (warp < kTmaWarp) {
    // ---- softmax and epilogue of one row tile
    const int x = warp >> 2;
    const int row = (warp & 3) * 32 + lane;
    const int row_tok = row / a.heads_per_tile, row_head = row % a.heads_per_tile;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;   // the TMEM of all 512 columns begins at 0
    const uint32_t taddr_o = lane_base + S::kO + x * HD;
    const uint32_t taddr = lane_base + x * S::kS;
    const float c = fmaxf(__fmul_rn(a.scale, kLog2e), 0x1p-126f);   // never 0: a hidden key's -inf stays one
    uint32_t s_count = 0, o_count = 0;   // S tiles and outputs waited for
    bool ok = true;
    Unit* u;
    for (int it = 0; ok && (u = unit_at(it)) != nullptr; ++it) {
      const int tok = u->tok[x] + row_tok;
      const bool valid = row < a.tokens * a.heads_per_tile && row_tok < u->toks[x];
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
        if (!(ok = __all_sync(0xffffffffu, wait_or_abort(bar_s + 8 * x, s_count & 1, abort)))) break;
        // (O is at rest: S[j] was issued after P[j-1] V[j-1])
        const int told = x * kTellRing + s_count % kTellRing;
        const int run0 = tell[told].x, run1 = tell[told].y;   // first keys of the two runs (the second: or past all keys)
        ++s_count;
        tc_fence_after();
        if (j > 0 && __any_sync(0xffffffffu, __fmul_rn(__fadd_rn(m_seen, -m_ref), c) > kSlack)) rescale(true);
        const int seen0 = sees - run0, seen1 = sees - run1;
        const bool masked = j >= partial;
        const float2 c2 = make_float2(c, c);
        uint32_t s[kKeys / 32][32];
        uint32_t w[kRun / 2];
        float2 sum;
        // The weights of this tile are taken against the reference as it is, while the tile's
        // maximum is still being formed; only where a row passes it by 2^kJump is the reference
        // moved at once and the tile read again.
        bool fresh = j == 0;   // no reference yet: only the maximum is formed
        for (;;) {
#pragma unroll
          for (int i = 0; i < kKeys / 32; ++i) tc_load32(taddr + 32 * i, s[i]);
          tc_wait_load(s[0]);
#pragma unroll
          for (int i = 1; i < kKeys / 32; ++i) tc_loaded(s[i]);
          if (masked) {
#pragma unroll
            for (int i = 0; i < kKeys; ++i)
              if (i % kRun >= (i < kRun ? seen0 : seen1)) s[i / 32][i % 32] = 0xff800000u;
          }
          float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int i = 0; i < kKeys; i += 8)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              m[k] = max3(m[k], __uint_as_float(s[i / 32][i % 32 + 2 * k]), __uint_as_float(s[i / 32][i % 32 + 2 * k + 1]));
          if (fresh) {
            fresh = false;
            m_seen = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
            rescale(false);
            continue;
          }
          const float start = m_ref == -INFINITY ? 0.0f : -__fmul_rn(m_ref, c);
          const float2 b2 = make_float2(start, start);
          sum = make_float2(0.0f, 0.0f);
#pragma unroll
          for (int i = 0; i < kRun; i += 16) weights16(s[i / 32] + i % 32, c2, b2, sum, w + i / 2);
          m_seen = fmaxf(max3(m_seen, m[0], m[1]), fmaxf(m[2], m[3]));
          // (a difference of two -inf is no number, and not above)
          if (!__any_sync(0xffffffffu, __fmul_rn(__fadd_rn(m_seen, -m_ref), c) > kJump)) break;
          rescale(j > 0);
        }
        const float start = m_ref == -INFINITY ? 0.0f : -__fmul_rn(m_ref, c);
        const float2 b2 = make_float2(start, start);
        store_weights<kRun / 2>(taddr, w);
        tc_wait_store();
        tc_fence_before();
        mbar_arrive(bar_p + 8 * x);              // the products of the first half of the keys may start
#pragma unroll
        for (int i = 0; i < kRun; i += 16) weights16(s[(kRun + i) / 32] + i % 32, c2, b2, sum, w + i / 2);
        store_weights<kRun / 2>(taddr + kRun / 2, w);
        l = __fadd_rn(l, __fadd_rn(sum.x, sum.y));
        tc_wait_store();
        tc_fence_before();
        mbar_arrive(bar_p2 + 8 * x);
      }
      if (n > 0 && ok) {
        ok = __all_sync(0xffffffffu, wait_or_abort(bar_o + 8 * x, o_count & 1, abort));
        ++o_count;
        tc_fence_after();
      }
      if (ok) {
        // The row of O, scaled, 128 bytes at a time.  Eight lanes hold eight rows of eight 16-byte pieces: they
        // exchange them (three steps of a transposition), so that a store writes whole rows of 128 bytes, eight
        // lanes each.  (No shared memory: a stage of the ring more is worth more there.)
        const float inv = l == 0.0f ? 0.0f : __fdiv_rn(1.0f, l);
        const int64_t out_row = u->q0 + tok;
        const int head = u->head0 + row_head;
        const int own = u->shared ? 0 : x;
        const int bad = *static_cast<volatile int*>(&u->bad[own]);
        const unsigned long long dst =
            valid ? reinterpret_cast<unsigned long long>(a.o + (out_row * a.heads + head) * HD) : 0ull;
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
            const int kv_head = u->head0 / a.group;
            for (int part = 0; part < 2 * kMostPartial; ++part) {
              if (!(bad >> (part / 2) & 1)) continue;
              const int from = part & 1 ? u->bad_at[own][part / 2].y : u->bad_at[own][part / 2].x;
              const int end = sees < from + kRun ? sees : from + kRun;
              for (int key = from > u->least[own] ? from : u->least[own]; key < end; ++key) {
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
          uint32_t w[8][4];
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            const float2 y = make_float2(__uint_as_float(o[k / 16][k % 16 * 2]), __uint_as_float(o[k / 16][k % 16 * 2 + 1]));
            w[k / 4][k % 4] = l == 0.0f ? 0u : float2_to_bf16x2(mul2(y, make_float2(inv, inv)));
          }
#pragma unroll
          for (int step = 1; step < 8; step <<= 1) {
            const bool upper = lane & step;
#pragma unroll
            for (int piece = 0; piece < 8; ++piece) {
              if (piece & step) continue;
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint32_t got = __shfl_xor_sync(0xffffffffu, upper ? w[piece][k] : w[piece | step][k], step);
                if (upper) {
                  w[piece][k] = got;
                } else {
                  w[piece | step][k] = got;
                }
              }
            }
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) {   // row k of the eight lanes' rows, piece lane % 8
            const unsigned long long to = __shfl_sync(0xffffffffu, dst, (lane & 24) + k);
            if (to != 0)
              store16(reinterpret_cast<uint16_t*>(to) + i + 8 * (lane & 7), make_uint4(w[k][0], w[k][1], w[k][2], w[k][3]));
          }
        }
        if (valid && a.lse != nullptr)
          a.lse[head * a.rows_q + out_row] =
              l == 0.0f ? -INFINITY : __fmul_rn(__fadd_rn(__fmul_rn(m_ref, c), log2f(l)), kLn2);
        tc_fence_before();   // O has been read before the next unit's first weights are announced
      }
      leave_unit(it);
    }
  } else if (warp == kTmaWarp) {
    // ---- the lists and the loads: the whole warp in step, one lane issues
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_q)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_k)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_v)) : "memory");
    const int q_rows = a.tokens * a.heads_per_tile;
    const int runs_each = 1 << (a.shift_k - 6);
    bool ok = true;
    uint32_t q_count[2] = {0, 0}, told[2] = {0, 0};   // Q tiles issued, K tiles told
    uint32_t stage = 0;                               // the next one
    uint32_t used = 0, use_phase = 0;                 // per stage: whether it has been filled, how often (its last bit)
    uint32_t full_phase = 0, raw_phase = 0;           // per stage: the phases of its full and v_raw barriers
    uint32_t last_raw = 0;                            // per stage: its last tile went to the check warp
    auto wait = [&](uint32_t bar, uint32_t parity) {
      return static_cast<bool>(__all_sync(0xffffffffu, wait_or_abort(bar, parity, abort)));
    };
    Unit* u;
    for (int it = 0; ok && (u = unit_at(it)) != nullptr; ++it) {
      const int kv_head = u->head0 / a.group, head0 = u->head0, len = u->len;
      const int row_q0 = static_cast<int>(u->q0), row_k0 = static_cast<int>(u->k0);
      const bool shared = u->shared != 0;
      const int tok[2] = {u->tok[0], u->tok[1]}, tiles[2] = {u->tiles[0], u->tiles[1]};
      const int partial[2] = {u->partial[0], u->partial[1]}, most[2] = {u->most[0], u->most[1]};
      const int32_t* const list[2] = {u->list[0], u->list[1]};
      leave_unit(it);
      const int blocks = (len + (1 << a.shift_k) - 1) >> a.shift_k;
      // Where each list is: its next entries, which of them count, and the run in the block that is next.
      int at[2] = {0, 0}, entry[2] = {0, 0}, above[2] = {-1, -1}, run_of[2] = {0, 0}, block[2] = {0, 0};
      uint32_t left[2] = {0, 0};
      int2 runs[2];   // of the last K tile
      // First key of the list's next run, or past all keys.
      auto next_run = [&](int x) {
        if (run_of[x] == 0) {
          while (left[x] == 0) {
            if (at[x] >= a.top) return 0x40000000;
            entry[x] = at[x] + lane < a.top ? list[x][at[x] + lane] : -1;
            at[x] += 32;
            left[x] = __ballot_sync(0xffffffffu, entry_counts(entry[x], blocks, above[x]));
          }
          block[x] = __shfl_sync(0xffffffffu, entry[x], __ffs(left[x]) - 1);
          left[x] &= left[x] - 1;
        }
        const int first = (block[x] << a.shift_k) + run_of[x] * kRun;
        run_of[x] = (run_of[x] + 1) & (runs_each - 1);
        return first < most[x] ? first : 0x40000000;
      };
      auto load_q = [&](int x) {
        if (tiles[x] == 0) return true;
        if (!wait(bar_qfree + 8 * x, (q_count[x] & 1) ^ 1u)) return false;
        ++q_count[x];
        if (lane == 0) {
          mbar_expect_tx(bar_q + 8 * x, q_rows * HD * 2);
          for (int h = 0; h < S::kHalves; ++h)
            tma_load_3d(base + x * S::kQBytes + h * (kTileRows * 128), &map_q, 64 * h, head0, row_q0 + tok[x],
                        bar_q + 8 * x);
        }
        return true;
      };
      auto free_stage = [&]() { return wait(bar_empty + 8 * stage, (use_phase >> stage & 1) ^ 1u); };
      // (blocks of 64 come in boxes of 64 keys; larger ones in boxes of a tile, whose runs follow each other)
      auto load_tile = [&](const CUtensorMap* map, const int2& r, bool raw) {
        const uint32_t bar = (raw ? bar_vraw : bar_full) + 8 * stage, bit = 1u << stage;
        used |= bit;
        use_phase ^= bit;
        last_raw = (last_raw & ~bit) | static_cast<uint32_t>(raw) << stage;
        (raw ? raw_phase : full_phase) ^= bit;
        if (lane == 0) {
          mbar_expect_tx(bar, S::kKvBytes);
          const int second = r.y < len ? r.y : r.x;   // (none: any keys, which are hidden, and cleaned from V)
          for (int h = 0; h < S::kHalves; ++h) {
            const uint32_t to = base + S::kOffKv + stage * S::kKvBytes + h * (kKeys * 128);
            tma_load_3d(to, map, 64 * h, kv_head, row_k0 + r.x, bar);
            if (a.shift_k == 6) tma_load_3d(to + kRun * 128, map, 64 * h, kv_head, row_k0 + second, bar);
          }
        }
        stage = stage + 1 == S::kStages ? 0 : stage + 1;
      };
      auto load_k = [&](int x) {
        runs[x].x = next_run(x);
        runs[x].y = next_run(x);
        if (!free_stage()) return false;
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          if (tiles[y] == 0 || (!shared && y != x)) continue;
          const int place = y * kTellRing + told[y]++ % kTellRing;
          if (lane == 0) {
            tell[place].x = runs[x].x;
            tell[place].y = runs[x].y;
          }
        }
        load_tile(&map_k, runs[x], false);
        return true;
      };
      auto load_v = [&](int x, int j) {
        if (!free_stage()) return false;
        load_tile(&map_v, runs[x], j >= partial[x]);
        return true;
      };
      auto want = [&]() {
        if (lane == 0) mbar_arrive(bar_want);
      };
      const int n = max(tiles[0], tiles[1]);
      if (n == 0) want();
      ok = load_q(0);
      if (shared) {
        for (int j = 0; j < n && ok; ++j) {
          if (j == n - 1) want();
          ok = load_k(0);
          if (ok && j == 0) ok = load_q(1);
          if (ok) ok = load_v(0, j);
        }
      } else {
        if (ok && tiles[0] > 0) ok = load_k(0);
        if (ok) ok = load_q(1);
        if (ok && tiles[1] > 0) ok = load_k(1);
        for (int j = 0; j < n && ok; ++j) {
          if (j == n - 1) want();
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (!ok || j >= tiles[x]) continue;
            ok = load_v(x, j);
            if (ok && j + 1 < tiles[x]) ok = load_k(x);
          }
        }
      }
    }
    // Before the CTA goes: every stage's last tile is released (the products' commits arrive
    // here); after an abort, every copy issued has landed.
    if (lane == 0) {
      for (uint32_t i = 0; i < S::kStages && !raised_here(abort); ++i)
        if (used >> i & 1) (void)wait_or_abort(bar_empty + 8 * i, (use_phase >> i & 1) ^ 1u, abort);
      if (raised_here(abort)) {
        for (uint32_t i = 0; i < S::kStages; ++i)
          if (used >> i & 1) {
            const bool raw = last_raw >> i & 1;
            (void)wait_bounded((raw ? bar_vraw : bar_full) + 8 * i, ((raw ? raw_phase : full_phase) >> i & 1) ^ 1u);
          }
        for (int x = 0; x < 2; ++x)
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
    // tensor cores.
    const uint32_t q_low = desc_low(base, 16);
    const uint32_t k_low = desc_low(base + S::kOffKv, 16);
    const uint32_t v_low = desc_low(base + S::kOffKv, kKeys * 128);   // 64 columns of V, then the next 64
    uint32_t next_stage = 0;                // of the ring, as the tiles come
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
            atomicExch(&g_blocks_fault, 1);
          }
          if (__any_sync(0xffffffffu, late || raised_here(abort))) return false;
        }
      }
    };
    auto wait = [&](uint32_t bar, uint32_t parity) { return wait_lanes(lane == 0 ? bar : 0u, parity); };
    // The next tile's stage, its barrier and parity.
    auto next_tile = [&](bool checked, uint32_t& stage, uint32_t& parity) {
      stage = next_stage;
      next_stage = next_stage + 1 == S::kStages ? 0 : next_stage + 1;
      parity = (checked ? ok_phase : full_phase) >> stage & 1;
      (checked ? ok_phase : full_phase) ^= 1u << stage;
      return (checked ? bar_vok : bar_full) + 8 * stage;
    };
    auto s_product = [&](int x, uint32_t stage) {   // S[x] = Q[x] K^T
      const uint32_t q = q_low + x * (S::kQBytes >> 4), k = k_low + stage * (S::kKvBytes >> 4);
#pragma unroll
      for (int i = 0; i < HD / 16; ++i)
        mma_ss(x * S::kS, q + (((i / 4) * (kTileRows * 128) + (i % 4) * 32) >> 4),
               k + (((i / 4) * (kKeys * 128) + (i % 4) * 32) >> 4), S::kIdescS, i > 0);
      commit_elected(bar_s + 8 * x);
    };
    // half of O[x] += P[x] V
    auto o_half = [&](int x, uint32_t stage, int j, int half) {
      const uint32_t v = v_low + stage * (S::kKvBytes >> 4);
      tc_fence_after();
#pragma unroll
      for (int i = half * kKeys / 32; i < (half + 1) * kKeys / 32; ++i)
        // rows of V 16 i ..: two 8-row groups of 1,024 bytes
        mma_ts(S::kO + x * HD, x * S::kS + 8 * i, v + (i * 2048 >> 4), S::kIdescO, j > 0 || i > 0);
    };
    auto release = [&](uint32_t stage) { commit_elected(bar_empty + 8 * stage); };
    Unit* u;
    for (int it = 0; ok && (u = unit_at(it)) != nullptr; ++it) {
      const bool shared = uniform(u->shared) != 0;
      const int n0 = uniform(u->tiles[0]), n1 = uniform(u->tiles[1]);
      const int partial0 = uniform(u->partial[0]), partial1 = uniform(u->partial[1]);
      leave_unit(it);
      const int tiles = n0 > n1 ? n0 : n1;
      if (tiles == 0) continue;
      uint32_t k_stage = 0, v_stage = 0;
      // the first S of each
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int n = x == 0 ? n0 : n1;
        if (!ok || n == 0) continue;
        uint32_t parity = 0;
        const uint32_t k_bar = !shared || x == 0 ? next_tile(false, k_stage, parity) : 0u;
        const uint32_t bar = lane == 0 ? bar_q + 8 * x : lane == 1 ? k_bar : 0u;
        const uint32_t q_parity = q_count[x]++ & 1;
        if (!(ok = wait_lanes(bar, lane == 0 ? q_parity : parity))) continue;
        tc_fence_after();
        s_product(x, k_stage);
        if (n == 1) commit_elected(bar_qfree + 8 * x);
        if (!shared || x == 1 || n1 == 0) release(k_stage);
      }
      // Commits go in where the queue of products is short (behind a full one they would keep the
      // warp until it has run), so a turn leaves its stages to the next.  With a list for each tile
      // the loads are the slower part and get their stages back at once (32,640 tokens of 56 heads over
      // 32 of 255 blocks 3.04 ms, against 3.22).
      int held_v = -1, held_k = -1;
      auto release_held = [&]() {
        if (held_v >= 0) release(held_v);
        if (held_k >= 0) release(held_k);
        held_v = held_k = -1;
      };
      for (int j = 0; j < tiles && ok; ++j) {
        uint32_t v_parity = 0, k_parity = 0, v_bar = 0, k_bar = 0;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int n = x == 0 ? n0 : n1;
          if (!ok || j >= n) continue;
          const bool first = !shared || x == 0, last = !shared || x == 1 || n1 == 0;
          if (first) {
            v_bar = next_tile(j >= (x == 0 ? partial0 : partial1), v_stage, v_parity);
            k_bar = j + 1 < n ? next_tile(false, k_stage, k_parity) : 0u;
          }
          // V[j], K[j + 1] and the first half of the weights, all at once
          const uint32_t parity = p_count[x]++ & 1;
          const uint32_t bar = lane == 0 ? bar_p + 8 * x : lane == 1 ? v_bar : lane == 2 ? k_bar : 0u;
          if (!(ok = wait_lanes(bar, lane == 0 ? parity : lane == 1 ? v_parity : k_parity))) continue;
          release_held();
          o_half(x, v_stage, j, 0);
          if (!(ok = wait(bar_p2 + 8 * x, parity))) continue;
          o_half(x, v_stage, j, 1);
          if (j + 1 < n) {
            s_product(x, k_stage);
            if (j + 2 == n) commit_elected(bar_qfree + 8 * x);
          } else {
            commit_elected(bar_o + 8 * x);
          }
          if (last) {
            held_v = v_stage;
            held_k = j + 1 < n ? static_cast<int>(k_stage) : -1;
            if (!shared) release_held();
          }
        }
      }
      if (ok) release_held();
    }
    // what is issued finishes before the TMEM is freed, whoever gave up and when
    commit_elected(bar_drain);
    (void)wait_bounded(bar_drain, 0);
    __syncwarp();
  } else if (warp == kCheckWarp) {
    uint32_t raw_phase = 0, count[2] = {0, 0};   // count: K tiles told of before this unit
    uint32_t base_stage = 0;                     // of the unit's first tile
    bool ok = true;
    Unit* u;
    for (int it = 0; ok && (u = unit_at(it)) != nullptr; ++it) {
      const bool shared = u->shared != 0;
      const int tiles[2] = {u->tiles[0], u->tiles[1]}, len = u->len;
      const int from_j = min(tiles[0] > 0 ? u->partial[0] : tiles[1], tiles[1] > 0 ? u->partial[1] : tiles[0]);
      for (int j = from_j; j < max(tiles[0], tiles[1]) && ok; ++j) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (!ok || j >= tiles[x] || j < u->partial[x] || (shared && x == 1)) continue;
          // tiles before this one: K V K V ..., or K0 K1, then V0 K0 V1 K1 a turn as far as each goes
          const int n0 = tiles[0], n1 = tiles[1], t0 = max(n0 - 1, 0), t1 = max(n1 - 1, 0);
          const int ahead = shared ? 2 * j + 1
                                   : (n0 > 0) + (n1 > 0) + min(j, n0) + min(j, t0) + min(j, n1) + min(j, t1) +
                                         (x == 1 ? (j < n0) + (j < t0) : 0);
          const uint32_t stage = (base_stage + ahead) % S::kStages;
          if (!(ok = __all_sync(0xffffffffu, wait_or_abort(bar_vraw + 8 * stage, raw_phase >> stage & 1, abort)))) continue;
          raw_phase ^= 1u << stage;
          const int told = x * kTellRing + (count[x] + j) % kTellRing;
          const int run0 = tell[told].x, run1 = tell[told].y;
          const int least = a.causal ? u->least[x] : len;   // only rows that some row of the unit does not see matter
          uint8_t* v = smem + S::kOffKv + stage * S::kKvBytes;
          bool bad = false;
#pragma unroll 1
          for (int h = 0; h < S::kHalves; ++h) {
            uint4* col = reinterpret_cast<uint4*>(v + h * (kKeys * 128));
#pragma unroll 4
            for (int i = lane; i < kKeys * 8; i += 32) {   // 128 bytes of a row: 8 pieces in some order
              const int r = i >> 3, key = r < kRun ? run0 + r : run1 + (r - kRun);
              if (key < least) continue;
              uint4 w = col[i];
              // a half whose exponent is all ones carries into its top bit
              auto odd = [](uint32_t y) { return ((y & 0x7f807f80u) + 0x00800080u) & 0x80008000u; };
              if (key >= len) {
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
          if (__any_sync(0xffffffffu, bad) && lane == 0) {
            u->bad_at[x][j - u->partial[x]] = make_int2(run0, run1);
            u->bad[x] |= 1 << (j - u->partial[x]);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // the products read what was written here
          mbar_arrive(bar_vok + 8 * stage);
        }
      }
      count[0] += tiles[0];
      count[1] += tiles[1];
      base_stage = (base_stage + 2 * (shared ? tiles[0] : tiles[0] + tiles[1])) % S::kStages;
      leave_unit(it);
    }
  } else {
    // ---- the plan: this block's unit, then those of blocks that have not started, which the CTA
    // takes over one after the other: no launch, allocation or empty pipeline between units, and
    // whichever CTA is free takes the next
    int64_t block = blockIdx.x;
    uint32_t asked = 0;   // blocks asked for
    for (int it = 0;; ++it) {
      // The next unit is looked for when the loads of the one before are at its last tile (a unit taken
      // earlier would wait here while another CTA has none).
      if (it > 0 && !__all_sync(0xffffffffu, wait_or_abort(bar_want, (it - 1) & 1, abort))) break;
      if (it >= kSlots &&   // its slot has been left by all
          !__all_sync(0xffffffffu, wait_or_abort(bar_slot + 8 * (it % kSlots), (it / kSlots - 1) & 1, abort)))
        break;
      Unit& slot = *unit_slot(it);
      int found = -1;
      int64_t rank = 0;
      int half = -1;
      // (a block past the last unit has none, but the one that the CTA is given in its place may)
      bool asking = true;
      while (block >= 0 && found < 0 && asking) {
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
        // the sequences' units are counted 32 at a time (units are split only where there are no more sequences)
        int64_t before = 0;
        for (int b0 = 0; b0 < a.batch && found < 0; b0 += 32) {
          const int b = b0 + lane;
          const int64_t mine = b < a.batch ? units_of(a, b) : 0;
          int64_t upto = mine;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += y;
          }
          int64_t unit = block, launched = __shfl_sync(0xffffffffu, upto, 31);
          if (a.split_sms > 0) {
            const UnitPart part = part_of(block, launched, a.split_sms);
            unit = part.unit;
            half = part.half;
            launched = part.blocks;
          }
          const int64_t r = unit - before;
          const uint32_t hit = __ballot_sync(0xffffffffu, r >= upto - mine && r < upto);
          if (hit) {
            found = b0 + __ffs(hit) - 1;
            rank = __shfl_sync(0xffffffffu, r - (upto - mine), __ffs(hit) - 1);
          }
          before += launched;
        }
        if (found >= 0) {
          write_unit<HD>(a, found, rank, half, slot);
          if (lane == 0) mbar_arrive(bar_unit + 8 * (it % kSlots));
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
      if (lane == 0) {   // no block left
        slot.n = -1;
        mbar_arrive(bar_unit + 8 * (it % kSlots));
      }
      __syncwarp();
      break;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(*tmem_slot), "r"(512) : "memory");
  }
}

// How the rows of a call are cut into tiles.
Args tiles_of(const BlockShape& b) {
  Args a{};
  a.cu_q = b.cu_q;
  a.cu_k = b.cu_k;
  a.batch = b.batch;
  a.rows_q = b.rows_q;
  a.rows_k = b.rows_k;
  a.heads = b.heads;
  a.group = b.heads / b.kv_heads;
  // heads of a row tile: the divisor of the group that fills the most of 128 rows, the
  // largest of those
  int best = 0;
  for (int d = 1; d <= a.group && d <= kTileRows; ++d)
    if (a.group % d == 0 && kTileRows / d * d >= best) {
      best = kTileRows / d * d;
      a.heads_per_tile = d;
    }
  a.tokens = kTileRows / a.heads_per_tile;
  if (a.tokens > b.block_q) a.tokens = b.block_q;
  a.tile_groups = b.heads / a.heads_per_tile;
  const int block_tiles = (b.block_q + a.tokens - 1) / a.tokens;
  a.block_pairs = block_tiles == 1 ? 0 : (block_tiles + 1) / 2;
  // heads whose keys and values are swept together: as many as stay in half of the L2
  const int64_t kv_bytes = b.rows_k * b.head_dim * 4;
  int64_t kv_chunk = kv_bytes > 0 ? (int64_t{64} << 20) / kv_bytes : b.kv_heads;
  kv_chunk = kv_chunk < 1 ? 1 : kv_chunk > b.kv_heads ? b.kv_heads : kv_chunk;
  a.head_chunk = static_cast<int>(kv_chunk * (a.group / a.heads_per_tile));
  a.shift_q = log2_of(b.block_q);
  a.shift_k = log2_of(b.block_k);
  a.list_rows = b.rows_q / b.block_q + b.batch;
  return a;
}

// At most this many pairs of row tiles, however the rows fall into sequences (each has a row).
int64_t most_pairs(const Args& a) {
  const int64_t most = a.block_pairs > 0 ? a.list_rows * a.block_pairs : (a.list_rows + a.batch + 1) / 2;
  return most < a.rows_q ? most : a.rows_q;
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
cudaError_t launch(const BlockShape& b, const uint16_t* q, int64_t ld_q, const uint16_t* k, int64_t ld_k, Args a,
                   cudaStream_t stream) {
  using S = Shape<HD>;
  static_assert(S::kSmem <= 227 * 1024, "shared memory");
  CUtensorMap map_q, map_k, map_v;
  const uint32_t box = b.block_k == kRun ? kRun : kKeys;
  cudaError_t err = head_map(&map_q, q, a.rows_q, a.heads, HD, ld_q, a.heads_per_tile, a.tokens);
  // a tensor of no keys has no map: any valid one, it is not read
  const bool keys = a.rows_k > 0;
  if (err == cudaSuccess)
    err = keys ? head_map(&map_k, k, a.rows_k, b.kv_heads, HD, ld_k, 1, box)
               : head_map(&map_k, q, a.rows_q, a.heads, HD, ld_q, 1, box);
  if (err == cudaSuccess)
    err = keys ? head_map(&map_v, a.v, a.rows_k, b.kv_heads, HD, a.ld_v, 1, box)
               : head_map(&map_v, q, a.rows_q, a.heads, HD, ld_q, 1, box);
  if (err != cudaSuccess) return err;
  int sms = 0;
  err = persistent_blocks(reinterpret_cast<const void*>(&attention_blocks_kernel<HD>), kThreads, S::kSmem,
                          int64_t{1} << 30, &sms);
  if (err != cudaSuccess) return err;
  const int64_t pairs = most_pairs(a);
  // The last units may be split in their row tiles where sequences have more than one of these on average (2,040
  // tokens of 8 heads, 64 units: 35 us, 43 without; 4 chunks, 640: 160 and 162), unless a CTA has so many units
  // that the last hardly matters.
  int64_t halves = 0;
  if (a.batch <= 32 && a.rows_q > static_cast<int64_t>(a.batch) * a.tokens && pairs * a.tile_groups < int64_t{16} * sms) {
    halves = most_halves((a.rows_q + 2 * a.tokens - 1) / (2 * a.tokens) * a.tile_groups, pairs * a.tile_groups, sms);
    if (halves > 0) a.split_sms = sms;
  }
  const int64_t blocks = pairs * a.tile_groups + halves;   // (below 2^31, see the API; halves only where there are few)
  attention_blocks_kernel<HD><<<static_cast<unsigned>(blocks), kThreads, S::kSmem, stream>>>(map_q, map_k, map_v, a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attention_blocks(const BlockShape& b, const uint16_t* q, int64_t ld_q, const uint16_t* k,
                                    int64_t ld_k, const uint16_t* v, int64_t ld_v, const int32_t* blocks, float scale,
                                    uint16_t* o, float* lse, cudaStream_t stream) {
  Args a = tiles_of(b);
  a.lists = blocks;
  a.top = b.top;
  a.causal = b.causal;
  a.scale = scale;
  a.v = v;
  a.ld_v = ld_v;
  a.o = o;
  a.lse = lse;
  return b.head_dim == 64 ? launch<64>(b, q, ld_q, k, ld_k, a, stream) : launch<128>(b, q, ld_q, k, ld_k, a, stream);
}

int64_t attention_blocks_units(const BlockShape& b) {
  const Args a = tiles_of(b);
  return most_pairs(a) * a.tile_groups;
}

cudaError_t attention_blocks_error_flag(int* flag) {
  int zero = 0;
  cudaError_t err = cudaMemcpyFromSymbol(flag, g_blocks_fault, sizeof(int));
  if (err == cudaSuccess) err = cudaMemcpyToSymbol(g_blocks_fault, &zero, sizeof(int));
  return err;
}

}  // namespace h3q
