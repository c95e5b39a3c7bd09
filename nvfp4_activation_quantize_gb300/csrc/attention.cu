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
//                     reads the row, moves the reference maximum only when the row's
//                     maximum has grown by more than 2^8 (weights then stay below 2^8 and
//                     the output is rescaled rarely), writes the weights as bf16
//                     over S, and sums them in fp32 unrounded.  A weight's rounding to
//                     bf16 (at most 2^-8 of it, the type of V that it is multiplied with) is
//                     the format's; maxima, sums and outputs are fp32.  At the end
//                     it scales its row of O and stores it.
//   warp 8, one lane  TMA: Q once, then K and V tiles in a ring
//   warp 9, one lane  the products: S = Q K^T (operands in shared memory), O += P V (P in
//                     TMEM, V as it lies in memory: its rows are the reduction)
//   warps 10, 11      V tiles that some row does not see whole: rows past the sequence's end
//                     become zero, and so do values that are no numbers (0 * NaN
//                     would reach rows that do not see them); the epilogue adds these back
//                     for the rows that do
//
// Every wait is bounded: one that runs out sets a device flag and tells the other roles
// to stop; the CTA drains what it has in flight, frees its TMEM and returns.
#include <cmath>

#include "h3q_async.cuh"
#include "h3q_device.cuh"
#include "h3q_internal.h"
#include "h3q_tcgen05.cuh"

namespace h3q {
namespace {

constexpr int kThreads = 384;
constexpr int kTmaWarp = 8;
constexpr int kMmaWarp = 9;
constexpr int kCheckWarp0 = 10;
constexpr int kCheckThreads = 64;
constexpr int kTileRows = 128;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kSlack = 8.0f;  // how far (log2) a row's maximum may pass its reference

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
  static constexpr int kOffBar = kOffKv + kStages * kKvBytes;
  static constexpr int kBars = 4 * kStages + 2 + 2 + 2 + 2 + 1;  // full, empty, v_raw, v_ok, q, s, p, o, drain
  static constexpr int kOffMisc = kOffBar + 8 * kBars;
  static constexpr int kSmem = kOffMisc + 64 + 1024;
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
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t start = now_ns();
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 255u) == 0) {
      if (*abort) return false;
      if (now_ns() - start > kWaitNs) break;
    }
  }
  *abort = 1;
  atomicExch(&g_attention_fault, 1);
  return false;
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// The CTA's work: one sequence's pair of row tiles of one group of heads.
struct Unit {
  int64_t q0, k0;        // first packed rows of the sequence
  int n, len;            // its queries and keys
  int head0;             // first head of the tile
  int tok[2];            // first token of each row tile
  int tiles[2];          // key tiles that each reads (0: none, or no rows)
  int partial[2];        // first of them that some row does not see whole
};

__device__ __forceinline__ int clamp_keys(int64_t x, int len) {
  return x < 0 ? 0 : x > len ? len : static_cast<int>(x);
}

template <int HD>
__device__ __forceinline__ Unit unit_of_block(const Args& a, int b, int64_t rank) {
  using S = Shape<HD>;
  Unit u;
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
    u.tok[x] = qt * span + x * a.tokens;
    const bool any = x < S::kTiles && u.tok[x] < u.n;
    const int last = u.tok[x] + a.tokens < u.n ? u.tok[x] + a.tokens - 1 : u.n - 1;
    const int most = !any ? 0 : a.causal ? clamp_keys(last + shift, u.len) : u.len;
    const int least = a.causal ? clamp_keys(u.tok[x] + shift, u.len) : u.len;
    u.tiles[x] = (most + S::kKeys - 1) / S::kKeys;
    u.partial[x] = least / S::kKeys;
  }
  return u;
}

__device__ __forceinline__ int64_t units_of(const Args& a, int b, int span) {
  const int64_t q0 = a.cu_q[b];
  int64_t n = static_cast<int64_t>(a.cu_q[b + 1]) - q0;
  if (n > a.rows_q - q0) n = a.rows_q - q0;
  if (q0 < 0 || n < 0) n = 0;
  return (n + span - 1) / span * a.tile_groups;
}

// One key tile of one row: S in, weights out, over S.  `seen`: how many of the tile's keys the row sees
// (MASK).  Returns through m_ref and l; `alpha` is what the row of O has to be scaled with.
template <int KEYS, bool MASK>
__device__ __forceinline__ float softmax_tile(uint32_t taddr, int seen, float c, float& m_ref, float& l) {
  uint32_t s[KEYS / 32][32];
#pragma unroll
  for (int i = 0; i < KEYS / 32; ++i) tc_load32(taddr + 32 * i, s[i]);
  tc_wait_load();
  float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int i = 0; i < KEYS / 32; ++i)
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      if (MASK && 32 * i + j >= seen) s[i][j] = 0xff800000u;
      m[j & 3] = fmaxf(m[j & 3], __uint_as_float(s[i][j]));
    }
  const float top = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
  float alpha = 1.0f;
  if (__fmul_rn(__fadd_rn(top, -m_ref), c) > kSlack) {   // (false where both are -inf)
    alpha = ex2(__fmul_rn(__fadd_rn(m_ref, -top), c));
    m_ref = top;
    l = __fmul_rn(l, alpha);
  }
  const float base = m_ref == -INFINITY ? 0.0f : -__fmul_rn(m_ref, c);
  const float2 c2 = make_float2(c, c), b2 = make_float2(base, base);
  float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int i = 0; i < KEYS / 32; ++i) {
    uint32_t w[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      float2 p = fma2(make_float2(__uint_as_float(s[i][2 * j]), __uint_as_float(s[i][2 * j + 1])), c2, b2);
      p.x = ex2(p.x);
      p.y = ex2(p.y);
      sum = add2(sum, p);
      w[j] = float2_to_bf16x2(p);
    }
    tc_store16(taddr + 16 * i, w);
  }
  l = __fadd_rn(l, __fadd_rn(sum.x, sum.y));
  return alpha;
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
  const uint32_t bar_vraw = bar_empty + 8 * S::kStages;    // a V tile that the checkers look at first ...
  const uint32_t bar_vok = bar_vraw + 8 * S::kStages;      // ... and have passed on
  const uint32_t bar_q = bar_vok + 8 * S::kStages;         // + 8 * row tile
  const uint32_t bar_s = bar_q + 16;                       // + 8 * S buffer
  const uint32_t bar_p = bar_s + 16;
  const uint32_t bar_o = bar_p + 16;                       // + 8 * row tile
  const uint32_t bar_drain = bar_o + 16;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::kOffMisc);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + S::kOffMisc + 4);
  int* bad_v = reinterpret_cast<int*>(smem + S::kOffMisc + 8);
  int* found_b = reinterpret_cast<int*>(smem + S::kOffMisc + 12);
  int64_t* found_rank = reinterpret_cast<int64_t*>(smem + S::kOffMisc + 16);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // ---- which unit: warp 0 counts the sequences' units, 32 at a time
  if (warp == 0) {
    const int span = a.tokens * S::kTiles;
    int64_t before = 0;
    int found = -1;
    for (int b0 = 0; b0 < a.batch && found < 0; b0 += 32) {
      const int b = b0 + lane;
      const int64_t mine = b < a.batch ? units_of(a, b, span) : 0;
      int64_t upto = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
      const int64_t u = static_cast<int64_t>(blockIdx.x) - before;
      const uint32_t hit = __ballot_sync(0xffffffffu, u >= upto - mine && u < upto);
      if (hit) {
        found = b0 + __ffs(hit) - 1;
        if (lane == __ffs(hit) - 1) *found_rank = u - (upto - mine);
      }
      before += __shfl_sync(0xffffffffu, upto, 31);
    }
    if (lane == 0) *found_b = found;
  }
  if (threadIdx.x == 32) {
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(bar_full + 8 * i, 1);
      mbar_init(bar_empty + 8 * i, 1);
      mbar_init(bar_vraw + 8 * i, 1);
      mbar_init(bar_vok + 8 * i, kCheckThreads);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar_q + 8 * i, 1);
      mbar_init(bar_s + 8 * i, 1);
      mbar_init(bar_p + 8 * i, kTileRows);
      mbar_init(bar_o + 8 * i, 1);
    }
    mbar_init(bar_drain, 1);
    *abort = 0;
    *bad_v = 0;
    mbar_init_fence();
  }
  __syncthreads();
  if (*found_b < 0) return;   // more CTAs than units
  const Unit u = unit_of_block<HD>(a, *found_b, *found_rank);
  const int tiles = u.tiles[0] > u.tiles[1] ? u.tiles[0] : u.tiles[1];
  const int partial = u.tiles[0] == 0 ? u.partial[1] : u.partial[0];   // a causal tile 0 sees less
  const int kv_head = u.head0 / a.group;
  // V tiles take every other stage of the ring; those from `partial` on are the last, and
  // arrive on barriers of their own, whose phases count them alone.
  auto checked_parity = [&](int j) { return static_cast<uint32_t>((j - partial) / (S::kStages / 2)) & 1u; };
  if (warp == kMmaWarp) {   // the whole warp allocates the CTA's TMEM (one CTA per SM)
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == kTmaWarp) {
    if (lane == 0) {
      bool ok = true;
      const int rows = a.tokens * a.heads_per_tile;
      auto load_q = [&](int x) {
        if (u.tiles[x] == 0) return;
        mbar_expect_tx(bar_q + 8 * x, rows * HD * 2);
        for (int h = 0; h < S::kHalves; ++h)
          tma_load_3d(base + x * S::kQBytes + h * (kTileRows * 128), &map_q, 64 * h, u.head0,
                      static_cast<int>(u.q0 + u.tok[x]), bar_q + 8 * x);
      };
      load_q(0);
      int pos = 0;
      for (; pos < 2 * tiles; ++pos) {   // K0 V0 K1 V1 ...
        const int stage = pos % S::kStages;
        if (!(ok = wait_or_abort(bar_empty + 8 * stage, ((pos / S::kStages) & 1) ^ 1u, abort))) break;
        const uint32_t bar = ((pos & 1) && (pos >> 1) >= partial ? bar_vraw : bar_full) + 8 * stage;
        mbar_expect_tx(bar, S::kKvBytes);
        for (int h = 0; h < S::kHalves; ++h)
          tma_load_3d(base + S::kOffKv + stage * S::kKvBytes + h * (S::kKeys * 128), pos & 1 ? &map_v : &map_k, 64 * h,
                      kv_head, static_cast<int>(u.k0) + (pos >> 1) * S::kKeys, bar);
        if (pos == 0 && S::kTiles == 2) load_q(1);
      }
      // Before the CTA goes: every stage's last use is released (the products' commits
      // arrive here), and after an abort every copy issued has landed.
      for (int i = pos - S::kStages < 0 ? 0 : pos - S::kStages; i < pos; ++i) {
        const int stage = i % S::kStages;
        if (ok) {
          (void)wait_or_abort(bar_empty + 8 * stage, (i / S::kStages) & 1, abort);
        } else if ((i & 1) && (i >> 1) >= partial) {
          (void)wait_bounded(bar_vraw + 8 * stage, checked_parity(i >> 1));
        } else {
          (void)wait_bounded(bar_full + 8 * stage, (i / S::kStages) & 1);
        }
      }
      if (!ok)
        for (int x = 0; x < S::kTiles; ++x)
          if (u.tiles[x] != 0 && (x == 0 || pos > 0)) (void)wait_bounded(bar_q + 8 * x, 0);
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    if (lane == 0 && tiles > 0) {
      bool ok = true;
      auto kv = [&](int pos) { return base + S::kOffKv + (pos % S::kStages) * S::kKvBytes; };
      auto wait_kv = [&](int pos) {
        return wait_or_abort(bar_full + 8 * (pos % S::kStages), (pos / S::kStages) & 1, abort);
      };
      auto wait_v = [&](int j) {
        const int pos = 2 * j + 1;
        if (j < partial) return wait_kv(pos);
        return wait_or_abort(bar_vok + 8 * (pos % S::kStages), checked_parity(j), abort);
      };
      auto s_product = [&](int x, int buf, int j) {   // S[buf] = Q[x] K[j]^T
        const uint32_t q = base + x * S::kQBytes, k = kv(2 * j);
#pragma unroll
        for (int i = 0; i < HD / 16; ++i)
          mma_ss(tmem + buf * S::kS, operand_desc(q + (i / 4) * (kTileRows * 128) + (i % 4) * 32),
                 operand_desc(k + (i / 4) * (S::kKeys * 128) + (i % 4) * 32), S::kIdescS, i > 0);
        tc_commit(bar_s + 8 * buf);
      };
      auto o_product = [&](int x, int buf, int j) {   // O[x] += P[buf] V[j]
        const uint32_t v = kv(2 * j + 1);
#pragma unroll
        for (int i = 0; i < S::kKeys / 16; ++i)       // rows of V 16 i ..: two 8-row groups of 1,024 bytes
          mma_ts(tmem + S::kO + x * HD, tmem + buf * S::kS + 8 * i, smem_desc(v + i * 2048, S::kKeys * 128, 1024, 2),
                 S::kIdescO, j > 0 || i > 0);
      };
      auto release = [&](int pos) { tc_commit(bar_empty + 8 * (pos % S::kStages)); };
      if constexpr (S::kTiles == 2) {
        const int n0 = u.tiles[0], n1 = u.tiles[1];
        ok = wait_kv(0);
        if (ok && n0 > 0 && (ok = wait_or_abort(bar_q, 0, abort))) {
          tc_fence_after();
          s_product(0, 0, 0);
        }
        if (ok && n1 > 0 && (ok = wait_or_abort(bar_q + 8, 0, abort))) {
          tc_fence_after();
          s_product(1, 1, 0);
        }
        if (ok) release(0);
        for (int j = 0; j < tiles && ok; ++j) {
          for (int x = 0; x < 2 && ok; ++x) {
            const int n = x == 0 ? n0 : n1, other = x == 0 ? n1 : n0;
            if (j >= n) continue;
            const bool first = x == 0 || j >= n0;             // the first of the tiles that use V[j]
            const bool last = x == 1 || j >= other;
            if (first && !(ok = wait_v(j))) break;
            if (!(ok = wait_or_abort(bar_p + 8 * x, j & 1, abort))) break;
            tc_fence_after();
            o_product(x, x, j);
            if (last) release(2 * j + 1);
            if (j + 1 < n) {
              if (!(ok = wait_kv(2 * j + 2))) break;          // (a phase already seen to be complete stays so)
              tc_fence_after();
              s_product(x, x, j + 1);
              if (x == 1 || j + 1 >= other) release(2 * j + 2);
            } else {
              tc_commit(bar_o + 8 * x);
            }
          }
        }
      } else {
        ok = wait_kv(0) && wait_or_abort(bar_q, 0, abort);
        if (ok) {
          tc_fence_after();
          s_product(0, 0, 0);
          release(0);
        }
        for (int j = 0; j < tiles && ok; ++j) {
          if (j + 1 < tiles) {   // the next S goes into the other buffer while this one's softmax runs
            if (!(ok = wait_kv(2 * j + 2))) break;
            tc_fence_after();
            s_product(0, (j + 1) & 1, j + 1);
            release(2 * j + 2);
          }
          if (!(ok = wait_v(j))) break;
          if (!(ok = wait_or_abort(bar_p + 8 * (j & 1), (j >> 1) & 1, abort))) break;
          tc_fence_after();
          o_product(0, j & 1, j);
          release(2 * j + 1);
          tc_commit(bar_o);
        }
      }
      if (!ok) {   // let what is issued finish before the TMEM is freed
        tc_commit(bar_drain);
        (void)wait_bounded(bar_drain, 0);
      }
    }
    __syncwarp();
  } else if (warp >= kCheckWarp0) {
    const int tid = threadIdx.x - kCheckWarp0 * 32;
    for (int j = partial; j < tiles; ++j) {
      const int pos = 2 * j + 1, stage = pos % S::kStages;
      if (!__all_sync(0xffffffffu, wait_or_abort(bar_vraw + 8 * stage, checked_parity(j), abort))) break;
      uint8_t* v = smem + S::kOffKv + stage * S::kKvBytes;
      const int live = u.len - j * S::kKeys;       // rows of the sequence in this tile
      bool bad = false;
      for (int i = tid; i < S::kKvBytes / 16; i += kCheckThreads) {
        uint4* p = reinterpret_cast<uint4*>(v) + i;
        const int row = (i >> 3) % S::kKeys;       // 128 bytes of a row are 8 pieces, whatever their order
        if (row >= live) {
          *p = make_uint4(0, 0, 0, 0);
        } else if (a.causal) {
          uint4 w = *p;
          // a half whose exponent is all ones carries into its top bit
          auto odd = [](uint32_t x) { return ((x & 0x7f807f80u) + 0x00800080u) & 0x80008000u; };
          if (odd(w.x) | odd(w.y) | odd(w.z) | odd(w.w)) {
            auto clean = [&](uint32_t x) {
              const uint32_t o = odd(x);
              return x & ~((o & 0x8000u ? 0xffffu : 0u) | (o & 0x80000000u ? 0xffff0000u : 0u));
            };
            *p = make_uint4(clean(w.x), clean(w.y), clean(w.z), clean(w.w));
            bad = true;
          }
        }
      }
      if (bad) atomicOr(bad_v, 1 << (j - partial));
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // the products read what was written here
      mbar_arrive(bar_vok + 8 * stage);
    }
  } else if (warp < 4 * S::kTiles) {
    // ---- softmax and epilogue of one row tile
    const int x = warp >> 2;
    const int row = (warp & 3) * 32 + lane;
    const int tok = u.tok[x] + row / a.heads_per_tile;
    const int head = u.head0 + row % a.heads_per_tile;
    const bool valid = row < a.tokens * a.heads_per_tile && tok < u.n;
    const int sees = !valid ? 0 : a.causal ? clamp_keys(static_cast<int64_t>(tok) + u.len - u.n + 1, u.len) : u.len;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t taddr_o = lane_base + S::kO + x * HD;
    const float c = fmaxf(__fmul_rn(a.scale, kLog2e), 0x1p-126f);   // never 0: a hidden key's -inf stays one
    const int n = u.tiles[x];
    float m_ref = -INFINITY, l = 0.0f;
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      const int buf = S::kTiles == 2 ? x : j & 1;
      const uint32_t parity = S::kTiles == 2 ? j & 1 : (j >> 1) & 1;
      if (!(ok = __all_sync(0xffffffffu, wait_or_abort(bar_s + 8 * buf, parity, abort)))) break;
      tc_fence_after();
      const uint32_t taddr = lane_base + buf * S::kS;
      const float alpha = j >= u.partial[x] ? softmax_tile<S::kKeys, true>(taddr, sees - j * S::kKeys, c, m_ref, l)
                                            : softmax_tile<S::kKeys, false>(taddr, 0, c, m_ref, l);
      // O is at rest: with two tiles S[j] was issued after P[j-1] V[j-1]; with one it was
      // issued before, so that product is waited for (each in turn: a phase that is two
      // behind looks like one to come).
      if constexpr (S::kTiles == 1) {
        if (j > 0 && !(ok = __all_sync(0xffffffffu, wait_or_abort(bar_o, (j - 1) & 1, abort)))) break;
        tc_fence_after();
      }
      if (j > 0 && __any_sync(0xffffffffu, alpha != 1.0f)) {
#pragma unroll 1
        for (int i = 0; i < HD; i += 32) {
          uint32_t o[32];
          tc_load32(taddr_o + i, o);
          tc_wait_load();
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__fmul_rn(__uint_as_float(o[k]), alpha));
          tc_store32(taddr_o + i, o);
        }
      }
      tc_wait_store();
      tc_fence_before();
      mbar_arrive(bar_p + 8 * buf);
    }
    if (n > 0 && ok) {
      const uint32_t parity = S::kTiles == 2 ? 0 : (n - 1) & 1;
      ok = __all_sync(0xffffffffu, wait_or_abort(bar_o + 8 * x, parity, abort));
      tc_fence_after();
    }
    if (ok) {
      const float inv = l == 0.0f ? 0.0f : __fdiv_rn(1.0f, l);
      const int64_t out_row = u.q0 + tok;
      const int bad = *static_cast<volatile int*>(bad_v);
      uint16_t* dst = a.o + (out_row * a.heads + head) * HD;
#pragma unroll 1
      for (int i = 0; i < HD; i += 32) {
        uint32_t o[32];
        if (n > 0) {
          __syncwarp();
          tc_load32(taddr_o + i, o);
          tc_wait_load();
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = 0;
        }
        if (bad != 0 && valid) {   // values that are no numbers, of keys that this row sees
          for (int j = partial; j < n; ++j) {
            if (!(bad >> (j - partial) & 1)) continue;
            const int end = sees < (j + 1) * S::kKeys ? sees : (j + 1) * S::kKeys;
            for (int key = j * S::kKeys; key < end; ++key) {
              const uint16_t* src = a.v + (u.k0 + key) * a.ld_v + static_cast<int64_t>(kv_head) * HD + i;
#pragma unroll
              for (int k = 0; k < 32; ++k) {
                const uint32_t w = src[k];
                if ((w & 0x7f80u) == 0x7f80u)
                  o[k] = __float_as_uint(__fadd_rn(__uint_as_float(o[k]), __uint_as_float(w << 16)));
              }
            }
          }
        }
        if (valid) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t w[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const float lo = __uint_as_float(o[16 * half + 2 * k]), hi = __uint_as_float(o[16 * half + 2 * k + 1]);
              w[k] = l == 0.0f ? 0u : float2_to_bf16x2(make_float2(__fmul_rn(lo, inv), __fmul_rn(hi, inv)));
            }
            store16(dst + i + 16 * half, make_uint4(w[0], w[1], w[2], w[3]));
            store16(dst + i + 16 * half + 8, make_uint4(w[4], w[5], w[6], w[7]));
          }
        }
      }
      if (valid && a.lse != nullptr)
        a.lse[head * a.rows_q + out_row] =
            l == 0.0f ? -INFINITY : __fmul_rn(__fadd_rn(__fmul_rn(m_ref, c), log2f(l)), kLn2);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
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
  // at most this many pairs of row tiles, however the rows fall into sequences
  const int64_t pairs = (a.rows_q + a.batch * (span - 1)) / span;
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
