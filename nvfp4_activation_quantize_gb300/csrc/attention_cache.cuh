// attention_cache.cuh -- what the two kernels of attention over the paged cache share: the
// count of the work, the way from codes to fp16, and the join of the parts of a group that
// several CTAs' ranges cut.
//
// A value of the cache is E2M1 * E4M3 / gsf.  The product has at most six significant bits, so
// it is exact in fp16 (scaled by 2^-8: 2^-18 .. 10.5), and 1 / gsf goes into the softmax scale
// and into the output: keys and values enter the tensor cores without a rounding.  A query
// row is scaled by the power of two that brings its largest magnitude into [2^14, 2^15), where
// every bf16 value down to 2^-29 of it is exact in fp16.
#pragma once

#include <cmath>

#include "h3q_async.cuh"
#include "h3q_cache.cuh"
#include "h3q_device.cuh"
#include "h3q_internal.h"
#include "h3q_roles.cuh"
#include "h3q_softmax.cuh"

namespace h3q {
namespace cached {

constexpr float kPShift = 14.0f;  // parts and sums hold 2^14 * e^(x - m)
constexpr int kMergeWarps = 4;    // of a CTA of the joining kernel
constexpr int kWholeTiles = 2;    // tiles that one CTA takes rather than leave parts of
constexpr int kMergeRows = 4;     // that it joins, a warp each in the end

struct Args {
  PagedCache cache;
  PagedRows at;
  const uint16_t* q;
  int64_t ld_q;
  int64_t rows;
  int heads, group;        // query heads, and per key head
  int max_rows;
  const int64_t* mask;     // or nullptr
  const float* k_gsf;
  const float* v_gsf;
  float scale;
  uint16_t* o;
  float* lse;              // or nullptr
  float* part;             // workspace: [ctas][2][tile rows][head_dim] unnormalised outputs
  float* part_ml;          // [ctas][2][tile rows][2] maxima and sums
  struct Cut* cut;         // [ctas]
  int whole;               // no range cuts a group
};

// What the joining kernel needs to know of the group that the start of a CTA's range cuts:
// written by that CTA; valid for the first range's start inside the group.
struct Cut {
  int64_t begin, end;      // the group, in units of work
  int64_t total;           // of all groups
  int valid, ctas;
  int b, kv_head, row_tile, pad;
};

// One sequence as the work is counted.
struct Seq {
  int64_t row0;            // its first packed row
  int n;                   // rows that are computed
  int ctx;                 // keys before its new tokens; negative where it has more rows than keys, and
                           // -64 or less hides every key (a mask has 64 bits)
  int len;                 // keys in the cache
  int tiles, groups;       // key tiles; (key head, row tile) pairs
  int row_tiles;
};

__device__ __forceinline__ Seq sequence(const Args& a, int b, int tile_rows, int tile_keys) {
  Seq s;
  const int64_t c0 = a.at.cu[b], c1 = a.at.cu[b + 1];
  int64_t n = c1 - c0;
  const int64_t cap = a.at.max_pages << a.cache.page_shift;
  int64_t len = a.at.kv_len[b];
  s.ctx = len - n < -64 ? -64 : static_cast<int>(len - n > 0x7fffffff ? 0x7fffffff : len - n);
  if (n > a.max_rows) n = a.max_rows;
  if (c0 + n > a.rows) n = a.rows - c0;
  if (c0 < 0 || n < 0) n = 0;
  len = len < 0 ? 0 : len > cap ? cap : len;
  s.row0 = c0;
  s.n = static_cast<int>(n);
  s.len = static_cast<int>(len);
  s.tiles = s.len > tile_keys ? static_cast<int>((static_cast<int64_t>(s.len) + tile_keys - 1) / tile_keys) : 1;
  s.row_tiles = (s.n * a.group + tile_rows - 1) / tile_rows;
  s.groups = s.row_tiles * a.cache.kv_heads;
  return s;
}

__device__ __forceinline__ int64_t tiles_of(const Seq& s) { return static_cast<int64_t>(s.tiles) * s.groups; }

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Four bytes of two E2M1 codes -> four pairs of fp16 (exact).
__device__ __forceinline__ void codes_to_half(uint32_t w, uint32_t (&o)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
      : "r"(w));
}

// The low seven bits of an E4M3 byte as fp16: its exponent and mantissa in place, which
// is its value times 2^-8, subnormals included (and finite for all bits set).
__device__ __forceinline__ uint32_t scale_half(uint32_t byte) { return (byte & 0x7fu) << 7; }

// Power of two that brings magnitude bits m (of a bf16) into [2^14, 2^15); 1 for zero and for what is no number.
__device__ __forceinline__ float query_factor(uint32_t m) {
  const int e = m >> 7;            // biased exponent of the row's largest magnitude
  const int fe = e == 255 || m == 0 ? 127 : 268 - e > 254 ? 254 : 268 - e;
  return __uint_as_float(static_cast<uint32_t>(fe) << 23);
}

// 1 / f of a power of two f in [2^-126, 2^127].
__device__ __forceinline__ float inverse_power(float f) {
  const uint32_t e = __float_as_uint(f) >> 23;
  return __uint_as_float(e == 254 ? 0x00400000u : (254u - e) << 23);
}

// Largest magnitude (bits) of two bf16 pairs' worth of words, folded into m; all ones in an exponent win.
template <int N>
__device__ __forceinline__ uint32_t magnitude_bits(const uint32_t (&w)[N]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) m = absmax_bf16x2(m, w[i]) & 0x7fff7fffu;
  m = max(m & 0xffffu, m >> 16);   // magnitudes order as their bits
#pragma unroll
  for (int i = 0; i < N; ++i)      // (the paired maximum skips a NaN)
    if ((w[i] & 0x7f80u) == 0x7f80u || (w[i] & 0x7f800000u) == 0x7f800000u) m = 0x7f80u;
  return m;
}

// a / b of numbers that are not negative, which mostly have 32 bits.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? static_cast<uint32_t>(a) / static_cast<uint32_t>(b) : a / b;
}

// Sums over the CTA of two values a thread, and the exclusive prefixes of this thread.
struct Pair {
  int64_t tiles, groups;
};
template <int WARPS>
__device__ __forceinline__ Pair block_scan(Pair v, Pair* scratch, Pair* prefix) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Pair x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x.tiles, o), z = __shfl_up_sync(0xffffffffu, x.groups, o);
    if (lane >= o) x.tiles += y, x.groups += z;
  }
  if (lane == 31) scratch[warp] = x;
  __syncthreads();
  Pair before{0, 0}, total{0, 0};
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    const Pair y = scratch[w];
    if (w < warp) before.tiles += y.tiles, before.groups += y.groups;
    total.tiles += y.tiles, total.groups += y.groups;
  }
  __syncthreads();
  prefix->tiles = before.tiles + x.tiles - v.tiles;
  prefix->groups = before.groups + x.groups - v.groups;
  return total;
}

// The tiles of sequence s that lie before its x-th unit of work, where a group is `unit` of them: `cost`,
// then its tiles (or one for all of it).
__device__ __forceinline__ int64_t tiles_before(const Seq& s, int64_t unit, int cost, int64_t x) {
  if (x <= 0) return 0;
  if (x >= unit * s.groups) return tiles_of(s);
  const int64_t q = quotient(x, unit), r = x - q * unit - cost;
  return q * s.tiles + (r > 0 ? r : 0);
}

// A CTA's part of the work: `count` tiles, from tile `tile` of a group of sequence b on.
struct Range {
  Seq s;
  int b, group, tile;
  int count;               // (2^31 tiles would be minutes)
  __device__ __forceinline__ int kv_head() const { return group / s.row_tiles; }
  // tiles of the group that are in the range
  __device__ __forceinline__ int here() const {
    return min(count, s.tiles - tile);
  }
  // On by n tiles, at most to the end of the group.
  __device__ __forceinline__ void advance(const Args& a, int n, int tile_rows, int tile_keys) {
    count -= n;
    tile += n;
    if (tile < s.tiles || count == 0) return;
    tile = 0;
    if (++group < s.groups) return;
    group = 0;
    do {
      s = sequence(a, ++b, tile_rows, tile_keys);
    } while (s.groups == 0);
  }
};

template <int WARPS>
struct PlanScratch {
  Pair scan[WARPS];
  int64_t base;            // units before the first range's sequence
  int64_t first, last;     // tiles before the range, and before its end
  int b;
};

// The range of this CTA, and its entry of a.cut; false for one that has nothing to do.  The work is
// counted in tiles, and COST more for each group (its queries, its join, its output): equal counts
// are equal times whether a range is one long group or many short ones.  Where there are no more
// tiles than CTAs each takes one.  With a.whole groups are counted instead.  The whole CTA calls it.
template <int WARPS, int COST>
__device__ __forceinline__ bool plan(const Args& a, int tile_rows, int tile_keys, PlanScratch<WARPS>& sh, Range& r) {
  const bool once = a.at.batch <= WARPS * 32;   // a sequence a thread
  Seq s;
  Pair mine, prefix, sum{0, 0};
  auto count = [&](int b0) {
    const int b = b0 + threadIdx.x;
    mine = Pair{0, 0};
    if (b < a.at.batch) {
      s = sequence(a, b, tile_rows, tile_keys);
      mine = Pair{tiles_of(s), s.groups};
    }
    return block_scan<WARPS>(mine, sh.scan, &prefix);
  };
  for (int b0 = 0; b0 < a.at.batch; b0 += WARPS * 32) {
    const Pair here = count(b0);
    sum.tiles += here.tiles, sum.groups += here.groups;
  }
  const int64_t tiles = sum.tiles, groups = sum.groups;
  const int cost = a.whole || tiles <= gridDim.x ? 0 : COST;
  const int64_t total = a.whole ? groups : tiles + cost * groups;
  auto unit_of = [&](const Seq& q) { return a.whole ? int64_t{1} : static_cast<int64_t>(q.tiles) + cost; };
  auto units_of = [&](const Pair& p) { return a.whole ? p.groups : p.tiles + cost * p.groups; };
  const int64_t most = total / (cost + 1);   // (a range has a tile: it is longer than cost)
  const int ctas = static_cast<int>(most < gridDim.x ? most : gridDim.x);
  if (static_cast<int>(blockIdx.x) >= ctas) {
    if (threadIdx.x == 0) a.cut[blockIdx.x].valid = 0;
    return false;
  }
  const int64_t t0 = quotient(total * blockIdx.x, ctas), t1 = quotient(total * (blockIdx.x + 1), ctas);
  Pair base{0, 0};
  for (int b0 = 0; b0 < a.at.batch && units_of(base) < t1; b0 += WARPS * 32) {
    const Pair here = once ? sum : count(b0);
    const int64_t first = base.tiles + prefix.tiles, at = units_of(base) + units_of(prefix), end = at + units_of(mine);
    if (at <= t0 && t0 < end) {
      sh.b = b0 + threadIdx.x;
      sh.base = at;
      sh.first = first + tiles_before(s, unit_of(s), cost, t0 - at);
    }
    if (at < t1 && t1 <= end) sh.last = first + tiles_before(s, unit_of(s), cost, t1 - at);
    base.tiles += here.tiles, base.groups += here.groups;
  }
  __syncthreads();
  r.count = static_cast<int>(sh.last - sh.first);
  r.b = sh.b;
  r.s = sequence(a, r.b, tile_rows, tile_keys);
  const int64_t unit = unit_of(r.s);
  r.group = static_cast<int>(quotient(t0 - sh.base, unit));
  const int64_t begin = sh.base + r.group * unit;
  r.tile = t0 - begin > cost ? static_cast<int>(t0 - begin) - cost : 0;
  if (threadIdx.x == 0) {
    Cut c;
    c.begin = begin;
    c.end = begin + unit;
    c.total = total;
    c.ctas = ctas;
    c.b = r.b;
    c.kv_head = r.kv_head();
    c.row_tile = r.group % r.s.row_tiles;
    c.valid = r.tile > 0 && quotient(total * (blockIdx.x - 1), ctas) <= begin + cost;   // blockIdx.x > 0 where tile > 0
    c.pad = 0;
    a.cut[blockIdx.x] = c;
  }
  return true;
}

// Joins the parts of the groups that the ranges' starts cut: CTA (c, r) takes kMergeRows rows of
// the group that the start of range c is the first to cut.  Its warps take the parts in turn
// (a group of 120,000 keys has 57), and are added up in their order.
template <int HD, int ROWS, int KEYS>
__global__ void __launch_bounds__(kMergeWarps * 32) join_parts_kernel(const Args a) {
  constexpr int kPer = HD / 32;
  __shared__ float sum[kMergeWarps][kMergeRows][HD];
  __shared__ float sum_l[kMergeWarps][kMergeRows];
  after_stream();   // the parts are written
  const int c = blockIdx.x + 1;
  const Cut cut = a.cut[c];
  if (!cut.valid) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rho0 = blockIdx.y * kMergeRows;
  const Seq s = sequence(a, cut.b, ROWS, KEYS);
  const int row0 = cut.row_tile * ROWS + rho0;
  if (row0 >= s.n * a.group) return;
  // the first range's part is its last segment: slot 0 if the range began in this group too
  const int64_t prev0 = quotient(cut.total * (c - 1), cut.ctas);
  const int64_t first = static_cast<int64_t>(c - 1) * 2 + (prev0 >= cut.begin ? 0 : 1);
  // one past the last range that starts inside the group: total * last / ctas < end
  const int64_t past = quotient(cut.end * cut.ctas + cut.total - 1, cut.total);
  const int last = static_cast<int>(past < cut.ctas ? past : cut.ctas);
  auto slot = [&](int k) { return (k == c - 1 ? first : static_cast<int64_t>(k) * 2) * ROWS + rho0; };
  const float2* ml = reinterpret_cast<const float2*>(a.part_ml);
  float top = -INFINITY;   // of row lane / 8
#pragma unroll 4
  for (int k = c - 1 + (lane & 7); k < last; k += 8) top = fmaxf(top, ml[slot(k) + (lane >> 3)].x);
#pragma unroll
  for (int o = 1; o <= 4; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  float m[kMergeRows], l[kMergeRows], v[kMergeRows][kPer];
#pragma unroll
  for (int r = 0; r < kMergeRows; ++r) {
    m[r] = __shfl_sync(0xffffffffu, top, 8 * r);
    l[r] = 0.0f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[r][i] = 0.0f;
  }
#pragma unroll 2
  for (int k = c - 1 + warp; k < last; k += kMergeWarps) {
    const int64_t at = slot(k);
#pragma unroll
    for (int r = 0; r < kMergeRows; ++r) {
      const float2 x = ml[at + r];
      const float f = x.x == -INFINITY ? 0.0f : ex2(__fadd_rn(x.x, -m[r]));
      l[r] = __fmaf_rn(x.y, f, l[r]);
      const float* src = a.part + (at + r) * HD + lane * kPer;
#pragma unroll
      for (int i = 0; i < kPer; i += 2) {
        const float2 y = *reinterpret_cast<const float2*>(src + i);
        v[r][i] = __fmaf_rn(y.x, f, v[r][i]);
        v[r][i + 1] = __fmaf_rn(y.y, f, v[r][i + 1]);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < kMergeRows; ++r) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) sum[warp][r][lane * kPer + i] = v[r][i];
    if (lane == 0) sum_l[warp][r] = l[r];
  }
  __syncthreads();
  // a warp a row
  if (row0 + warp >= s.n * a.group) return;
  const float mw = __shfl_sync(0xffffffffu, top, 8 * warp);
  float lw = 0.0f, o[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) o[i] = 0.0f;
#pragma unroll
  for (int w = 0; w < kMergeWarps; ++w) {
    lw = __fadd_rn(lw, sum_l[w][warp]);
#pragma unroll
    for (int i = 0; i < kPer; ++i) o[i] = __fadd_rn(o[i], sum[w][warp][lane * kPer + i]);
  }
  const int tok = (row0 + warp) / a.group;
  const int head = cut.kv_head * a.group + (row0 + warp) - tok * a.group;
  const int64_t out_row = s.row0 + tok;
  const float f = lw == 0.0f ? 0.0f : __fdiv_rn(1.0f, lw);
  const float v_factor = __fdiv_rn(256.0f, *a.v_gsf);   // (their product may be too small for fp32)
  uint16_t* dst = a.o + (out_row * a.heads + head) * HD + lane * kPer;
#pragma unroll
  for (int i = 0; i < kPer; i += 2)
    *reinterpret_cast<uint32_t*>(dst + i) =
        float2_to_bf16x2(make_float2(__fmul_rn(__fmul_rn(o[i], f), v_factor), __fmul_rn(__fmul_rn(o[i + 1], f), v_factor)));
  if (a.lse != nullptr && lane == 0)
    a.lse[head * a.rows + out_row] =
        lw == 0.0f ? -INFINITY : __fmul_rn(__fadd_rn(mw, __fadd_rn(log2f(lw), -kPShift)), kLn2);
}

// Whether ranges are of whole groups, so that nothing has to be joined: the tables hold one tile a
// sequence; or two, and there is a CTA for every group.  (One token, 2 key heads of 64, GPU time: 101
// positions 7.2 us with the joining kernel, 6.2 without; 301 positions, two tiles, 8.9 and 8.7; 777, four,
// 9.1 and 13.7.  On the host the second launch is 2.4 us.)
inline bool whole_groups(const Args& a, int blocks, int tile_rows, int tile_keys) {
  const int64_t cap = a.at.max_pages << a.cache.page_shift;
  const int64_t row_tiles = (static_cast<int64_t>(a.max_rows) * a.group + tile_rows - 1) / tile_rows;
  return cap <= tile_keys || (cap <= kWholeTiles * tile_keys && row_tiles * a.cache.kv_heads <= blocks / a.at.batch);
}

// The kernel that joins the parts, after the one before it on the stream.
template <int HD, int ROWS, int KEYS>
cudaError_t launch_join(const Args& a, int blocks, cudaStream_t stream) {
  return launch_early(&join_parts_kernel<HD, ROWS, KEYS>, dim3(static_cast<unsigned>(blocks - 1), ROWS / kMergeRows, 1),
                      kMergeWarps * 32, 0, stream, a);
}

// Addresses of the workspace's regions for CTAs of `rows` rows.
inline void place_workspace(Args& a, uint8_t* workspace, int ctas, int rows) {
  a.cut = reinterpret_cast<Cut*>(workspace);
  static_assert(sizeof(Cut) <= kCacheAttentionCutBytes, "workspace");
  a.part_ml = reinterpret_cast<float*>(workspace + kCacheAttentionCutBytes * kCacheAttentionMaxCtas);
  a.part = a.part_ml + static_cast<int64_t>(ctas) * 2 * rows * 2;
}

}  // namespace cached

// The kernel for many rows (attention_cache_wide.cu): head_dim 64 or 128, and a workspace for
// more than 16 rows a key head.
cudaError_t launch_cache_attention_wide(const cached::Args& a, uint8_t* workspace, cudaStream_t stream);
cudaError_t cache_attention_wide_error_flag(int* flag);

}  // namespace h3q
