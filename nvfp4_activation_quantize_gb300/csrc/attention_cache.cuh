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
#include "h3q_softmax.cuh"

namespace h3q {
namespace cached {

constexpr float kPShift = 14.0f;  // parts and sums hold 2^14 * e^(x - m)
constexpr int kMergeWarps = 4;    // rows per CTA of the joining kernel

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
};

// What the joining kernel needs to know of the group that the start of a CTA's range cuts:
// written by that CTA; valid for the first range's start inside the group.
struct Cut {
  int64_t begin, end;      // the group's tiles
  int64_t total;           // all tiles
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

// A sum over the CTA of one value a thread, and the exclusive prefix of this thread.
template <int WARPS>
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* scratch, int64_t* prefix) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) scratch[warp] = x;
  __syncthreads();
  int64_t before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) before += scratch[w];
    total += scratch[w];
  }
  __syncthreads();
  *prefix = before + x - v;
  return total;
}

// Joins the parts of the groups that the ranges' starts cut: CTA (c, r) takes the group
// that the start of range c is the first to cut, a warp each of its rows.
template <int HD, int ROWS, int KEYS>
__global__ void __launch_bounds__(kMergeWarps * 32) join_parts_kernel(const Args a) {
  constexpr int kPer = HD / 32;
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the parts are written
  const int c = blockIdx.x + 1;
  const Cut cut = a.cut[c];
  if (!cut.valid) return;
  const int lane = threadIdx.x & 31;
  const int rho = blockIdx.y * kMergeWarps + (threadIdx.x >> 5);
  const Seq s = sequence(a, cut.b, ROWS, KEYS);
  const int tile_row0 = cut.row_tile * ROWS;
  if (tile_row0 + rho >= s.n * a.group) return;
  // the first range's part is its last segment: slot 0 if the range began in this group too
  const int64_t prev0 = cut.total * (c - 1) / cut.ctas;
  const int64_t first = static_cast<int64_t>(c - 1) * 2 + (prev0 >= cut.begin ? 0 : 1);
  const float2* ml = reinterpret_cast<const float2*>(a.part_ml);
  int last = c;   // one past the last range that starts inside the group
  while (last < cut.ctas && cut.total * last / cut.ctas < cut.end) ++last;
  auto slot = [&](int k) { return (k == c - 1 ? first : static_cast<int64_t>(k) * 2) * ROWS + rho; };
  float m = -INFINITY;
  for (int k = c - 1 + lane; k < last; k += 32) m = fmaxf(m, ml[slot(k)].x);
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float use = m == -INFINITY ? 0.0f : m;
  float l = 0.0f, v[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) v[i] = 0.0f;
#pragma unroll 4
  for (int k = c - 1; k < last; ++k) {
    const float2 x = ml[slot(k)];
    const float f = x.x == -INFINITY ? 0.0f : ex2(__fadd_rn(x.x, -use));
    l = __fmaf_rn(x.y, f, l);
    const float* src = a.part + slot(k) * HD + lane * kPer;
#pragma unroll
    for (int i = 0; i < kPer; i += 2) {
      const float2 y = *reinterpret_cast<const float2*>(src + i);
      v[i] = __fmaf_rn(y.x, f, v[i]);
      v[i + 1] = __fmaf_rn(y.y, f, v[i + 1]);
    }
  }
  const int tok = (tile_row0 + rho) / a.group;
  const int head = cut.kv_head * a.group + (tile_row0 + rho) - tok * a.group;
  const int64_t out_row = s.row0 + tok;
  const float f = l == 0.0f ? 0.0f : __fdiv_rn(__fdiv_rn(256.0f, *a.v_gsf), l);
  uint16_t* dst = a.o + (out_row * a.heads + head) * HD + lane * kPer;
#pragma unroll
  for (int i = 0; i < kPer; i += 2)
    *reinterpret_cast<uint32_t*>(dst + i) =
        float2_to_bf16x2(make_float2(__fmul_rn(v[i], f), __fmul_rn(v[i + 1], f)));
  if (a.lse != nullptr && lane == 0)
    a.lse[head * a.rows + out_row] =
        l == 0.0f ? -INFINITY : __fmul_rn(__fadd_rn(m, __fadd_rn(log2f(l), -kPShift)), kLn2);
}


// The kernel that joins the parts, after the one before it on the stream.
template <int HD, int ROWS, int KEYS>
cudaError_t launch_join(const Args& a, int blocks, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks - 1), ROWS / kMergeWarps, 1);
  cfg.blockDim = dim3(kMergeWarps * 32, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_parts_kernel<HD, ROWS, KEYS>, a);
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
