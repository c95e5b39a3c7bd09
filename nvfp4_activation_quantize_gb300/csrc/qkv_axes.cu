// qkv_axes.cu -- QKV epilogue with rotary positions of several axes: bias, RMSNorm of each head
// with its weight, and a rotation by angles made from the rows' positions.
//
// Per row and head, in fp32 with one rounding to bf16 at the end:
//   x' = x + b;   n = x' * rsqrt(mean(x'^2) + eps) * w;
//   pair j = 0 .. ROT/2 - 1 belongs to axis a(j) and turns by p[a(j)] * f[j]:
//   (n_a, n_b) -> (n_a cos - n_b sin, n_a sin + n_b cos).
//
// The angle is taken in turns.  F[j] = f[j] / (2 pi) as a fraction of 2^64: the product of two
// 64-bit integers that wraps, p * F[j], is the turn's fraction with all whole turns gone, for
// positive and negative p, off by p times what F is.  (F comes from doubles: log2(theta), its quotient and product with the
// pair's number err by 2^-51 of an exponent of |log2 theta| at most, the power, scale and 2 pi by 2^-50 of f, a negative
// fraction's distance from a turn by 2^-54.)  So a position of a million is as exact as one of ten; only the fraction, in
// [-1/2, 1/2), is rounded to fp32.
//
// A warp makes the ROT/2 angles of its row once, each lane two of 64, and passes them through
// shared memory; the weights are folded into them,
//   out_i = rstd * (x'_i * A_i + x'_partner * B_i),  A_i = w_i cos, B_i = -+ w_partner sin,
// so a head costs two products a value.  A lane has 8 values of a head; a rotate-half partner is
// ROT/16 lanes away (a shuffle), an interleaved one in the same lane.
//
// Bound: every value is read and written once, 4 bytes, which is DRAM's time; the arithmetic, about
// 80 instructions for 256 values, runs beside it.  A unit of work is a row's heads of q, k or v, or some of
// them where there are few rows: all of q's, then k's, then v's, because DRAM reads and writes one
// tensor faster than three at once (65,280 rows of 56 heads of 128: 883 us, 6.4 TB/s, with the rows' three
// units together 929).  A warp's values land in a ring of its own in shared memory, a load of 1 KB ahead of
// the one that it works on, also of its next unit.
#include "h3q_async.cuh"
#include "h3q_device.cuh"
#include "h3q_internal.h"

namespace h3q {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 2;   // head groups that are loaded together
constexpr int kRing = 2;     // such loads of a warp: of one it works, the other is under way
constexpr int kMaxPairs = 128;

struct AxesArgs {
  const uint16_t* x[3];  // q, k, v
  int64_t ld[3];
  const uint16_t* bias[3];    // or nullptr
  const uint16_t* weight[2];  // q and k: [head_dim], or nullptr
  uint16_t* out[3];
  int heads[3];
  int units[3];               // of a row, for each tensor
  int unit_groups;            // head groups of a unit
  const int32_t* positions;   // [rows, axes]
  int axes;
  int rot;
  int norm;
  int64_t rows;
  float eps;
  RopeTurns turns;
};

// Eight values of a head, biased, in fp32.
__device__ __forceinline__ void biased(const uint4& xw, const uint4& bw, float2 (&x)[4]) {
  x[0] = add_bf16x2_f32(bw.x, bf16x2_to_float2(xw.x));
  x[1] = add_bf16x2_f32(bw.y, bf16x2_to_float2(xw.y));
  x[2] = add_bf16x2_f32(bw.z, bf16x2_to_float2(xw.z));
  x[3] = add_bf16x2_f32(bw.w, bf16x2_to_float2(xw.w));
}

constexpr uint32_t kMinusZeros = 0x80008000u;   // x + -0 = x, the sign of a zero included

// 8 * LPH values a head: LPH lanes each, 32 / LPH heads at a time.
template <int LPH, bool ILV>
__global__ void __launch_bounds__(kThreads, 4) qkv_axes_kernel(const __grid_constant__ AxesArgs a) {
  constexpr int kHd = 8 * LPH;
  constexpr int kHeadsPerWarp = 32 / LPH;
  __shared__ unsigned long long turns[kMaxPairs];
  __shared__ uint8_t axis[kMaxPairs];
  __shared__ __align__(16) float2 angles[kWarps][kHd / 2];   // cos, sin
  __shared__ uint4 ring[kWarps][kRing][kUnroll][32];         // (each lane reads what it has loaded)
  const int pairs = a.rot / 2;
  for (int j = threadIdx.x; j < pairs; j += kThreads) {
    turns[j] = a.turns.of_pair[j];
    axis[j] = a.turns.axis[j];
  }
  __syncthreads();

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = lane % LPH;                 // chunk of the head
  const int rot_chunks = a.rot >> 3, half = rot_chunks >> 1;
  const bool rotated = c < rot_chunks;
  const int src = (lane - c) + (c < half ? c + half : rotated ? c - half : c);   // rotate-half partner
  const int64_t units = a.rows * (a.units[0] + a.units[1] + a.units[2]);
  const int64_t nwarps = static_cast<int64_t>(gridDim.x) * kWarps;

  const int col0 = (lane / LPH) * kHd + c * 8;
  const int rounds = (pairs + 31) / 32;

  struct Unit {
    int64_t row;
    int tensor, g, g_end;   // head groups [g, g_end)
  };
  auto unit_of = [&](int64_t u) {
    Unit w;
    w.tensor = 0;
    while (u >= a.rows * a.units[w.tensor]) u -= a.rows * a.units[w.tensor++];   // (all of q, then k, then v)
    w.row = a.units[w.tensor] == 1 ? u : u / a.units[w.tensor];
    const int part = static_cast<int>(u - w.row * a.units[w.tensor]);
    const int all = (a.heads[w.tensor] + kHeadsPerWarp - 1) / kHeadsPerWarp;
    w.g = part * a.unit_groups;
    w.g_end = w.g + a.unit_groups < all ? w.g + a.unit_groups : all;
    return w;
  };

  int64_t u = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  if (u >= units) return;
  Unit w = unit_of(u), f = w;   // worked on; loaded
  int64_t fu = u;
  int slot = 0, fslot = 0;
  // The next load (zeros where there is no head), or none after the last unit's.
  auto load = [&]() {
    if (fu < units) {
      const uint16_t* const x = a.x[f.tensor] + f.row * a.ld[f.tensor] + col0;
#pragma unroll
      for (int j = 0; j < kUnroll; ++j) {
        const bool there = f.g + j < f.g_end && (f.g + j) * kHeadsPerWarp + lane / LPH < a.heads[f.tensor];
        const uint16_t* const from = there ? x + static_cast<int64_t>(f.g + j) * (kHeadsPerWarp * kHd) : a.x[f.tensor];
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(&ring[warp][fslot][j][lane])), "l"(from),
                     "r"(there ? 16 : 0)
                     : "memory");
      }
      fslot = (fslot + 1) % kRing;
      f.g += kUnroll;
      if (f.g >= f.g_end) {
        fu += nwarps;
        if (fu < units) f = unit_of(fu);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < kRing - 1; ++i) load();
  for (;;) {
    const int heads = a.heads[w.tensor];
    uint16_t* const out = a.out[w.tensor] + w.row * (static_cast<int64_t>(heads) * kHd) + col0;
    const uint16_t* const bias = a.bias[w.tensor] ? a.bias[w.tensor] + col0 : nullptr;

    // the row's angles, while its first values are on their way
    float2 A[4], B[4];   // out_i = rstd * (x_i A_i + partner_i B_i)
    if (w.tensor < 2) {
      __syncwarp();
      for (int i = 0; i < rounds; ++i) {
        const int j = lane + 32 * i;
        if (j < pairs) {
          const long long p = a.positions[w.row * a.axes + axis[j]];
          const long long t = static_cast<long long>(static_cast<unsigned long long>(p) * turns[j]);
          float s, co;
          sincospif(__fmul_rn(__ll2float_rn(t), 0x1p-63f), &s, &co);
          angles[warp][j] = make_float2(co, s);
        }
      }
      __syncwarp();
      const uint16_t* const weight = a.weight[w.tensor];
      constexpr uint32_t kOnes = 0x3f803f80u;
      uint4 wv = make_uint4(kOnes, kOnes, kOnes, kOnes), wp = wv;
      if (weight != nullptr) {
        wv = load16_reused(weight + c * 8);
        wp = ILV ? wv : load16_reused(weight + (src % LPH) * 8);
      }
      const uint32_t ww[4] = {wv.x, wv.y, wv.z, wv.w}, wq[4] = {wp.x, wp.y, wp.z, wp.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 wi = bf16x2_to_float2(ww[i]), wo = bf16x2_to_float2(wq[i]);
        A[i] = wi;
        B[i] = make_float2(0.0f, 0.0f);
        if (rotated) {
          if constexpr (ILV) {
            const float2 cs = angles[warp][4 * c + i];
            A[i] = make_float2(__fmul_rn(wi.x, cs.x), __fmul_rn(wi.y, cs.x));
            B[i] = make_float2(-__fmul_rn(wi.y, cs.y), __fmul_rn(wi.x, cs.y));
          } else {
            const int j = 8 * (c < half ? c : c - half) + 2 * i;
            const float2 c0 = angles[warp][j], c1 = angles[warp][j + 1];
            const float sign = c < half ? -1.0f : 1.0f;
            A[i] = make_float2(__fmul_rn(wi.x, c0.x), __fmul_rn(wi.y, c1.x));
            B[i] = make_float2(__fmul_rn(wo.x, sign * c0.y), __fmul_rn(wo.y, sign * c1.y));
          }
        }
      }
    }

    for (int g = w.g; g < w.g_end; g += kUnroll) {
      load();
      asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
      uint4 xw[kUnroll];
#pragma unroll
      for (int j = 0; j < kUnroll; ++j) xw[j] = ring[warp][slot][j][lane];
      slot = (slot + 1) % kRing;
#pragma unroll
      for (int j = 0; j < kUnroll; ++j) {
        if (g + j >= w.g_end) break;  // warp-uniform
        const bool mine = (g + j) * kHeadsPerWarp + lane / LPH < heads;
        const int64_t at = static_cast<int64_t>(g + j) * (kHeadsPerWarp * kHd);
        const uint4 b = mine && bias != nullptr ? load16_reused(bias + at)
                                                : make_uint4(kMinusZeros, kMinusZeros, kMinusZeros, kMinusZeros);
        if (w.tensor == 2) {   // (one rounding: the sum of two bf16 values)
          if (mine)
            store16(out + at, make_uint4(add_bf16x2(xw[j].x, b.x), add_bf16x2(xw[j].y, b.y), add_bf16x2(xw[j].z, b.z),
                                         add_bf16x2(xw[j].w, b.w)));
          continue;
        }
        float2 x[4];
        biased(xw[j], b, x);
        float rstd = 1.0f;
        if (a.norm) {
          const float2 s2 = fma2(x[3], x[3], fma2(x[2], x[2], fma2(x[1], x[1], mul2(x[0], x[0]))));
          float ss = __fadd_rn(s2.x, s2.y);
#pragma unroll
          for (int o = LPH / 2; o >= 1; o >>= 1) ss = __fadd_rn(ss, __shfl_xor_sync(0xffffffffu, ss, o));
          rstd = rsqrtf(__fadd_rn(__fmul_rn(ss, 1.0f / kHd), a.eps));
        }
        float2 y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float2 p = make_float2(x[i].y, x[i].x);
          if constexpr (!ILV)
            p = make_float2(__shfl_sync(0xffffffffu, x[i].x, src), __shfl_sync(0xffffffffu, x[i].y, src));
          y[i] = mul2(x[i], A[i]);
          if (rotated) y[i] = fma2(p, B[i], y[i]);
        }
        const float2 r2 = make_float2(rstd, rstd);
        if (mine)
          store16(out + at, make_uint4(float2_to_bf16x2(mul2(y[0], r2)), float2_to_bf16x2(mul2(y[1], r2)),
                                       float2_to_bf16x2(mul2(y[2], r2)), float2_to_bf16x2(mul2(y[3], r2))));
      }
    }
    u += nwarps;
    if (u >= units) break;
    w = unit_of(u);
  }
}

template <int LPH, bool ILV>
cudaError_t launch(AxesArgs& a, cudaStream_t stream) {
  const void* kernel = reinterpret_cast<const void*>(&qkv_axes_kernel<LPH, ILV>);
  int blocks = 0;
  cudaError_t err = persistent_blocks(kernel, kThreads, 0, int64_t{1} << 30, &blocks);
  if (err != cudaSuccess) return err;
  // A unit takes all heads of a row where the rows give every warp some eight units, down to one load's:
  // its angles are made again for every unit of the row, but the warps end together.
  constexpr int kHeadsPerWarp = 32 / LPH;
  int most = 0;
  for (int t = 0; t < 3; ++t) {
    const int groups = (a.heads[t] + kHeadsPerWarp - 1) / kHeadsPerWarp;
    most = groups > most ? groups : most;
  }
  const int64_t warps = static_cast<int64_t>(blocks) * kWarps;
  int64_t parts = 8 * warps / (3 * a.rows);
  const int64_t batches = (most + kUnroll - 1) / kUnroll;
  if (parts > batches) parts = batches;
  if (parts < 1) parts = 1;
  a.unit_groups = static_cast<int>((batches + parts - 1) / parts) * kUnroll;
  int64_t units = 0;
  for (int t = 0; t < 3; ++t) {
    const int groups = (a.heads[t] + kHeadsPerWarp - 1) / kHeadsPerWarp;
    a.units[t] = (groups + a.unit_groups - 1) / a.unit_groups;
    units += a.units[t];
  }
  units *= a.rows;
  const int64_t need = (units + kWarps - 1) / kWarps;
  if (need < blocks) blocks = static_cast<int>(need);
  qkv_axes_kernel<LPH, ILV><<<blocks, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_qkv_axes(const uint16_t* const x[3], const int64_t ld[3], const uint16_t* const bias[3],
                            const uint16_t* const weight[2], uint16_t* const out[3], const int32_t* positions, int axes,
                            const RopeTurns& turns, int rot, int interleaved, int norm, int64_t rows, int heads,
                            int kv_heads, int head_dim, float eps, cudaStream_t stream) {
  AxesArgs a{};
  for (int i = 0; i < 3; ++i) {
    a.x[i] = x[i];
    a.ld[i] = ld[i];
    a.bias[i] = bias[i];
    a.out[i] = out[i];
    a.heads[i] = i == 0 ? heads : kv_heads;
  }
  a.weight[0] = weight[0];
  a.weight[1] = weight[1];
  a.positions = positions;
  a.axes = axes;
  a.rot = rot;
  a.norm = norm;
  a.rows = rows;
  a.eps = eps;
  a.turns = turns;
  switch (head_dim) {
    case 64: return interleaved ? launch<8, true>(a, stream) : launch<8, false>(a, stream);
    case 128: return interleaved ? launch<16, true>(a, stream) : launch<16, false>(a, stream);
    default: return interleaved ? launch<32, true>(a, stream) : launch<32, false>(a, stream);
  }
}

}  // namespace h3q
