// postnorm.cu -- the norm after a block, its gate and scaled residual, the norm before the next
// block with its modulation, and NVFP4.
//
// Per row, with t the row's frame:
//   u  = bf16(fl(o + bias))                (u = o without a bias)
//   n  = fl(fl(u * rstd(u)) * gamma_post), times gate[t] where there is one
//   h' = fl(fl(s * h) + n)                 written back to the fp32 residual h
//   y  = bf16(fl(fl(h' * rstd(h')) * gamma)), or with a modulation table
//        bf16(fl(fl(fl(fl(h' * rstd(h')) * gamma) * fl(1 + scale[t])) + shift[t]))
//   and the NVFP4 quantize of y.
// Both rstd in the canonical order (chunk c on lane c % 128, eight fmaf partials per lane, the
// lane total, a butterfly per warp, (T0+T1)+(T2+T3)).
//
// One CTA of 128 threads owns one row at a time, three CTAs an SM (four up to 4,096 columns): the
// second norm needs all of h', which needs all of u, so a row stays in registers from its load to its
// codes, with two sums over the CTA between.  The other CTAs' rows fill the waits, and a row is asked
// for (a bulk prefetch into L2) when the one before is begun.  Neighbouring rows go to different CTAs, so
// that all of them are in the same frame or two and the tables, 12 bytes a column, are read through L1.
// 65,280 x 7,168 take 827 us, 5.9 TB/s.  (Two CTAs with the tables in shared memory and the next row
// in registers took 909, four with spills 957, no prefetch 841, one two rows ahead 1,000.)
// What is absent is a value of one (gate), zero (scale) or minus zero (bias and shift: x + -0 = x, zeros
// keeping their sign), so a launch has one path.
//
// Bound: 4 + 2 + 4 + 0.5 + 1/16 bytes of DRAM traffic an element, and the latency of a row's chain of two
// sums with 12 warps an SM (168 registers a thread hold a row).
#include "h3q_device.cuh"
#include "h3q_internal.h"

namespace h3q {
namespace {

constexpr int kThreads = 128;  // the lanes of the canonical order

__device__ __forceinline__ int64_t frame_of(const PostnormArgs& a, int64_t row) {
  if (a.gate == nullptr && a.table == nullptr) return 0;
  const int64_t t = a.row_frame ? static_cast<int64_t>(a.row_frame[row]) : row / a.rows_per_frame;
  return t < 0 ? 0 : (t >= a.num_frames ? a.num_frames - 1 : t);  // memory safety only
}

__device__ __forceinline__ void ld_h8(const float* p, float (&v)[8]) {
  asm volatile("ld.global.L1::no_allocate.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]),
                 "=f"(v[6]), "=f"(v[7])
               : "l"(p));
}

__device__ __forceinline__ void st_h8(float* p, const float (&v)[8]) {
  asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(v[0]), "f"(v[1]),
               "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

__device__ __forceinline__ uint4 filled(uint32_t w) { return make_uint4(w, w, w, w); }

// The row's rstd from each thread's eight partials (four pairs).  One barrier; `totals` must not be in use.
__device__ __forceinline__ float row_rstd_of(const float2 (&acc)[4], float* totals, float cols_f, float eps) {
  float tot = __fadd_rn(__fadd_rn(__fadd_rn(acc[0].x, acc[0].y), __fadd_rn(acc[1].x, acc[1].y)),
                        __fadd_rn(__fadd_rn(acc[2].x, acc[2].y), __fadd_rn(acc[3].x, acc[3].y)));
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) tot = __fadd_rn(tot, __shfl_xor_sync(0xffffffffu, tot, off));
  if ((threadIdx.x & 31) == 0) totals[threadIdx.x >> 5] = tot;
  __syncthreads();
  const float ss = __fadd_rn(__fadd_rn(totals[0], totals[1]), __fadd_rn(totals[2], totals[3]));
  return __frcp_rn(__fsqrt_rn(__fadd_rn(__fdiv_rn(ss, cols_f), eps)));
}

// Rows of up to 1,024 * C1 columns (FULL: exactly).
template <int C1, bool FULL>
__global__ void __launch_bounds__(kThreads, C1 > 4 ? 3 : 4) postnorm_kernel(const __grid_constant__ PostnormArgs a) {
  __shared__ float inv_table[128];
  __shared__ float totals[4][4];      // [row parity * 2 + norm]
  const float gsf = *a.gsf;
  fill_inverse_scales(inv_table, gsf);
  __syncthreads();

  const int t = threadIdx.x;
  const int chunks = static_cast<int>(a.cols >> 3);
  const int64_t quads = a.cols >> 6;
  const float cols_f = static_cast<float>(a.cols);  // exact: cols <= 8,192
  constexpr uint32_t kOnes = 0x3f803f80u, kMinusZeros = 0x80008000u;
  const uint16_t* const bias = a.bias ? a.bias + t * 8 : nullptr;
  auto entry = [&](const uint16_t* table, int j, uint32_t absent) {   // eight columns of a table
    return table != nullptr && (FULL || t + j * kThreads < chunks) ? load16_reused(table + j * (kThreads * 8)) : filled(absent);
  };

  int parity = 0;
  int64_t frame = frame_of(a, blockIdx.x);
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x, parity ^= 1) {
    float h[C1][8];
    uint4 o[C1];
    const int64_t next = r + gridDim.x;
    if (next < a.rows && t < 2) {
      const void* from = t == 0 ? static_cast<const void*>(a.o + next * a.ld_o) : static_cast<const void*>(a.h + next * a.ld_h);
      asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(from), "r"(static_cast<uint32_t>(a.cols) * (t == 0 ? 2u : 4u))
                   : "memory");
    }
    const int64_t next_frame = next < a.rows ? frame_of(a, next) : 0;
    float* const hr = a.h + r * a.ld_h + t * 8;
    const uint16_t* const orow = a.o + r * a.ld_o + t * 8;
#pragma unroll
    for (int j = 0; j < C1; ++j)
      o[j] = FULL || t + j * kThreads < chunks ? load16_stream(orow + j * (kThreads * 8)) : filled(0u);
#pragma unroll
    for (int j = 0; j < C1; ++j) {
      if (FULL || t + j * kThreads < chunks) {
        ld_h8(hr + j * (kThreads * 8), h[j]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) h[j][e] = 0.0f;
      }
    }
    const uint16_t* const gate = a.gate ? a.gate + frame * a.cols + t * 8 : nullptr;
    const uint16_t* const shift = a.table ? a.table + frame * 2 * a.cols + t * 8 : nullptr;
    const uint16_t* const scale = a.table ? shift + a.cols : nullptr;
    // u, over o, and its squares (exact in fp32)
    float2 acc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int j = 0; j < C1; ++j) {
      const int c = t + j * kThreads;
      if (FULL || c < chunks) {
        const uint4 b = entry(bias, j, kMinusZeros);
        o[j] = make_uint4(add_bf16x2(o[j].x, b.x), add_bf16x2(o[j].y, b.y), add_bf16x2(o[j].z, b.z),
                          add_bf16x2(o[j].w, b.w));
        const uint32_t w[4] = {o[j].x, o[j].y, o[j].z, o[j].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 v = bf16x2_to_float2(w[i]);
          acc[i] = fma2(v, v, acc[i]);
        }
      }
    }
    const float rstd_u = row_rstd_of(acc, totals[2 * parity], cols_f, a.eps);
    // the residual, written back, and its squares
    const float2 rstd_u2 = make_float2(rstd_u, rstd_u), keep2 = make_float2(a.keep, a.keep);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int j = 0; j < C1; ++j) {
      const int c = t + j * kThreads;
      if (FULL || c < chunks) {
        const uint4 p4 = entry(a.gamma_post + t * 8, j, 0u), g4 = entry(gate, j, kOnes);
        const uint32_t w[4] = {o[j].x, o[j].y, o[j].z, o[j].w}, pw[4] = {p4.x, p4.y, p4.z, p4.w},
                       gw[4] = {g4.x, g4.y, g4.z, g4.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 n = mul2(mul2(mul2(bf16x2_to_float2(w[i]), rstd_u2), bf16x2_to_float2(pw[i])),
                                bf16x2_to_float2(gw[i]));
          const float2 k = mul2(make_float2(h[j][2 * i], h[j][2 * i + 1]), keep2);
          // scalar adds: a paired add of a paired product would be contracted
          h[j][2 * i] = __fadd_rn(k.x, n.x);
          h[j][2 * i + 1] = __fadd_rn(k.y, n.y);
          const float2 v = make_float2(h[j][2 * i], h[j][2 * i + 1]);
          acc[i] = fma2(v, v, acc[i]);
        }
        st_h8(hr + j * (kThreads * 8), h[j]);
      }
    }
    const float rstd = row_rstd_of(acc, totals[2 * parity + 1], cols_f, a.eps);
    if (a.row_rstd != nullptr && t == 0) a.row_rstd[r] = rstd;
    // The norm, the modulation and the quantize: the two threads of a 16-element block (lanes 2k,
    // 2k+1) exchange their half maxima, the even one writes the scale byte.
    const float2 rstd2 = make_float2(rstd, rstd);
    uint8_t* const codes_at = a.codes + r * (a.cols >> 1) + t * 4;
    uint8_t* const scale_at = a.scales + scale_row_offset(r, quads) + (t >> 3) * 512 + ((t >> 1) & 3);
#pragma unroll
    for (int j = 0; j < C1; ++j) {
      const int c = t + j * kThreads;
      const bool valid = FULL || c < chunks;
      const uint4 g4 = entry(a.gamma + t * 8, j, 0u), s4 = entry(scale, j, 0u), t4 = entry(shift, j, kMinusZeros);
      const uint32_t gw[4] = {g4.x, g4.y, g4.z, g4.w}, sw[4] = {s4.x, s4.y, s4.z, s4.w},
                     tw[4] = {t4.x, t4.y, t4.z, t4.w};
      uint32_t y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 m = mul2(mul2(mul2(make_float2(h[j][2 * i], h[j][2 * i + 1]), rstd2), bf16x2_to_float2(gw[i])),
                              add_bf16x2_f32(sw[i], make_float2(1.0f, 1.0f)));
        y[i] = float2_to_bf16x2(add_bf16x2_f32(tw[i], m));
      }
      float amax = halves_amax(absmax_bf16x2(absmax_bf16x2(y[0], y[1]), absmax_bf16x2(y[2], y[3])));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      const uint32_t sf = block_scale(amax, gsf);
      const uint32_t codes = codes8(y, inv_table[sf]);
      if (valid) store_word(codes_at + j * (kThreads * 4), codes);
      if (valid && !(t & 1)) store_byte(scale_at + j * (kThreads / 8 * 512), sf);
    }
    frame = next_frame;
  }

  // zero the scale words of the padding rows rows..pad128(rows)-1
  const int64_t prows = (a.rows + 127) >> 7 << 7;
  for (int64_t p = a.rows + blockIdx.x; p < prows; p += gridDim.x)
    for (int64_t q = t; q < quads; q += kThreads)
      store_word(a.scales + scale_word_offset(p, q, quads), 0u);
}

template <int C1>
cudaError_t launch_c1(const PostnormArgs& a, cudaStream_t stream) {
  const bool full = a.cols == int64_t(1024) * C1;
  const void* kernel = full ? reinterpret_cast<const void*>(&postnorm_kernel<C1, true>)
                            : reinterpret_cast<const void*>(&postnorm_kernel<C1, false>);
  int blocks = 0;
  cudaError_t err = persistent_blocks(kernel, kThreads, 0, a.rows, &blocks);
  if (err != cudaSuccess) return err;
  if (full)
    postnorm_kernel<C1, true><<<blocks, kThreads, 0, stream>>>(a);
  else
    postnorm_kernel<C1, false><<<blocks, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_postnorm(const PostnormArgs& a, cudaStream_t stream) {
  const int64_t per_lane = (a.cols / 8 + kThreads - 1) / kThreads;
  if (per_lane <= 1) return launch_c1<1>(a, stream);
  if (per_lane <= 2) return launch_c1<2>(a, stream);
  if (per_lane <= 4) return launch_c1<4>(a, stream);
  if (per_lane <= 7) return launch_c1<7>(a, stream);
  if (per_lane <= 8) return launch_c1<8>(a, stream);
  return cudaErrorInvalidValue;  // the API refuses rows wider than 8,192 first
}

}  // namespace h3q
