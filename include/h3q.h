/*
 * h3q.h -- C ABI of the fused NVFP4 activation producers (GB300, sm_103a).
 *
 * Producers that turn bf16 activations into NVFP4 GEMM inputs with the
 * quantize fused into the kernel that produces them: RMSNorm + AdaLN, SwiGLU
 * and the standalone (attention-output) quantize; the residual fold before the
 * norm and the SwiGLU of a packed projection with its bias; abs-max passes for
 * dynamic and calibrated global scales.  Beside them, the QKV epilogue (bias,
 * per-head RMSNorm and rotate-half RoPE, bf16 outputs), a dequantize used
 * for checking, and what takes the epilogue's outputs on to the next projection:
 * a paged key/value cache that holds its rows in NVFP4 (write, read), attention of
 * packed sequences over bf16 keys and values, and attention of a few new tokens a
 * sequence over that cache; the epilogue with rotary positions of several axes, the norms on
 * both sides of a block with its gate and residual, and sparse attention over blocks of keys that a
 * cheap score selects.  Every NVFP4 producer writes:
 *
 *   codes   uint8 [rows, cols/2]: E2M1 codes, two per byte, the even column in
 *           the low nibble (FastVideo compare "fasth3-spark-exact-perf",
 *           minimax_h3_swiglu_quant.cuh, fp4_pair).  Row pitch cols/2 bytes.
 *   scales  uint8 [h3q_padded_rows(rows), cols/16]: one E4M3 block scale per
 *           16 elements, in the 128x4 swizzled layout; the byte of (row r,
 *           scale column g) is at
 *             ((r/128)*(cols/64) + g/4)*512 + (r%32)*16 + ((r/32)%4)*4 + g%4.
 *           Padding rows rows..h3q_padded_rows(rows)-1 are written as zero.
 *           (FastVideo API page fastvideo.models.vaes.minimax_h3_nvfp4_fused:
 *           introduction -- "E4M3 block scales, layout_128x4 swizzle, zeroed
 *           padding rows" -- and new_quantized; the index is written out in
 *           quant_probe of the FastVideo compare page.)
 *
 * Block quantize (16 consecutive elements y of one row, global scale gsf):
 *   sf = E4M3_rn_satfinite(fl(gsf * fl(amax/6))), dec = fl(E4M3value(sf)/gsf),
 *   inv = dec != 0 ? fl(1/dec) : 0, code_i = E2M1_rn_satfinite(fl(y_i * inv)).
 * This is quant_probe of the FastVideo compare page with every approximate
 * reciprocal replaced by a correctly rounded division.
 *
 * Common conventions
 * ------------------
 * Memory    All pointers are DEVICE pointers into memory owned by the caller
 *           (the host-buffer call also takes host pointers).  No call allocates
 *           device or host memory, frees, or keeps a caller's pointer after it
 *           returns.  Buffers must stay alive until the work queued on `stream`
 *           has finished.  The one thing the library creates is the pair of
 *           streams and 11 events of h3q_rmsnorm_adaln_nvfp4_host, once per CUDA
 *           context on that call's first use in it, kept until the process ends
 *           (see there).
 * Stream    `stream` is a cudaStream_t passed as void* (NULL = the legacy
 *           default stream).  Every call is asynchronous: it validates its
 *           arguments on the host, launches its kernel on `stream` (the
 *           dynamic-scale quantize launches three, in order) and returns.
 *           No call synchronises.  The device is the calling thread's current
 *           CUDA device.
 * Global    `global_scale` points to one fp32 on the device: the static
 *   scale   per-tensor scale gsf (finite, > 0; not checked, reading it would
 *           need a synchronisation).  It is read by the kernel, so it may be
 *           updated on the stream between calls and captured in a graph.
 * Shapes    rows >= 0 (rows == 0 is a successful no-op); cols > 0, a multiple
 *           of 64 (four scale columns form one swizzle atom), at most 2^24.
 *           ld_* is the row stride of an input in ELEMENTS: >= cols and a
 *           multiple of 16.  Indexing is 64-bit throughout: inputs larger
 *           than 2^31 elements are supported (FastVideo commit log, branch
 *           vae-parallel-decode, the int64 program-id fix).
 * Alignment bf16 inputs and fp32 outputs: 32-byte aligned.  codes, scales and
 *           the QKV epilogue's bf16 outputs: 16-byte aligned.  row_frame,
 *           global_scale, amax, row_rstd: 4-byte.
 * Aliasing  Outputs must not overlap inputs or each other.
 * Errors    H3Q_OK (0) on success.  H3Q_ERR_INVALID_ARGUMENT (1): an argument
 *           broke a rule above; nothing was launched and no output was
 *           touched.  H3Q_ERR_CUDA (2): the CUDA runtime reported an error
 *           (no device, launch failure, or a sticky error from earlier work).
 *           h3q_last_error() returns a message for the calling thread's most
 *           recent failure.  No call aborts, traps or prints.
 * Threads   The calls keep two kinds of state between calls, both per CUDA
 *           context (keyed on the context's unique id, so a context destroyed
 *           and re-created, e.g. by cudaDeviceReset, starts afresh): a cache of
 *           launch sizes (occupancy, and the raised shared-memory limit of the
 *           kernels that need one), and the host-buffer call's streams and
 *           events.  They are safe to call from several threads.  The one
 *           exception is h3q_quantize_nvfp4_dynamic, whose abs-max partials live
 *           in a device array inside the library: calls of it that overlap on
 *           one device race (see there).
 */
#ifndef H3Q_H
#define H3Q_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define H3Q_OK 0
#define H3Q_ERR_INVALID_ARGUMENT 1
#define H3Q_ERR_CUDA 2

#define H3Q_ABI_VERSION 4

/* Rows of the scale matrix: rows rounded up to a multiple of 128. */
static inline int64_t h3q_padded_rows(int64_t rows) { return (rows + 127) / 128 * 128; }
/* Bytes of the swizzled scale matrix. */
static inline int64_t h3q_scale_bytes(int64_t rows, int64_t cols)
{
    return h3q_padded_rows(rows) * (cols / 16);
}
/* n rounded up to a multiple of 256 bytes. */
static inline int64_t h3q_align256(int64_t n) { return (n + 255) / 256 * 256; }
/* Device workspace of h3q_rmsnorm_adaln_nvfp4_host: three staging slots of
 * chunk_rows rows, each an x chunk, a code chunk and a scale chunk (each part
 * rounded up to 256 bytes, in that order), then -- when the frames come from
 * rows_per_frame (with_frames != 0) -- the rows' frame indices, rows int32. */
static inline int64_t h3q_host_workspace_bytes(int64_t chunk_rows, int64_t cols, int64_t rows,
                                               int with_frames)
{
    int64_t slot = h3q_align256(chunk_rows * cols * 2) + h3q_align256(chunk_rows * cols / 2) +
                   h3q_align256(chunk_rows * cols / 16);
    return 3 * slot + (with_frames ? h3q_align256(rows * 4) : 0);
}
/* Bytes of the packed code matrix. */
static inline int64_t h3q_code_bytes(int64_t rows, int64_t cols) { return rows * (cols / 2); }
/* Byte offset, in the scale matrix, of the scales of row `row0` onwards when
 * row0 is a multiple of 128: the 512-byte atoms are laid out row-tile major, so
 * the scales of rows [row0, row0 + n) with n a multiple of 128 (or the tensor's
 * last rows) form one contiguous range starting here.  A call on those rows
 * writes exactly that range, which lets a large tensor be processed in
 * 128-row-aligned pieces. */
static inline int64_t h3q_scale_offset_of_row_tile(int64_t row0, int64_t cols)
{
    return row0 / 128 * (cols / 64) * 512;
}

/*
 * Standalone NVFP4 quantize, e.g. of the attention output viewed as
 * [tokens, heads*head_dim].  (TensorRT-LLM PR #21483 "Fuse the MiniMax-H3
 * NVFP4 activation quantize into the AdaLN, SwiGLU and attention-output
 * producers", commit "...quantize it with a bandwidth-bound kernel";
 * FastVideo API page, quantize.)
 *
 *   x             bf16 [rows, cols], row stride ld_x elements.
 *   global_scale  device fp32 gsf.
 *   codes         out, rows*cols/2 bytes.    scales  out, h3q_scale_bytes.
 */
int h3q_quantize_nvfp4(const void *x, int64_t ld_x, int64_t rows, int64_t cols,
                       const float *global_scale, uint8_t *codes, uint8_t *scales,
                       void *stream);

/*
 * RMSNorm with fp32 statistics, AdaLN modulation, NVFP4.  (TensorRT-LLM
 * PR #21483, summary and commit "...SwiGLU producers": the AdaLN RMSNorm +
 * modulation kernel emits packed E2M1 codes and swizzled E4M3 scales
 * directly; FastVideo API page, introduction: fp32 statistics, sequential
 * FMA per thread, no contraction of products that eager rounds.)
 *
 * Per row r with frame t:
 *   ss   = sum of x^2 in the canonical order: 8-element chunk c goes to lane
 *          c % 128; each lane keeps 8 fp32 partials, element e of its chunks
 *          (chunks in increasing order) is fused-multiply-added into partial e;
 *          lane total ((p0+p1)+(p2+p3))+((p4+p5)+(p6+p7)); within each group of
 *          32 lanes a butterfly over xor-distances 16,8,4,2,1 gives the group
 *          total T_w; ss = (T_0+T_1)+(T_2+T_3).
 *   rstd = fl(1 / fl(sqrt(fl(fl(ss / cols) + eps))))
 *   y    = bf16(fl(fl(fl(fl(x * rstd) * gamma) * fl(1 + scale[t])) + shift[t]))
 * then y is block-quantized.
 *
 *   x               bf16 [rows, cols], row stride ld_x elements.
 *   gamma           bf16 [cols].
 *   mod_table       bf16 [num_frames, 2, cols], contiguous: [t][0] is the shift,
 *                   [t][1] the scale.
 *   row_frame       int32 [rows] frame of each row, or NULL.  Entries must lie in
 *                   [0, num_frames) (the index contract of the FastVideo commit
 *                   log's modulation wrappers).  They are not checked on the
 *                   host (that would need a synchronisation); the kernel clamps
 *                   them into range so memory stays safe, and the output of a
 *                   row with an out-of-range entry is unspecified.
 *   rows_per_frame  used when row_frame is NULL: frame = row / rows_per_frame;
 *                   must be >= 1 with (rows-1)/rows_per_frame < num_frames.
 *   eps             finite, >= 0.  With eps = 0 a row whose sum of squares is 0 has
 *                   rstd = 1/0 = +inf and NaN values (0 * inf); its codes and scales
 *                   are then unspecified, like those of NaN or infinite inputs.
 *   row_rstd        optional out fp32 [rows]: rstd of each row, or NULL.
 */
int h3q_rmsnorm_adaln_nvfp4(const void *x, int64_t ld_x, const void *gamma,
                            const void *mod_table, int64_t num_frames, const int32_t *row_frame,
                            int64_t rows_per_frame, float eps, int64_t rows, int64_t cols,
                            const float *global_scale, uint8_t *codes, uint8_t *scales,
                            float *row_rstd, void *stream);

/*
 * SwiGLU producer: y = bf16(fl(fl(g * sigma) * u)) with
 * sigma = fl(1 / fl(1 + exp_c(-g))), then NVFP4.  (FastVideo compare page,
 * minimax_h3_swiglu_quant.cuh, swiglu_bf16: value * silu(gate) rounded to
 * bf16; TensorRT-LLM PR #21483, SiLU-and-mul producer.)  exp_c is a fixed
 * sequence of binary32 operations: Cody-Waite reduction by a two-part ln 2
 * applied with FMAs and a degree-7 Taylor polynomial in Horner form.
 *
 *   gate, up  bf16 [rows, cols], row strides ld_gate, ld_up elements (a
 *             gate/up pair packed in one [rows, 2*cols] projection is two views
 *             with ld = 2*cols).
 */
int h3q_swiglu_nvfp4(const void *gate, int64_t ld_gate, const void *up, int64_t ld_up,
                     int64_t rows, int64_t cols, const float *global_scale, uint8_t *codes,
                     uint8_t *scales, void *stream);

/*
 * SwiGLU of a value-first packed projection with its bias (FastVideo API page,
 * swiglu_quantize: o [M, 2F], value first, gate second, bias not yet added).
 * Each half gets its bias in binary32 and is rounded to bf16,
 *   v = bf16(fl(o[:, j] + bias[j])),  g = bf16(fl(o[:, F + j] + bias[F + j])),
 * then as h3q_swiglu_nvfp4: y = bf16(fl(fl(g * sigma(g)) * v)), quantized.
 *
 *   o       bf16 [rows, 2F], row stride ld_o (>= 2F, a multiple of 16), 32-byte aligned.
 *   bias    bf16 [2F] (value biases, then gate biases), 32-byte aligned, or NULL.
 *   f       F, a multiple of 64; codes [rows, F/2] and scales [pad128(rows), F/16].
 */
int h3q_swiglu_packed_nvfp4(const void *o, int64_t ld_o, const void *bias, int64_t rows,
                            int64_t f, const float *global_scale, uint8_t *codes, uint8_t *scales,
                            void *stream);

/*
 * Dequantize (checking path): out[r][j] = fl((E2M1value(c) * E4M3value(sf)) / gsf),
 * the value a block-scaled NVFP4 GEMM with alpha = 1/gsf sees for the element.
 * No page defines it; it is the inverse the producers' consumers apply.
 *
 *   codes, scales  as written by the producers (scales in the swizzled layout).
 *   out            fp32 [rows, cols], contiguous.
 */
int h3q_dequantize_nvfp4(const uint8_t *codes, const uint8_t *scales, int64_t rows, int64_t cols,
                         const float *global_scale, float *out, void *stream);

/*
 * Residual fold + RMSNorm + AdaLN -> NVFP4 (the residual add folded into the
 * next norm).  TensorRT-LLM PR #21483, commit "...norm1 ... from a second
 * table": a block folds its MLP residual into the next block's norm1 kernel,
 * reading the gate from its own AdaLN table while the scale and shift come from
 * the next block's.  FastVideo API page, residual_norm_quantize: in place
 * h += bf16(o + bias) * scale on a contiguous fp32 residual, then NVFP4 of the
 * normed h.  Per row r with frame t:
 *   u   = bf16(fl(o + bias))           (u = o when bias is NULL)
 *   h'  = fl(h + fl(u * gate[t]))      written back to h
 *   then h3q_rmsnorm_adaln_nvfp4's arithmetic on the fp32 values h' (same
 *   canonical reduction order, squares of fp32 values) and the NVFP4 quantize.
 *
 *   h           fp32 [rows, cols], row stride ld_h (>= cols, a multiple of 8),
 *               32-byte aligned; read and overwritten with h'.
 *   o           bf16 [rows, cols], row stride ld_o, as x of the other producers.
 *   bias        bf16 [cols] or NULL.
 *   gate_table  bf16 [num_frames, cols]: the gate of each frame (this block's).
 *   gamma, mod_table, num_frames, row_frame, rows_per_frame, eps, global_scale,
 *   codes, scales, row_rstd: as h3q_rmsnorm_adaln_nvfp4 (the next block's
 *               modulation table; the frame of a row indexes both tables).
 * Limits: cols <= 8,192.  h, codes, scales and row_rstd must not overlap an
 * input or each other.  Status codes as the other producers.
 */
int h3q_residual_rmsnorm_adaln_nvfp4(float *h, int64_t ld_h, const void *o, int64_t ld_o,
                                     const void *bias, const void *gate_table, const void *gamma,
                                     const void *mod_table, int64_t num_frames,
                                     const int32_t *row_frame, int64_t rows_per_frame, float eps,
                                     int64_t rows, int64_t cols, const float *global_scale,
                                     uint8_t *codes, uint8_t *scales, float *row_rstd,
                                     void *stream);

/*
 * Dynamic and calibrated global scales.
 *
 * FastVideo API page, NVFP4DecoderLinear: a dynamic layer scales each call by
 * the abs-max of its input, and a calibrating layer folds each call's abs-max
 * into a persistent running maximum (input_amax).  FlashRT PR #142, commit
 * "...amax pipeline": the abs-max is taken on the device in a pass of its own
 * and read by the quantize pass with no host synchronisation.
 *
 * The three abs-max passes compute the producer's bf16 output y exactly as the
 * producer does (same arguments, same arithmetic) without storing it, and fold
 * max |y| into *amax: *amax = max(*amax, max |y|).  Zero *amax first for a
 * per-call abs-max; keep it across calls for a running maximum.
 *
 *   amax  device fp32 scalar, 4-byte aligned, holding a value >= 0 (+0.0, not
 *         -0.0) on entry; updated with an atomic maximum, so several passes
 *         may fold into it, on one stream or several.
 *
 * Then h3q_global_scale_from_amax writes *global_scale = fl(2688 / *amax) on the
 * device (2688 = 448 * 6), with two readings where that has no finite positive
 * value: amax = 0 gives 1, and +inf (a producer output that overflowed bf16) is
 * clamped to the largest finite binary32 first.  The producer then reads it.
 * Nothing synchronises; the calls are ordered by the stream.
 *
 * Preconditions and status codes are those of the matching producer (shapes,
 * alignment, ld, frames), plus: amax not NULL and not overlapping an input.
 *
 * h3q_rmsnorm_adaln_amax also writes each row's rstd to row_rstd when it is not
 * NULL (fp32 [rows], 4-byte aligned, overlapping neither an input nor amax): the
 * pass forms the row statistics anyway, in the producer's canonical order, so
 * h3q_rmsnorm_adaln_nvfp4_from_rstd can then quantize without forming them again.
 */
int h3q_amax_bf16(const void *x, int64_t ld_x, int64_t rows, int64_t cols, float *amax,
                  void *stream);

int h3q_rmsnorm_adaln_amax(const void *x, int64_t ld_x, const void *gamma,
                           const void *mod_table, int64_t num_frames, const int32_t *row_frame,
                           int64_t rows_per_frame, float eps, int64_t rows, int64_t cols,
                           float *amax, float *row_rstd, void *stream);

/*
 * The RMSNorm + AdaLN producer with each row's rstd given: the second pass of a
 * dynamic scale, after h3q_rmsnorm_adaln_amax wrote row_rstd.  y and its NVFP4 are
 * those of h3q_rmsnorm_adaln_nvfp4 with rstd = row_rstd[r] in place of the row's
 * own statistics (so, with the abs-max pass's row_rstd, byte for byte the same
 * output); eps has no role.  Arguments as h3q_rmsnorm_adaln_nvfp4, plus:
 *
 *   row_rstd  fp32 [rows] on the device, 4-byte aligned, not NULL, overlapping no
 *             output.
 */
int h3q_rmsnorm_adaln_nvfp4_from_rstd(const void *x, int64_t ld_x, const void *gamma,
                                      const void *mod_table, int64_t num_frames,
                                      const int32_t *row_frame, int64_t rows_per_frame,
                                      const float *row_rstd, int64_t rows, int64_t cols,
                                      const float *global_scale, uint8_t *codes, uint8_t *scales,
                                      void *stream);

int h3q_swiglu_amax(const void *gate, int64_t ld_gate, const void *up, int64_t ld_up,
                    int64_t rows, int64_t cols, float *amax, void *stream);

int h3q_global_scale_from_amax(const float *amax, float *global_scale, void *stream);

/*
 * Dynamic quantize that needs no scratch from the caller and allocates nothing.
 * No page has a counterpart: it is this library's convenience form of the
 * dynamic scale above for the standalone quantize.  On the stream it runs an
 * abs-max pass over x whose CTAs write their partial maxima into a fixed
 * device array inside the library (a file-scope __device__ array of 4,096
 * floats, one per CUDA context, its address looked up in the current context
 * on every call: a lookup, not an allocation); then the quantize, launched as a
 * programmatic dependent of that pass, reduces them into the global scale
 * fl(2688 / max |x|) (0 -> 1, +inf clamped) in each of its CTAs and quantizes x
 * as h3q_quantize_nvfp4 does with that scale.  Outputs: codes, scales and the
 * global scale used (a device fp32 scalar written here).
 *
 * Limit: a shape whose abs-max pass needs more than 4,096 partial maxima (CTAs)
 * is rejected with H3Q_ERR_INVALID_ARGUMENT; on one GPU the pass launches at
 * most its occupancy times the SM count (1,216 CTAs on a 152-SM GB300).
 * Calls that overlap on one device (different streams, or threads without
 * ordering between them) share the array and race; order them on one stream.
 * Other preconditions and status codes as h3q_quantize_nvfp4.
 */
int h3q_quantize_nvfp4_dynamic(const void *x, int64_t ld_x, int64_t rows, int64_t cols,
                               float *global_scale, uint8_t *codes, uint8_t *scales,
                               void *stream);

/*
 * QKV epilogue: bias + per-head RMSNorm + partial rotate-half RoPE on q and k,
 * bias only on v (the step after the QKV projection GEMM; bf16 out, no
 * quantize).  FastVideo API page, qkv_epilogue: projected q/k/v [M, H*HD] bf16
 * with the bias not yet added -> roped q, k and biased v, each [M, H, HD];
 * cos/sin bf16 [M, ROT] (the eager path's cos.to(query.dtype)); an eps and no
 * norm weights.  FastVideo commit log (the q/k norm + partial RoPE kernel):
 * offsets are 64-bit, so M * H * HD may exceed 2^31.  Per row and head, with
 * x' = bf16(fl(x + b)) for each of the HD values:
 *   v:     out = x'
 *   q, k:  ss = the head's sum of squares of x' (eight fmaf partials per chunk
 *          of 8 values, the chunk total ((p0+p1)+(p2+p3))+((p4+p5)+(p6+p7)),
 *          a butterfly over the head's HD/8 chunk totals);
 *          rstd = fl(1 / fl(sqrt(fl(fl(ss / HD) + eps)))), n = bf16(fl(x' * rstd));
 *          out_i = bf16(fl(bf16(fl(n_i * cos_i)) + bf16(fl(r_i * sin_i)))) for
 *          i < ROT, r_i = -n_{i+ROT/2} (i < ROT/2) or n_{i-ROT/2} (rotate-half
 *          pairs), or with `interleaved` r_{2j} = -n_{2j+1}, r_{2j+1} = n_{2j}
 *          (FlashRT PR #142 page, the fused RMSNorm + RoPE kernel: interleaved
 *          RoPE on the [B, S, H, D] layout); out_i = n_i for i >= ROT.
 *
 *   q, k, v        bf16 [rows, heads * head_dim], row strides ld_q, ld_k, ld_v
 *                  (>= heads * head_dim, multiples of 16), 32-byte aligned.
 *   bias_q/k/v     bf16 [heads * head_dim], 32-byte aligned, not NULL.
 *   cos, sin       bf16 [rows, rot] contiguous, 16-byte aligned; NULL when rot = 0.
 *   rot            ROT, a multiple of 16 with 0 <= rot <= head_dim.
 *   interleaved    0: rotate-half pairs (i, i + ROT/2); 1: pairs (2j, 2j + 1).
 *   heads          H >= 1; head_dim HD in {64, 128, 256}; heads * head_dim <= 2^24.
 *   eps            finite, >= 0 (with eps = 0 an all-zero head gives NaN values, whose
 *                  bit patterns are unspecified).
 *   q_out, k_out, v_out  bf16 [rows, heads, head_dim] contiguous, 16-byte
 *                  aligned, caller-owned; they must not overlap an input or
 *                  each other.
 * rows = 0 returns H3Q_OK with no launch.  Status codes as the other calls.
 */
int h3q_qkv_epilogue(const void *q, int64_t ld_q, const void *k, int64_t ld_k, const void *v,
                     int64_t ld_v, const void *bias_q, const void *bias_k, const void *bias_v,
                     const void *cos, const void *sin, int64_t rot, int interleaved, int64_t rows,
                     int64_t heads, int64_t head_dim, float eps, void *q_out, void *k_out,
                     void *v_out, void *stream);

/*
 * The FFN-up projection as a block-scaled NVFP4 GEMM on the tensor cores, with
 * the SwiGLU and the NVFP4 quantize of its output in the epilogue.  (FastVideo
 * compare "fasth3-spark-exact-perf", minimax_h3_swiglu_gemm.cu:
 * launch_gemm_swiglu -- NVFP4 A and B, value/gate-paired weight columns, alpha
 * and the global scale as device pointers -- and h3_epilogue::Store -- value =
 * bf16(alpha * acc), gate = bf16(alpha * acc), SwiGLU, block quantize.)
 *
 *   acc[i][j] = sum over k of A[i][k] * B[j][k]        (fp32, tensor-core order)
 *   u = bf16(fl(alpha * acc[i][2j])),  g = bf16(fl(alpha * acc[i][2j + 1]))
 *   y[i][j] = bf16(fl(fl(g * sigma(g)) * u))           (as h3q_swiglu_nvfp4)
 * then y [m, n/2] is block-quantized with global_scale.  A element =
 * E2M1value(code) * E4M3value(scale); the products are exact and the sum is
 * accumulated in binary32 by the tensor cores in their own order (it
 * approximates the exact sum; everything after acc is bit-exact arithmetic).
 *
 *   a_codes   uint8 [m, k/2] contiguous: the activation's E2M1 codes (as the
 *             producers write them).  16-byte aligned.
 *   a_scales  uint8 [h3q_padded_rows(m), k/16] in the 128x4 layout (as the
 *             producers write them).  16-byte aligned.
 *   b_codes   uint8 [n, k/2] contiguous, b_scales uint8 [n, k/16] in the 128x4
 *             layout: the weight, row 2j the value and row 2j+1 the gate of
 *             output j.  16-byte aligned.
 *   m         rows of A, 0 <= m <= 2^31 - 128 (m = 0 is a no-op).
 *   k         a multiple of 256, at most 2^24.   n  a multiple of 256, at most 2^24.
 *   alpha     device fp32: the dequantization factor of the product (for
 *             operands quantized with global scales g_A and g_B,
 *             fl(1 / fl(g_A * g_B))).
 *   global_scale  device fp32 gsf of the output quantize.
 *   codes     out, [m, n/4].   scales  out, h3q_scale_bytes(m, n/2).
 *   y         optional out, bf16 [m, n/2] (NULL: not written).
 *   acc       optional out, fp32 [m, n]: the accumulator before alpha (NULL:
 *             not written; for checking).
 * Alignment: codes, scales, y and acc 16-byte aligned.  Outputs must not
 * overlap an input or each other.  Status codes as the other calls.  The
 * kernel keeps one CTA per SM with all 512 TMEM columns of it; its waits are
 * bounded (2 s): if one runs out the kernel stops early, the outputs are
 * unspecified, and h3q_kernel_error_flag reports it.
 */
int h3q_gemm_swiglu_nvfp4(const uint8_t *a_codes, const uint8_t *a_scales, int64_t m, int64_t k,
                          const uint8_t *b_codes, const uint8_t *b_scales, int64_t n,
                          const float *alpha, const float *global_scale, uint8_t *codes,
                          uint8_t *scales, void *y, float *acc, void *stream);

/*
 * *flag = 1 if a kernel launched on the current device since the last call had one of
 * its bounded waits run out, else 0; the flag is cleared.  The kernels that wait on
 * mbarriers between their warps (the GEMM of h3q_gemm_swiglu_nvfp4, and those of
 * h3q_attention_varlen, h3q_attention_cache_nvfp4 and h3q_attention_blocks) bound every wait
 * (2 s) and then stop early, leaving that call's outputs unspecified.  Synchronous: it waits
 * for the device, all streams.  Not on any page; a diagnostic of this library.
 */
int h3q_kernel_error_flag(int *flag);

/*
 * h3q_rmsnorm_adaln_nvfp4 on HOST buffers: x read from host memory, codes and
 * scales written to host memory, the copies inside the call.  The rows are cut
 * into chunks of chunk_rows rows (a multiple of 128); the producer runs on the
 * caller's stream on chunk i while a library stream copies chunk i+1 in and
 * another copies chunk i-1's codes and scales out (the scales of a 128-row tile
 * are one contiguous range, h3q_scale_offset_of_row_tile).  The outputs equal
 * h3q_rmsnorm_adaln_nvfp4's byte for byte.
 *
 *   x_host          bf16 [rows, cols], contiguous, in host memory (page-locked
 *                   for the copies to run asynchronously and overlap).
 *   codes_host      out, host uint8 [rows, cols/2], contiguous.
 *   scales_host     out, host uint8 [h3q_padded_rows(rows), cols/16], contiguous.
 *   gamma, mod_table, num_frames, row_frame, rows_per_frame, eps, global_scale:
 *                   as h3q_rmsnorm_adaln_nvfp4, in device memory (row_frame
 *                   int32 [rows] or NULL).
 *   workspace       device memory of at least h3q_host_workspace_bytes(chunk_rows,
 *                   cols, rows, row_frame == NULL) bytes, 256-byte aligned, owned
 *                   by the caller and not touched by other work until the stream
 *                   has passed this call.
 *   chunk_rows      a positive multiple of 128.
 * Ordering: the call runs after the work queued on `stream` before it, and work
 * queued on `stream` after it starts after its last copy back, so the host
 * outputs may be read once `stream` has been synchronised.  On its first call on
 * a device the library creates two non-blocking streams and a few events for
 * that device and keeps them; it allocates no memory.  Calls on one device are
 * enqueued one at a time (a lock), and stay asynchronous.  Status codes as the
 * other calls; a failure after the first copy was queued leaves the outputs
 * unspecified.  The streams and events belong to the CUDA context current at the
 * call (2 streams, 11 events per context, never destroyed: a context that the
 * caller destroys takes them with it).  At most 64 contexts over the process's
 * life can use this call; the 65th gets H3Q_ERR_CUDA (cudaErrorNotSupported).
 */
int h3q_rmsnorm_adaln_nvfp4_host(const void *x_host, int64_t rows, int64_t cols, const void *gamma,
                                 const void *mod_table, int64_t num_frames, const int32_t *row_frame,
                                 int64_t rows_per_frame, float eps, const float *global_scale,
                                 uint8_t *codes_host, uint8_t *scales_host, void *workspace,
                                 int64_t workspace_bytes, int64_t chunk_rows, void *stream);

/*
 * The paged NVFP4 key/value cache, what stands between the QKV epilogue and the
 * attention of the tokens to come: keys and values quantized as they are written, in
 * the block format of the producers (16 elements of one head share a scale).
 *
 *   codes   k_codes, v_codes  uint8 [num_pages, kv_heads, page_size, head_dim/2]: two
 *           E2M1 codes a byte, the even element in the low nibble.  16-byte aligned.
 *   scales  k_scales, v_scales  uint8 [num_pages, kv_heads, page_size, head_dim/16]:
 *           one E4M3 scale per 16 elements, in order (not swizzled).  16-byte aligned.
 *           Its low seven bits are read; all of them set (what a NaN leaves in the cache)
 *           count as 480, in reading rows back as in attention.
 *   k_global_scale, v_global_scale  device fp32, finite and > 0 (not checked): the
 *           static per-tensor scales, one for keys and one for values.
 *   num_pages  1 .. 2^31 - 1.    page_size  16, 32, 64 or 128.
 *   kv_heads   >= 1.             head_dim   64, 128 or 256; kv_heads * head_dim <= 2^24.
 *
 * The rows of several sequences come packed, and lists on the device say where they
 * live (read by the kernels, so they may change between the replays of a graph):
 *
 *   cu_rows      int32 [batch + 1], not decreasing: rows cu_rows[b] .. cu_rows[b+1]-1
 *                belong to sequence b.  Rows before cu_rows[0] or from cu_rows[batch]
 *                on belong to none.
 *   kv_len       int32 [batch]: the positions of sequence b in the cache, its packed
 *                rows included: n = cu_rows[b+1] - cu_rows[b] rows stand at its LAST n
 *                positions, kv_len[b] - n .. kv_len[b] - 1.
 *   block_table  int32 [batch, max_pages]: position p of sequence b is row
 *                p % page_size of page block_table[b][p / page_size].
 * batch 0 .. 2^24, max_pages >= 1; batch * max_pages <= 2^40.  Lists are 4-byte aligned.
 * Their entries are not checked on the host (that would need a synchronisation); no
 * entry makes a kernel touch memory outside the buffers.
 */

/*
 * Quantize new rows into the cache: k, v bf16 [rows, kv_heads * head_dim] (row strides
 * ld_k, ld_v; 32-byte aligned), each block of 16 as h3q_quantize_nvfp4 does.  Nothing
 * is written for a row of no sequence, for one whose position is negative or past the
 * block table, or whose page is not in [0, num_pages); every other byte of the cache
 * stays as it was.  Two rows that reach the same place in the cache (a page listed
 * twice) leave unspecified codes and scales there.
 */
int h3q_kv_cache_write_nvfp4(const void *k, int64_t ld_k, const void *v, int64_t ld_v, int64_t rows,
                             const int32_t *cu_rows, const int32_t *kv_len, const int32_t *block_table,
                             int64_t batch, int64_t max_pages, const float *k_global_scale,
                             const float *v_global_scale, uint8_t *k_codes, uint8_t *k_scales,
                             uint8_t *v_codes, uint8_t *v_scales, int64_t num_pages, int64_t page_size,
                             int64_t kv_heads, int64_t head_dim, void *stream);

/*
 * Read rows of the cache back: bf16(fl((E2M1value(c) * E4M3value(sf)) / gsf)) of the
 * same places that h3q_kv_cache_write_nvfp4 writes with these lists (a sequence's
 * whole prefix: n = kv_len[b]), packed.
 *
 *   k_out, v_out  bf16 [rows, kv_heads, head_dim] contiguous, 32-byte aligned.  Rows
 *                 that the cache does not hold (see above) are written as zero; rows of
 *                 no sequence stay as they were.
 */
int h3q_kv_cache_read_nvfp4(const uint8_t *k_codes, const uint8_t *k_scales, const uint8_t *v_codes,
                            const uint8_t *v_scales, int64_t num_pages, int64_t page_size,
                            int64_t kv_heads, int64_t head_dim, const float *k_global_scale,
                            const float *v_global_scale, int64_t rows, const int32_t *cu_rows,
                            const int32_t *kv_len, const int32_t *block_table, int64_t batch,
                            int64_t max_pages, void *k_out, void *v_out, void *stream);

/*
 * Softmax attention over whole packed sequences: prompts, chunks of prompts over their
 * prefixes (h3q_kv_cache_read_nvfp4), the tokens of video frames.  For query token i of
 * sequence b and head h, with key head h / (heads / kv_heads),
 *   x_j = scale * (q . k_j),  o = sum_j e^(x_j - m) v_j / sum_j e^(x_j - m),  m = max x_j,
 * over the sequence's keys j, with `causal` those with j <= i + (keys - queries): the
 * last query sees the last key.  lse = m + log(sum_j e^(x_j - m)), natural.  A query that
 * sees no key gets o = 0 and lse = -inf.  Products are of bf16 values with fp32 sums, the
 * weights are rounded to bf16, everything else is fp32.  The sums are formed before they
 * are divided, so finite values give finite outputs up to a magnitude of 2^86.  A key or
 * value that is no number reaches only the rows that see it (an infinite value as if its
 * weight were positive).
 *
 *   q           bf16 [rows_q, heads * head_dim], row stride ld_q; k, v bf16 [rows_k,
 *               kv_heads * head_dim], row strides ld_k, ld_v.  32-byte aligned.
 *   cu_q, cu_k  int32 [batch + 1] on the device, not decreasing: sequence b has queries
 *               cu_q[b] .. cu_q[b+1]-1 and keys cu_k[b] .. cu_k[b+1]-1.  Not checked on the
 *               host; no contents make the kernel touch memory outside the buffers.
 *   batch       0 .. 2^24.   rows_q  0 .. 2^31 - 512.   rows_k  0 .. 2^25.
 *   heads       a multiple of kv_heads; heads * head_dim <= 2^24.
 *   head_dim    64, 128 or 256.        scale  finite, > 0 (e.g. head_dim^-0.5).
 *   causal      0 or 1.
 *   o           out, bf16 [rows_q, heads, head_dim] contiguous, 16-byte aligned.
 *   lse         out, fp32 [heads, rows_q], 4-byte aligned, or NULL.
 *               Rows of no sequence are left as they were in both.
 * The kernel's waits are bounded (2 s): if one runs out it stops early, the outputs are
 * unspecified, and h3q_kernel_error_flag reports it.
 */
int h3q_attention_varlen(const void *q, int64_t ld_q, const void *k, int64_t ld_k, const void *v, int64_t ld_v,
                         const int32_t *cu_q, const int32_t *cu_k, int64_t batch, int64_t rows_q,
                         int64_t rows_k, int64_t heads, int64_t kv_heads, int64_t head_dim, int causal,
                         float scale, void *o, float *lse, void *stream);

/*
 * Attention of one or a few new tokens a sequence over the paged cache that holds the
 * sequence's context and, at its last positions, the new tokens themselves (written
 * before by h3q_kv_cache_write_nvfp4 with the same lists): decoding (one token), several
 * drafted tokens in a chain, or a tree of them.  For token i of sequence b and head h,
 * with key head h / (heads / kv_heads) and the values k, v that the cache holds,
 *   x_j = scale * (q . k_j),  o = sum_j e^(x_j - m) v_j / sum_j e^(x_j - m),  m = max x_j,
 * over the keys j that the token sees: all positions before the sequence's new tokens,
 * and of the new tokens those whose bit is set in its mask (bit j: token j of the same
 * sequence; a token sees itself only if its own bit is set), or without masks itself
 * and those before it.  lse = m + log(sum_j e^(x_j - m)), natural.  A token that sees
 * nothing gets o = 0 and lse = -inf.  Weights are rounded to fp16, sums are fp32.
 *
 *   q           bf16 [rows, heads * head_dim], row stride ld_q, 32-byte aligned.
 *   max_rows    1 .. 64: at least the new tokens of any sequence (more of a sequence are
 *               left as they were).
 *   tree_mask   int64 [rows] on the device, 8-byte aligned, or NULL.
 *   heads       a multiple of kv_heads; heads * head_dim <= 2^24.
 *   scale       finite, > 0 (e.g. head_dim^-0.5).
 *   o           out, bf16 [rows, heads, head_dim] contiguous, 16-byte aligned.
 *   lse         out, fp32 [heads, rows], 4-byte aligned, or NULL.
 *               Rows of no sequence are left as they were in both.
 *   workspace   device memory of h3q_attention_cache_workspace_bytes bytes, 256-byte
 *               aligned, any contents; not touched by other work until the stream has
 *               passed this call (two calls that may run at once need one each).
 * The cache and the lists as above.  A page that is not in [0, num_pages) is read as
 * page 0, and the outputs of its sequence are unspecified; kv_len counts at most
 * max_pages * page_size positions.  Launches one or two kernels.  The result does not
 * depend on what else runs.
 */
static inline int64_t h3q_attention_cache_workspace_bytes(int64_t max_rows, int64_t heads, int64_t kv_heads,
                                                          int64_t head_dim)
{
    int64_t shared = max_rows * (heads / kv_heads);
    int64_t tile = shared <= 8 ? 8 : shared <= 16 || head_dim == 256 ? 16 : 32;
    return 608 * (64 + 2 * tile * (head_dim + 2) * 4);
}
int h3q_attention_cache_nvfp4(const void *q, int64_t ld_q, int64_t rows, int64_t heads, int64_t max_rows,
                              const int32_t *cu_rows, const int32_t *kv_len, const int32_t *block_table,
                              int64_t batch, int64_t max_pages, const int64_t *tree_mask,
                              const uint8_t *k_codes, const uint8_t *k_scales, const uint8_t *v_codes,
                              const uint8_t *v_scales, int64_t num_pages, int64_t page_size,
                              int64_t kv_heads, int64_t head_dim, const float *k_global_scale,
                              const float *v_global_scale, float scale, void *o, float *lse,
                              void *workspace, int64_t workspace_bytes, void *stream);

/*
 * QKV epilogue with rotary positions of several axes (the time, height and width of a video's
 * or an image's tokens): bias, RMSNorm of each head with its weight, and a rotation by
 * angles made here from the rows' positions; grouped heads.  Per row and head, in fp32
 * with one rounding to bf16 at the end:
 *   x' = x + b;  n = x' * rsqrt(mean(x'^2) + eps) * w  (q and k; n = x' without the norm);
 *   for pair j = 0 .. ROT/2 - 1, of axis a(j): angle = positions[row][a(j)] * f[j],
 *   (n_a, n_b) -> (n_a cos - n_b sin, n_a sin + n_b cos); the values beyond ROT = the sum of
 *   axis_dims stay.  v: out = bf16(x').
 * The pairs are (j, j + ROT/2), or with `interleaved` (2j, 2j + 1); the axes take them in order,
 * axis_dims[i] / 2 each.  f of pair i of an axis of d values is scale * theta^(-2i/d); with
 * `sections` it is scale * theta^(-2j/ROT) of the pair's number j in all of ROT.  The angle is
 * reduced to a turn in integers before it becomes fp32, so a position of a million loses no more than the frequency has
 * lost, which comes from doubles: the angle is off by at most position * (f * (2 + |log2 theta|) * 2^-51 + 2^-50), and 2^-23
 * of a turn (theta = 10,000 and frequencies up to one: 2^-46 of the position).
 *
 *   q              bf16 [rows, heads * head_dim], k and v [rows, kv_heads * head_dim], row
 *                  strides ld_q, ld_k, ld_v (multiples of 16), 32-byte aligned.
 *   bias_q/k/v     bf16 [columns of it], 32-byte aligned, or NULL: none.
 *   weight_q/k     bf16 [head_dim], 32-byte aligned, or NULL: ones; NULL where norm = 0.
 *   positions      int32 [rows, axes] contiguous, 4-byte aligned (any values).
 *   axes           1 .. 4.   axis_dims, theta, scale: HOST arrays of that length, read during the
 *                  call; axis_dims even and > 0, their sum ROT a multiple of 16, at most head_dim;
 *                  theta finite, > 0; scale finite (a position's unit: a frame rate, an
 *                  interpolation).  With `sections` the first axis's theta serves all.
 *   norm           1, or 0: no norm (weights NULL).   sections, interleaved: 0 or 1.
 *   heads          a multiple of kv_heads; heads * head_dim <= 2^24.  head_dim 64, 128 or 256.
 *   eps            finite, >= 0 (with eps = 0 an all-zero head gives NaN values).
 *   q_out          bf16 [rows, heads, head_dim], k_out and v_out [rows, kv_heads, head_dim],
 *                  contiguous, 16-byte aligned; no output overlaps an input or another.
 * rows = 0 returns H3Q_OK with no launch.  No page has a counterpart; the pages' own epilogue
 * is h3q_qkv_epilogue.
 */
int h3q_qkv_epilogue_axes(const void *q, int64_t ld_q, const void *k, int64_t ld_k, const void *v,
                          int64_t ld_v, const void *bias_q, const void *bias_k, const void *bias_v,
                          const void *weight_q, const void *weight_k, const int32_t *positions,
                          int64_t axes, const int64_t *axis_dims, const double *theta, const double *scale,
                          int sections, int interleaved, int norm, int64_t rows, int64_t heads,
                          int64_t kv_heads, int64_t head_dim, float eps, void *q_out, void *k_out,
                          void *v_out, void *stream);

/*
 * Norms on both sides of a block with its gate and scaled residual, and NVFP4 of the result:
 *   u  = bf16(fl(o + bias))                       (u = o without a bias)
 *   n  = fl(fl(u * rstd(u)) * gamma_post),        then fl(n * gate[t]) with a gate table
 *   h' = fl(fl(residual_scale * h) + n)           written back to h
 *   y  = bf16(m), m = fl(fl(h' * rstd(h')) * gamma), with a modulation table
 *        m = fl(fl(m * fl(1 + scale[t])) + shift[t])
 * and the NVFP4 quantize of y.  t is the row's frame; both rstd have the canonical order and
 * the eps of h3q_rmsnorm_adaln_nvfp4, so results are bit-exact.  Without tables it is the sandwich
 * norm of language models.  h3q_residual_rmsnorm_adaln_nvfp4 is the same without the first norm.
 *
 *   h           fp32 [rows, cols], row stride ld_h (a multiple of 8), 32-byte aligned, updated.
 *   o           bf16 [rows, cols], row stride ld_o.   bias  bf16 [cols] or NULL.
 *   gamma_post, gamma  bf16 [cols].                   residual_scale  finite.
 *   gate_table  bf16 [num_frames, cols] or NULL.      mod_table  bf16 [num_frames, 2, cols]
 *               ([t, 0] shift, [t, 1] scale) or NULL.  32-byte aligned.
 *   num_frames, row_frame, rows_per_frame: as h3q_rmsnorm_adaln_nvfp4; not looked at where there
 *               is no table.
 *   cols        at most 8,192.   codes, scales, row_rstd (of h'; may be NULL): as there.
 * Other preconditions and status codes as h3q_residual_rmsnorm_adaln_nvfp4.
 */
int h3q_postnorm_residual_adaln_nvfp4(float *h, int64_t ld_h, const void *o, int64_t ld_o, const void *bias,
                                      const void *gamma_post, const void *gate_table, float residual_scale,
                                      const void *gamma, const void *mod_table, int64_t num_frames,
                                      const int32_t *row_frame, int64_t rows_per_frame, float eps,
                                      int64_t rows, int64_t cols, const float *global_scale,
                                      uint8_t *codes, uint8_t *scales, float *row_rstd, void *stream);

/*
 * Sparse attention over blocks: each block of block_q consecutive queries of a sequence
 * attends, for each key head, to a list of blocks of block_k consecutive keys of the sequence.
 * h3q_select_blocks makes the lists, h3q_attention_blocks attends over them (or over any others).
 *
 *   cu_q, cu_k, batch, rows_q, rows_k, heads, kv_heads: packed sequences as in
 *                h3q_attention_varlen.  head_dim 64 or 128.  `causal`: query i of a sequence sees
 *                its keys j <= i + (keys - queries).
 *   block_q, block_k  64, 128 or 256.  The last block of a sequence may be shorter.
 *   blocks       int32 [kv_heads, h3q_block_rows(rows_q, batch, block_q), top]: query block i
 *                of sequence b has row cu_q[b] / block_q + b + i.  Rows of no query block are
 *                there too.
 *   top          1 .. 4,096.
 */
static inline int64_t h3q_block_rows(int64_t rows, int64_t batch, int64_t block)
{
    return rows / block + batch;
}

/*
 * The blocks that a query block attends to, by a cheap score: the mean of its query rows
 * (over the heads of the group too) times the mean of the block's keys.  Each list holds
 * the numbers of the `top` blocks with the highest scores (of equal ones those with the
 * lowest numbers) in ascending order, then -1 where there are fewer blocks.  Always among them,
 * whatever their scores: the first `first` blocks, and with `causal` those that hold the query
 * block's own positions (keys - queries + i of query i); causal blocks of later keys alone are
 * not candidates.  The choice is that of the exact scores, but where two differ by less than 2^-37 of |q| |k|, the
 * lengths of the means as vectors (k: the longest of the sequence): where fp32 is too coarse to tell, they are formed
 * again from sums held in pairs of fp32.  (Those are exact where the values
 * of a block's columns lie within a factor of 2^18 of each other, up to 256 of them, and else off by
 * 2^-20 of the largest at most.  The length of a block's sums as a vector and the scores of sums have to fit
 * fp32, not what comes up on the way.)  A score that is no number counts as the lowest.
 *
 *   q            bf16 [rows_q, heads * head_dim], row stride ld_q; k bf16 [rows_k, kv_heads *
 *                head_dim], row stride ld_k; 32-byte aligned.
 *   first        0 .. top.  With causal, top >= first + ceil(block_q / block_k) + 1.
 *   blocks       out, 4-byte aligned; rows of no query block get -1.
 *   scores       out, fp32 of the same shape: the entries' scores, off by 176 * 2^-24 of |q| |k| (the entry's own) and
 *                2^-22 of themselves at most, -inf beside -1; or NULL.
 *   workspace    device memory of h3q_select_blocks_workspace_bytes bytes, 256-byte aligned, any
 *                contents; not touched by other work until the stream has passed this call.
 * rows_q <= 2^31 - 512.  Two launches.  Where rows_k / block_k is above 16,000 (of all sequences together) the
 * workspace has room for rows of scores too: those of a sequence that has so many blocks by itself are kept
 * there, and take longer to choose from.
 */
static inline int64_t h3q_select_blocks_workspace_bytes(int64_t rows_q, int64_t rows_k, int64_t batch,
                                                        int64_t kv_heads, int64_t head_dim, int64_t block_q,
                                                        int64_t block_k)
{
    int64_t rows = h3q_block_rows(rows_q, batch, block_q) + h3q_block_rows(rows_k, batch, block_k);
    int64_t bytes = rows * kv_heads * (head_dim + 1) * 8 +
                    (h3q_block_rows(rows_k, batch, block_k) * kv_heads + 7) / 8 * 8 * head_dim * 4 + 256;
    if (rows_k / block_k > 16000) {
        int64_t lists = h3q_block_rows(rows_q, batch, block_q) * kv_heads;
        bytes += (lists < 1024 ? lists : 1024) * ((rows_k / block_k + 32) / 32 * 32) * 4;
    }
    return bytes;
}
int h3q_select_blocks(const void *q, int64_t ld_q, const void *k, int64_t ld_k, const int32_t *cu_q,
                      const int32_t *cu_k, int64_t batch, int64_t rows_q, int64_t rows_k, int64_t heads,
                      int64_t kv_heads, int64_t head_dim, int64_t block_q, int64_t block_k, int64_t top,
                      int causal, int64_t first, int32_t *blocks, float *scores, void *workspace,
                      int64_t workspace_bytes, void *stream);

/*
 * Softmax attention as h3q_attention_varlen's over the keys of the listed blocks alone: prompts,
 * video, and single new tokens (a sequence of one query).  An entry of a list counts
 * if it is the number of a block of the sequence and above all entries before it that count
 * (so a block named twice counts once); all others are passed over.  A query that sees no key gets
 * o = 0 and lse = -inf.  Rounding, magnitudes, numbers that are none, o and lse as there.
 * Fewer than 2^31 units of work, pairs of row tiles of up to 128 rows of a sequence's tokens and heads.
 * The kernel's waits are bounded (2 s): if one runs out it stops early, the outputs are
 * unspecified, and h3q_kernel_error_flag reports it.
 */
int h3q_attention_blocks(const void *q, int64_t ld_q, const void *k, int64_t ld_k, const void *v, int64_t ld_v,
                         const int32_t *cu_q, const int32_t *cu_k, int64_t batch, int64_t rows_q,
                         int64_t rows_k, int64_t heads, int64_t kv_heads, int64_t head_dim, int64_t block_q,
                         int64_t block_k, const int32_t *blocks, int64_t top, int causal, float scale,
                         void *o, float *lse, void *stream);

/* Message for the calling thread's most recent failed call ("" if none). */
const char *h3q_last_error(void);

/* H3Q_ABI_VERSION of the loaded library. */
int h3q_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* H3Q_H */
