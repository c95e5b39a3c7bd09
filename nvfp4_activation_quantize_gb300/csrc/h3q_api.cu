// h3q_api.cu -- the exported C ABI (include/h3q.h): host-side validation, then
// one kernel launch on the caller's stream.  No allocation, no synchronisation.
// An argument that breaks the contract returns H3Q_ERR_INVALID_ARGUMENT before
// any CUDA call, so these checks also run on machines without a GPU.
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <mutex>
#include <string>

#include <cuda.h>  // driver types only; the two driver calls are fetched at run time

#include "../../include/h3q.h"
#include "h3q_internal.h"

namespace {

thread_local std::string g_last_error;

int fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return code;
}

int invalid(const char* fn, const char* what) {
  return fail(H3Q_ERR_INVALID_ARGUMENT, "%s: %s", fn, what);
}

int cuda_failed(const char* fn, cudaError_t err) {
  return fail(H3Q_ERR_CUDA, "%s: CUDA error %d (%s): %s", fn, static_cast<int>(err),
              cudaGetErrorName(err), cudaGetErrorString(err));
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

constexpr int64_t kMaxCols = int64_t(1) << 24;
constexpr int64_t kMaxRows = int64_t(1) << 40;
// Sequences of a call: the kernels count them in 32 bits, up to a thousand past the last, and the prompt
// kernel looks a unit's up 32 at a time while its other warps wait for it, at most 2 s.
constexpr int64_t kMaxBatch = int64_t(1) << 24;

// Byte range [p, p + n) of a buffer, for overlap checks.
struct Span {
  uintptr_t lo, hi;
};
Span span(const void* p, int64_t bytes) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return {lo, lo + static_cast<uintptr_t>(bytes)};
}
bool overlap(Span a, Span b) { return a.lo < b.hi && b.lo < a.hi; }

// Bytes spanned by a bf16 [rows, cols] view with row stride ld.
int64_t view_bytes(int64_t rows, int64_t cols, int64_t ld) { return ((rows - 1) * ld + cols) * 2; }

// Shared shape checks; returns 0 or an error code (message already set).
int check_shape(const char* fn, int64_t rows, int64_t cols) {
  if (rows < 0) return invalid(fn, "rows must be >= 0");
  if (rows > kMaxRows) return invalid(fn, "rows exceeds 2^40");
  if (cols <= 0 || cols % 64 != 0) return invalid(fn, "cols must be a positive multiple of 64");
  if (cols > kMaxCols) return invalid(fn, "cols exceeds 2^24");
  return 0;
}

int check_input(const char* fn, const char* name, const void* p, int64_t ld, int64_t rows,
                int64_t cols) {
  char msg[160];
  if (p == nullptr) return snprintf(msg, sizeof msg, "%s is NULL", name), invalid(fn, msg);
  if (!aligned(p, 32)) return snprintf(msg, sizeof msg, "%s must be 32-byte aligned", name), invalid(fn, msg);
  if (ld < cols || ld % 16 != 0)
    return snprintf(msg, sizeof msg, "ld of %s must be >= cols and a multiple of 16", name), invalid(fn, msg);
  if (ld > (int64_t(1) << 62) / (rows > 0 ? rows : 1))
    return snprintf(msg, sizeof msg, "%s: rows * ld overflows", name), invalid(fn, msg);
  return 0;
}

int check_outputs(const char* fn, const uint8_t* codes, const uint8_t* scales,
                  const float* gsf) {
  if (codes == nullptr || scales == nullptr) return invalid(fn, "codes and scales must not be NULL");
  if (!aligned(codes, 16) || !aligned(scales, 16))
    return invalid(fn, "codes and scales must be 16-byte aligned");
  if (gsf == nullptr || !aligned(gsf, 4)) return invalid(fn, "global_scale must be a 4-byte aligned pointer");
  return 0;
}

// --- per-context, per-kernel launch-size cache ------------------------------

// A kernel whose attributes a runtime call can query: the query loads the
// library's module into the current context, which binds the device's primary
// context to the calling thread when none is current.
__global__ void context_probe_kernel() {}

struct OccupancyEntry {
  const void* kernel;
  unsigned long long context;
  int threads;
  int smem_bytes;
  int blocks_per_sm;
  int sms;
};
constexpr int kOccEntries = 256;
std::mutex g_occ_mutex;
OccupancyEntry g_occ[kOccEntries];
int g_occ_n = 0;
int g_occ_next = 0;

}  // namespace

namespace h3q {

cudaError_t current_context_id(unsigned long long* id) {
  using GetCurrent = CUresult (*)(CUcontext*);
  using GetId = CUresult (*)(CUcontext, unsigned long long*);
  static std::once_flag once;
  static GetCurrent get_current = nullptr;
  static GetId get_id = nullptr;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuCtxGetCurrent", &f, 12000, cudaEnableDefault, &found) ==
            cudaSuccess && found == cudaDriverEntryPointSuccess)
      get_current = reinterpret_cast<GetCurrent>(f);
    if (cudaGetDriverEntryPointByVersion("cuCtxGetId", &f, 12000, cudaEnableDefault, &found) ==
            cudaSuccess && found == cudaDriverEntryPointSuccess)
      get_id = reinterpret_cast<GetId>(f);
  });
  if (get_current == nullptr || get_id == nullptr) return cudaErrorNotSupported;
  CUcontext ctx = nullptr;
  if (get_current(&ctx) != CUDA_SUCCESS) return cudaErrorDeviceUninitialized;
  if (ctx == nullptr) {  // no context on this thread yet: let the runtime bind the primary one
    cudaFuncAttributes attr;
    cudaError_t err = cudaFuncGetAttributes(&attr, reinterpret_cast<const void*>(&context_probe_kernel));
    if (err != cudaSuccess) return err;
    if (get_current(&ctx) != CUDA_SUCCESS || ctx == nullptr) return cudaErrorDeviceUninitialized;
  }
  return get_id(ctx, id) == CUDA_SUCCESS ? cudaSuccess : cudaErrorDeviceUninitialized;
}

cudaError_t persistent_blocks(const void* kernel, int threads, int smem_bytes, int64_t max_blocks,
                              int* blocks) {
  int device = 0;
  cudaError_t err = cudaGetDevice(&device);
  if (err != cudaSuccess) return err;
  // Keyed on the context, not the device ordinal: the shared-memory limit set
  // below belongs to the context, and a context the caller re-creates (after
  // cudaDeviceReset, say) starts without it.
  unsigned long long context = 0;
  if ((err = current_context_id(&context)) != cudaSuccess) return err;
  int per_sm = 0, sms = 0;
  {
    std::lock_guard<std::mutex> lock(g_occ_mutex);
    for (int i = 0; i < g_occ_n; ++i)
      if (g_occ[i].kernel == kernel && g_occ[i].context == context && g_occ[i].threads == threads &&
          g_occ[i].smem_bytes == smem_bytes) {
        per_sm = g_occ[i].blocks_per_sm;
        sms = g_occ[i].sms;
      }
  }
  if (per_sm == 0) {
    err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device);
    if (err != cudaSuccess) return err;
    if (smem_bytes > 0) {  // the default limit leaves no room beside static shared memory
      err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes);
      if (err != cudaSuccess) return err;
    }
    err = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, smem_bytes);
    if (err != cudaSuccess) return err;
    if (per_sm < 1) return cudaErrorInvalidConfiguration;
    std::lock_guard<std::mutex> lock(g_occ_mutex);
    if (g_occ_n < kOccEntries) {
      g_occ[g_occ_n++] = {kernel, context, threads, smem_bytes, per_sm, sms};
    } else {  // full (many contexts over the process's life): reuse the slots in turn
      g_occ[g_occ_next] = {kernel, context, threads, smem_bytes, per_sm, sms};
      g_occ_next = (g_occ_next + 1) % kOccEntries;
    }
  }
  int64_t n = static_cast<int64_t>(per_sm) * sms;
  if (max_blocks < n) n = max_blocks;
  *blocks = static_cast<int>(n < 1 ? 1 : n);
  return cudaSuccess;
}

}  // namespace h3q

extern "C" {

const char* h3q_last_error(void) { return g_last_error.c_str(); }

int h3q_abi_version(void) { return H3Q_ABI_VERSION; }

int h3q_quantize_nvfp4(const void* x, int64_t ld_x, int64_t rows, int64_t cols,
                       const float* global_scale, uint8_t* codes, uint8_t* scales,
                       void* stream) {
  static const char* fn = "h3q_quantize_nvfp4";
  g_last_error.clear();
  if (int e = check_shape(fn, rows, cols)) return e;
  if (rows == 0) return H3Q_OK;
  if (int e = check_input(fn, "x", x, ld_x, rows, cols)) return e;
  if (int e = check_outputs(fn, codes, scales, global_scale)) return e;
  const Span in = span(x, view_bytes(rows, cols, ld_x));
  const Span c = span(codes, h3q_code_bytes(rows, cols));
  const Span s = span(scales, h3q_scale_bytes(rows, cols));
  if (overlap(in, c) || overlap(in, s) || overlap(c, s)) return invalid(fn, "outputs overlap an input or each other");
  cudaError_t err = h3q::launch_quantize(static_cast<const uint16_t*>(x), ld_x, rows, cols,
                                         global_scale, codes, scales,
                                         static_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? H3Q_OK : cuda_failed(fn, err);
}

int h3q_rmsnorm_adaln_nvfp4(const void* x, int64_t ld_x, const void* gamma, const void* mod_table,
                            int64_t num_frames, const int32_t* row_frame, int64_t rows_per_frame,
                            float eps, int64_t rows, int64_t cols, const float* global_scale,
                            uint8_t* codes, uint8_t* scales, float* row_rstd, void* stream) {
  static const char* fn = "h3q_rmsnorm_adaln_nvfp4";
  g_last_error.clear();
  if (int e = check_shape(fn, rows, cols)) return e;
  if (!std::isfinite(eps) || eps < 0.0f) return invalid(fn, "eps must be finite and >= 0");
  if (num_frames < 1) return invalid(fn, "num_frames must be >= 1");
  if (num_frames > (int64_t(1) << 31)) return invalid(fn, "num_frames exceeds 2^31");
  if (rows == 0) return H3Q_OK;
  if (int e = check_input(fn, "x", x, ld_x, rows, cols)) return e;
  if (int e = check_input(fn, "gamma", gamma, cols, 1, cols)) return e;
  if (int e = check_input(fn, "mod_table", mod_table, cols, 2 * num_frames, cols)) return e;
  if (int e = check_outputs(fn, codes, scales, global_scale)) return e;
  if (row_frame != nullptr) {
    if (!aligned(row_frame, 4)) return invalid(fn, "row_frame must be 4-byte aligned");
  } else {
    if (rows_per_frame < 1) return invalid(fn, "rows_per_frame must be >= 1 when row_frame is NULL");
    if ((rows - 1) / rows_per_frame >= num_frames)
      return invalid(fn, "rows / rows_per_frame reaches past the modulation table");
  }
  if (row_rstd != nullptr && !aligned(row_rstd, 4)) return invalid(fn, "row_rstd must be 4-byte aligned");
  const Span c = span(codes, h3q_code_bytes(rows, cols));
  const Span s = span(scales, h3q_scale_bytes(rows, cols));
  const Span ins[4] = {span(x, view_bytes(rows, cols, ld_x)), span(gamma, cols * 2),
                       span(mod_table, num_frames * 4 * cols),
                       row_frame ? span(row_frame, rows * 4) : Span{0, 0}};
  if (overlap(c, s)) return invalid(fn, "codes and scales overlap");
  for (const Span& in : ins)
    if (overlap(in, c) || overlap(in, s)) return invalid(fn, "an output overlaps an input");
  if (row_rstd != nullptr) {
    const Span r = span(row_rstd, rows * 4);
    if (overlap(r, c) || overlap(r, s)) return invalid(fn, "row_rstd overlaps an output");
    for (const Span& in : ins)
      if (overlap(in, r)) return invalid(fn, "row_rstd overlaps an input");
  }
  cudaError_t err = h3q::launch_adaln(
      static_cast<const uint16_t*>(x), ld_x, static_cast<const uint16_t*>(gamma),
      static_cast<const uint16_t*>(mod_table), num_frames, row_frame, rows_per_frame, eps, rows,
      cols, global_scale, codes, scales, row_rstd, static_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? H3Q_OK : cuda_failed(fn, err);
}

int h3q_rmsnorm_adaln_nvfp4_from_rstd(const void* x, int64_t ld_x, const void* gamma, const void* mod_table,
                                      int64_t num_frames, const int32_t* row_frame, int64_t rows_per_frame,
                                      const float* row_rstd, int64_t rows, int64_t cols,
                                      const float* global_scale, uint8_t* codes, uint8_t* scales, void* stream) {
  static const char* fn = "h3q_rmsnorm_adaln_nvfp4_from_rstd";
  g_last_error.clear();
  if (int e = check_shape(fn, rows, cols)) return e;
  if (num_frames < 1) return invalid(fn, "num_frames must be >= 1");
  if (num_frames > (int64_t(1) << 31)) return invalid(fn, "num_frames exceeds 2^31");
  if (rows == 0) return H3Q_OK;
  if (int e = check_input(fn, "x", x, ld_x, rows, cols)) return e;
  if (int e = check_input(fn, "gamma", gamma, cols, 1, cols)) return e;
  if (int e = check_input(fn, "mod_table", mod_table, cols, 2 * num_frames, cols)) return e;
  if (int e = check_outputs(fn, codes, scales, global_scale)) return e;
  if (row_frame != nullptr) {
    if (!aligned(row_frame, 4)) return invalid(fn, "row_frame must be 4-byte aligned");
  } else {
    if (rows_per_frame < 1) return invalid(fn, "rows_per_frame must be >= 1 when row_frame is NULL");
    if ((rows - 1) / rows_per_frame >= num_frames)
      return invalid(fn, "rows / rows_per_frame reaches past the modulation table");
  }
  if (row_rstd == nullptr) return invalid(fn, "row_rstd is NULL");
  if (!aligned(row_rstd, 4)) return invalid(fn, "row_rstd must be 4-byte aligned");
  const Span c = span(codes, h3q_code_bytes(rows, cols));
  const Span s = span(scales, h3q_scale_bytes(rows, cols));
  const Span ins[5] = {span(x, view_bytes(rows, cols, ld_x)), span(gamma, cols * 2),
                       span(mod_table, num_frames * 4 * cols),
                       row_frame ? span(row_frame, rows * 4) : Span{0, 0}, span(row_rstd, rows * 4)};
  if (overlap(c, s)) return invalid(fn, "codes and scales overlap");
  for (const Span& in : ins)
    if (overlap(in, c) || overlap(in, s)) return invalid(fn, "an output overlaps an input");
  cudaError_t err = h3q::launch_adaln_from_rstd(
      static_cast<const uint16_t*>(x), ld_x, static_cast<const uint16_t*>(gamma),
      static_cast<const uint16_t*>(mod_table), num_frames, row_frame, rows_per_frame, row_rstd, rows, cols,
      global_scale, codes, scales, static_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? H3Q_OK : cuda_failed(fn, err);
}

int h3q_swiglu_nvfp4(const void* gate, int64_t ld_gate, const void* up, int64_t ld_up,
                     int64_t rows, int64_t cols, const float* global_scale, uint8_t* codes,
                     uint8_t* scales, void* stream) {
  static const char* fn = "h3q_swiglu_nvfp4";
  g_last_error.clear();
  if (int e = check_shape(fn, rows, cols)) return e;
  if (rows == 0) return H3Q_OK;
  if (int e = check_input(fn, "gate", gate, ld_gate, rows, cols)) return e;
  if (int e = check_input(fn, "up", up, ld_up, rows, cols)) return e;
  if (int e = check_outputs(fn, codes, scales, global_scale)) return e;
  const Span g = span(gate, view_bytes(rows, cols, ld_gate));
  const Span u = span(up, view_bytes(rows, cols, ld_up));
  const Span c = span(codes, h3q_code_bytes(rows, cols));
  const Span s = span(scales, h3q_scale_bytes(rows, cols));
  if (overlap(g, c) || overlap(g, s) || overlap(u, c) || overlap(u, s) || overlap(c, s))
    return invalid(fn, "outputs overlap an input or each other");
  cudaError_t err = h3q::launch_swiglu(static_cast<const uint16_t*>(gate), ld_gate,
                                       static_cast<const uint16_t*>(up), ld_up, rows, cols,
                                       global_scale, codes, scales,
                                       static_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? H3Q_OK : cuda_failed(fn, err);
}

int h3q_residual_rmsnorm_adaln_nvfp4(float* h, int64_t ld_h, const void* o, int64_t ld_o,
                                     const void* bias, const void* gate_table, const void* gamma,
                                     const void* mod_table, int64_t num_frames,
                                     const int32_t* row_frame, int64_t rows_per_frame, float eps,
                                     int64_t rows, int64_t cols, const float* global_scale,
                                     uint8_t* codes, uint8_t* scales, float* row_rstd,
                                     void* stream) {
  static const char* fn = "h3q_residual_rmsnorm_adaln_nvfp4";
  g_last_error.clear();
  if (int e = check_shape(fn, rows, cols)) return e;
  if (cols > 8192) return invalid(fn, "cols exceeds 8,192");
  if (!std::isfinite(eps) || eps < 0.0f) return invalid(fn, "eps must be finite and >= 0");
  if (num_frames < 1) return invalid(fn, "num_frames must be >= 1");
  if (num_frames > (int64_t(1) << 31)) return invalid(fn, "num_frames exceeds 2^31");
  if (rows == 0) return H3Q_OK;
  if (h == nullptr || !aligned(h, 32)) return invalid(fn, "h must be a 32-byte aligned pointer");
  if (ld_h < cols || ld_h % 8 != 0) return invalid(fn, "ld of h must be >= cols and a multiple of 8");
  if (ld_h > (int64_t(1) << 61) / rows) return invalid(fn, "h: rows * ld overflows");
  if (int e = check_input(fn, "o", o, ld_o, rows, cols)) return e;
  if (bias != nullptr)
    if (int e = check_input(fn, "bias", bias, cols, 1, cols)) return e;
  if (int e = check_input(fn, "gate_table", gate_table, cols, num_frames, cols)) return e;
  if (int e = check_input(fn, "gamma", gamma, cols, 1, cols)) return e;
  if (int e = check_input(fn, "mod_table", mod_table, cols, 2 * num_frames, cols)) return e;
  if (int e = check_outputs(fn, codes, scales, global_scale)) return e;
  if (row_frame != nullptr) {
    if (!aligned(row_frame, 4)) return invalid(fn, "row_frame must be 4-byte aligned");
  } else {
    if (rows_per_frame < 1) return invalid(fn, "rows_per_frame must be >= 1 when row_frame is NULL");
    if ((rows - 1) / rows_per_frame >= num_frames)
      return invalid(fn, "rows / rows_per_frame reaches past the modulation table");
  }
  if (row_rstd != nullptr && !aligned(row_rstd, 4)) return invalid(fn, "row_rstd must be 4-byte aligned");
  const Span hs = span(h, ((rows - 1) * ld_h + cols) * 4);
  const Span c = span(codes, h3q_code_bytes(rows, cols));
  const Span sc = span(scales, h3q_scale_bytes(rows, cols));
  const Span r = row_rstd ? span(row_rstd, rows * 4) : Span{0, 0};
  const Span ins[7] = {span(o, view_bytes(rows, cols, ld_o)), bias ? span(bias, cols * 2) : Span{0, 0},
                       span(gate_table, num_frames * 2 * cols), span(gamma, cols * 2),
                       span(mod_table, num_frames * 4 * cols),
                       row_frame ? span(row_frame, rows * 4) : Span{0, 0}, span(global_scale, 4)};
  const Span outs[4] = {hs, c, sc, r};
  for (int i = 0; i < 4; ++i) {
    for (const Span& in : ins)
      if (overlap(outs[i], in)) return invalid(fn, "an output (h, codes, scales, row_rstd) overlaps an input");
    for (int k = i + 1; k < 4; ++k)
      if (overlap(outs[i], outs[k])) return invalid(fn, "outputs overlap each other");
  }
  cudaError_t err = h3q::launch_residual_adaln(
      h, ld_h, static_cast<const uint16_t*>(o), ld_o, static_cast<const uint16_t*>(bias),
      static_cast<const uint16_t*>(gate_table), static_cast<const uint16_t*>(gamma),
      static_cast<const uint16_t*>(mod_table), num_frames, row_frame, rows_per_frame, eps, rows,
      cols, global_scale, codes, scales, row_rstd, static_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? H3Q_OK : cuda_failed(fn, err);
}

// --- dynamic and calibrated scales ------------------------------------------

namespace {
int check_amax(const char* fn, const float* amax) {
  if (amax == nullptr || !aligned(amax, 4)) return invalid(fn, "amax must be a 4-byte aligned pointer");
  return 0;
}
}  // namespace

int h3q_amax_bf16(const void* x, int64_t ld_x, int64_t rows, int64_t cols, float* amax,
                  void* stream) {
  static const char* fn = "h3q_amax_bf16";
  g_last_error.clear();
  if (int e = check_shape(fn, rows, cols)) return e;
  if (rows == 0) return H3Q_OK;
  if (int e = check_input(fn, "x", x, ld_x, rows, cols)) return e;
  if (int e = check_amax(fn, amax)) return e;
  if (overlap(span(x, view_bytes(rows, cols, ld_x)), span(amax, 4))) return invalid(fn, "amax overlaps x");
  cudaError_t err = h3q::launch_amax_bf16(static_cast<const uint16_t*>(x), ld_x, rows, cols, amax,
                                          static_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? H3Q_OK : cuda_failed(fn, err);
}

int h3q_rmsnorm_adaln_amax(const void* x, int64_t ld_x, const void* gamma, const void* mod_table,
                           int64_t num_frames, const int32_t* row_frame, int64_t rows_per_frame,
                           float eps, int64_t rows, int64_t cols, float* amax, float* row_rstd,
                           void* stream) {
  static const char* fn = "h3q_rmsnorm_adaln_amax";
  g_last_error.clear();
  if (int e = check_shape(fn, rows, cols)) return e;
  if (!std::isfinite(eps) || eps < 0.0f) return invalid(fn, "eps must be finite and >= 0");
  if (num_frames < 1) return invalid(fn, "num_frames must be >= 1");
  if (num_frames > (int64_t(1) << 31)) return invalid(fn, "num_frames exceeds 2^31");
  if (rows == 0) return H3Q_OK;
  if (int e = check_input(fn, "x", x, ld_x, rows, cols)) return e;
  if (int e = check_input(fn, "gamma", gamma, cols, 1, cols)) return e;
  if (int e = check_input(fn, "mod_table", mod_table, cols, 2 * num_frames, cols)) return e;
  if (int e = check_amax(fn, amax)) return e;
  if (row_frame != nullptr) {
    if (!aligned(row_frame, 4)) return invalid(fn, "row_frame must be 4-byte aligned");
  } else {
    if (rows_per_frame < 1) return invalid(fn, "rows_per_frame must be >= 1 when row_frame is NULL");
    if ((rows - 1) / rows_per_frame >= num_frames)
      return invalid(fn, "rows / rows_per_frame reaches past the modulation table");
  }
  const Span am = span(amax, 4);
  const Span ins[4] = {span(x, view_bytes(rows, cols, ld_x)), span(gamma, cols * 2),
                       span(mod_table, num_frames * 4 * cols),
                       row_frame ? span(row_frame, rows * 4) : Span{0, 0}};
  for (const Span& in : ins)
    if (overlap(am, in)) return invalid(fn, "amax overlaps an input");
  if (row_rstd != nullptr) {
    if (!aligned(row_rstd, 4)) return invalid(fn, "row_rstd must be 4-byte aligned");
    const Span r = span(row_rstd, rows * 4);
    if (overlap(r, am)) return invalid(fn, "row_rstd overlaps amax");
    for (const Span& in : ins)
      if (overlap(r, in)) return invalid(fn, "row_rstd overlaps an input");
  }
  cudaError_t err = h3q::launch_adaln_amax(
      static_cast<const uint16_t*>(x), ld_x, static_cast<const uint16_t*>(gamma),
      static_cast<const uint16_t*>(mod_table), num_frames, row_frame, rows_per_frame, eps, rows,
      cols, amax, row_rstd, static_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? H3Q_OK : cuda_failed(fn, err);
}

int h3q_swiglu_amax(const void* gate, int64_t ld_gate, const void* up, int64_t ld_up,
                    int64_t rows, int64_t cols, float* amax, void* stream) {
  static const char* fn = "h3q_swiglu_amax";
  g_last_error.clear();
  if (int e = check_shape(fn, rows, cols)) return e;
  if (rows == 0) return H3Q_OK;
  if (int e = check_input(fn, "gate", gate, ld_gate, rows, cols)) return e;
  if (int e = check_input(fn, "up", up, ld_up, rows, cols)) return e;
  if (int e = check_amax(fn, amax)) return e;
  const Span am = span(amax, 4);
  if (overlap(am, span(gate, view_bytes(rows, cols, ld_gate))) ||
      overlap(am, span(up, view_bytes(rows, cols, ld_up))))
    return invalid(fn, "amax overlaps an input");
  cudaError_t err = h3q::launch_swiglu_amax(static_cast<const uint16_t*>(gate), ld_gate,
                                            static_cast<const uint16_t*>(up), ld_up, rows, cols,
                                            amax, static_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? H3Q_OK : cuda_failed(fn, err);
}

int h3q_global_scale_from_amax(const float* amax, float* global_scale, void* stream) {
  static const char* fn = "h3q_global_scale_from_amax";
  g_last_error.clear();
  if (int e = check_amax(fn, amax)) return e;
  if (global_scale == nullptr || !aligned(global_scale, 4))
    return invalid(fn, "global_scale must be a 4-byte aligned pointer");
  cudaError_t err = h3q::launch_global_scale(amax, global_scale, static_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? H3Q_OK : cuda_failed(fn, err);
}

int h3q_quantize_nvfp4_dynamic(const void* x, int64_t ld_x, int64_t rows, int64_t cols,
                               float* global_scale, uint8_t* codes, uint8_t* scales,
                               void* stream) {
  static const char* fn = "h3q_quantize_nvfp4_dynamic";
  g_last_error.clear();
  if (int e = check_shape(fn, rows, cols)) return e;
  if (rows == 0) return H3Q_OK;
  if (int e = check_input(fn, "x", x, ld_x, rows, cols)) return e;
  if (int e = check_outputs(fn, codes, scales, global_scale)) return e;
  const Span in = span(x, view_bytes(rows, cols, ld_x));
  const Span c = span(codes, h3q_code_bytes(rows, cols));
  const Span s = span(scales, h3q_scale_bytes(rows, cols));
  const Span g = span(global_scale, 4);
  if (overlap(in, c) || overlap(in, s) || overlap(c, s) || overlap(g, in) || overlap(g, c) ||
      overlap(g, s))
    return invalid(fn, "outputs overlap an input or each other");
  int blocks = 0;
  cudaError_t err = h3q::dynamic_scale_partials(rows, cols, &blocks);
  if (err != cudaSuccess) return cuda_failed(fn, err);
  if (blocks > h3q::kMaxDynamicPartials)
    return fail(H3Q_ERR_INVALID_ARGUMENT, "%s: the abs-max pass needs %d partial maxima, more than "
                "the %d the static scratch holds", fn, blocks, h3q::kMaxDynamicPartials);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const float* partials = nullptr;
  err = h3q::launch_dynamic_partials(static_cast<const uint16_t*>(x), ld_x, rows, cols, blocks, &partials, st);
  if (err != cudaSuccess) return cuda_failed(fn, err);
  err = h3q::launch_quantize_after_partials(static_cast<const uint16_t*>(x), ld_x, rows, cols, partials, blocks,
                                            global_scale, codes, scales, st);
  return err == cudaSuccess ? H3Q_OK : cuda_failed(fn, err);
}

int h3q_gemm_swiglu_nvfp4(const uint8_t* a_codes, const uint8_t* a_scales, int64_t m, int64_t k,
                          const uint8_t* b_codes, const uint8_t* b_scales, int64_t n, const float* alpha,
                          const float* global_scale, uint8_t* codes, uint8_t* scales, void* y, float* acc,
                          void* stream) {
  static const char* fn = "h3q_gemm_swiglu_nvfp4";
  g_last_error.clear();
  if (m < 0) return invalid(fn, "m must be >= 0");
  if (m > (int64_t(1) << 31) - 128) return invalid(fn, "m exceeds 2^31 - 128");
  if (k <= 0 || k % 256 != 0 || k > kMaxCols) return invalid(fn, "k must be a positive multiple of 256, at most 2^24");
  if (n <= 0 || n % 256 != 0 || n > kMaxCols) return invalid(fn, "n must be a positive multiple of 256, at most 2^24");
  if (m == 0) return H3Q_OK;
  if (a_codes == nullptr || b_codes == nullptr || a_scales == nullptr || b_scales == nullptr)
    return invalid(fn, "a_codes, a_scales, b_codes and b_scales must not be NULL");
  if (!aligned(a_codes, 16) || !aligned(b_codes, 16) || !aligned(a_scales, 16) || !aligned(b_scales, 16))
    return invalid(fn, "a_codes, a_scales, b_codes and b_scales must be 16-byte aligned");
  if (alpha == nullptr || !aligned(alpha, 4)) return invalid(fn, "alpha must be a 4-byte aligned pointer");
  if (int e = check_outputs(fn, codes, scales, global_scale)) return e;
  if ((y != nullptr && !aligned(y, 16)) || (acc != nullptr && !aligned(acc, 16)))
    return invalid(fn, "y and acc must be 16-byte aligned (or NULL)");
  const int64_t f = n / 2;
  const Span in[] = {span(a_codes, m * (k / 2)), span(a_scales, h3q_scale_bytes(m, k)),
                     span(b_codes, n * (k / 2)), span(b_scales, h3q_scale_bytes(n, k)), span(alpha, 4),
                     span(global_scale, 4)};
  const Span out[] = {span(codes, h3q_code_bytes(m, f)), span(scales, h3q_scale_bytes(m, f)),
                      y ? span(y, m * f * 2) : Span{0, 0}, acc ? span(acc, m * n * 4) : Span{0, 0}};
  for (int i = 0; i < 4; ++i) {
    for (const Span& x : in)
      if (overlap(out[i], x)) return invalid(fn, "outputs overlap an input");
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return invalid(fn, "outputs overlap each other");
  }
  cudaError_t err = h3q::launch_gemm_swiglu(a_codes, a_scales, m, k, b_codes, b_scales, n, alpha, global_scale,
                                            codes, scales, static_cast<uint16_t*>(y), acc,
                                            static_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? H3Q_OK : cuda_failed(fn, err);
}

int h3q_kernel_error_flag(int* flag) {
  static const char* fn = "h3q_kernel_error_flag";
  g_last_error.clear();
  if (flag == nullptr) return invalid(fn, "flag must not be NULL");
  int gemm = 0, cache = 0, attention = 0, blocks = 0;
  // (the copies below wait for the legacy default stream alone, which streams made non-blocking do not join)
  cudaError_t err = cudaDeviceSynchronize();
  if (err == cudaSuccess) err = h3q::gemm_error_flag(&gemm);
  if (err == cudaSuccess) err = h3q::cache_attention_error_flag(&cache);
  if (err == cudaSuccess) err = h3q::attention_error_flag(&attention);
  if (err == cudaSuccess) err = h3q::attention_blocks_error_flag(&blocks);
  *flag = gemm | cache | attention | blocks;
  return err == cudaSuccess ? H3Q_OK : cuda_failed(fn, err);
}

int h3q_swiglu_packed_nvfp4(const void* o, int64_t ld_o, const void* bias, int64_t rows,
                            int64_t f, const float* global_scale, uint8_t* codes, uint8_t* scales,
                            void* stream) {
  static const char* fn = "h3q_swiglu_packed_nvfp4";
  g_last_error.clear();
  if (int e = check_shape(fn, rows, f)) return e;
  if (rows == 0) return H3Q_OK;
  if (int e = check_input(fn, "o", o, ld_o, rows, 2 * f)) return e;
  if (bias != nullptr)
    if (int e = check_input(fn, "bias", bias, 2 * f, 1, 2 * f)) return e;
  if (int e = check_outputs(fn, codes, scales, global_scale)) return e;
  const Span in = span(o, view_bytes(rows, 2 * f, ld_o));
  const Span b = bias ? span(bias, 4 * f) : Span{0, 0};
  const Span c = span(codes, h3q_code_bytes(rows, f));
  const Span s = span(scales, h3q_scale_bytes(rows, f));
  if (overlap(in, c) || overlap(in, s) || overlap(b, c) || overlap(b, s) || overlap(c, s))
    return invalid(fn, "outputs overlap an input or each other");
  cudaError_t err = h3q::launch_swiglu_packed(static_cast<const uint16_t*>(o), ld_o,
                                              static_cast<const uint16_t*>(bias), rows, f,
                                              global_scale, codes, scales,
                                              static_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? H3Q_OK : cuda_failed(fn, err);
}

int h3q_dequantize_nvfp4(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols,
                         const float* global_scale, float* out, void* stream) {
  static const char* fn = "h3q_dequantize_nvfp4";
  g_last_error.clear();
  if (int e = check_shape(fn, rows, cols)) return e;
  if (rows == 0) return H3Q_OK;
  if (codes == nullptr || scales == nullptr || out == nullptr)
    return invalid(fn, "codes, scales and out must not be NULL");
  if (!aligned(codes, 16) || !aligned(scales, 16)) return invalid(fn, "codes and scales must be 16-byte aligned");
  if (!aligned(out, 32)) return invalid(fn, "out must be 32-byte aligned");
  if (global_scale == nullptr || !aligned(global_scale, 4))
    return invalid(fn, "global_scale must be a 4-byte aligned pointer");
  const Span o = span(out, rows * cols * 4);
  if (overlap(o, span(codes, h3q_code_bytes(rows, cols))) ||
      overlap(o, span(scales, h3q_scale_bytes(rows, cols))))
    return invalid(fn, "out overlaps an input");
  cudaError_t err = h3q::launch_dequantize(codes, scales, rows, cols, global_scale, out,
                                           static_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? H3Q_OK : cuda_failed(fn, err);
}

int h3q_qkv_epilogue(const void* q, int64_t ld_q, const void* k, int64_t ld_k, const void* v,
                     int64_t ld_v, const void* bias_q, const void* bias_k, const void* bias_v,
                     const void* cos, const void* sin, int64_t rot, int interleaved, int64_t rows,
                     int64_t heads, int64_t head_dim, float eps, void* q_out, void* k_out,
                     void* v_out, void* stream) {
  static const char* fn = "h3q_qkv_epilogue";
  g_last_error.clear();
  if (rows < 0) return invalid(fn, "rows must be >= 0");
  if (rows > kMaxRows) return invalid(fn, "rows exceeds 2^40");
  if (heads < 1) return invalid(fn, "heads must be >= 1");
  if (head_dim != 64 && head_dim != 128 && head_dim != 256)
    return invalid(fn, "head_dim must be 64, 128 or 256");
  if (heads > kMaxCols / head_dim) return invalid(fn, "heads * head_dim exceeds 2^24");
  if (rot < 0 || rot > head_dim || rot % 16 != 0)
    return invalid(fn, "rot must be a multiple of 16 in [0, head_dim]");
  if (interleaved != 0 && interleaved != 1) return invalid(fn, "interleaved must be 0 or 1");
  if (!std::isfinite(eps) || eps < 0.0f) return invalid(fn, "eps must be finite and >= 0");
  if (rows == 0) return H3Q_OK;
  const int64_t d = heads * head_dim;
  const void* xs[3] = {q, k, v};
  const int64_t lds[3] = {ld_q, ld_k, ld_v};
  const void* bs[3] = {bias_q, bias_k, bias_v};
  void* outs[3] = {q_out, k_out, v_out};
  static const char* xn[3] = {"q", "k", "v"};
  static const char* bn[3] = {"bias_q", "bias_k", "bias_v"};
  for (int i = 0; i < 3; ++i) {
    if (int e = check_input(fn, xn[i], xs[i], lds[i], rows, d)) return e;
    if (int e = check_input(fn, bn[i], bs[i], d, 1, d)) return e;
    if (outs[i] == nullptr || !aligned(outs[i], 16))
      return invalid(fn, "q_out, k_out and v_out must be 16-byte aligned and not NULL");
  }
  if (rot > 0) {
    if (cos == nullptr || sin == nullptr) return invalid(fn, "cos and sin must not be NULL when rot > 0");
    if (!aligned(cos, 16) || !aligned(sin, 16)) return invalid(fn, "cos and sin must be 16-byte aligned");
  }
  Span ins[8];
  int n_in = 0;
  for (int i = 0; i < 3; ++i) {
    ins[n_in++] = span(xs[i], view_bytes(rows, d, lds[i]));
    ins[n_in++] = span(bs[i], d * 2);
  }
  if (rot > 0) {
    ins[n_in++] = span(cos, rows * rot * 2);
    ins[n_in++] = span(sin, rows * rot * 2);
  }
  Span os[3];
  for (int i = 0; i < 3; ++i) os[i] = span(outs[i], rows * d * 2);
  for (int i = 0; i < 3; ++i) {
    for (int j = 0; j < n_in; ++j)
      if (overlap(os[i], ins[j])) return invalid(fn, "outputs overlap an input or each other");
    for (int j = i + 1; j < 3; ++j)
      if (overlap(os[i], os[j])) return invalid(fn, "outputs overlap an input or each other");
  }
  const uint16_t* x16[3];
  const uint16_t* b16[3];
  uint16_t* o16[3];
  for (int i = 0; i < 3; ++i) {
    x16[i] = static_cast<const uint16_t*>(xs[i]);
    b16[i] = static_cast<const uint16_t*>(bs[i]);
    o16[i] = static_cast<uint16_t*>(outs[i]);
  }
  cudaError_t err = h3q::launch_qkv_epilogue(
      x16, lds, b16, o16, static_cast<const uint16_t*>(cos), static_cast<const uint16_t*>(sin), rot,
      interleaved, rows, heads, head_dim, eps, static_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? H3Q_OK : cuda_failed(fn, err);
}

int h3q_rmsnorm_adaln_nvfp4_host(const void* x_host, int64_t rows, int64_t cols, const void* gamma,
                                 const void* mod_table, int64_t num_frames, const int32_t* row_frame,
                                 int64_t rows_per_frame, float eps, const float* global_scale,
                                 uint8_t* codes_host, uint8_t* scales_host, void* workspace,
                                 int64_t workspace_bytes, int64_t chunk_rows, void* stream) {
  static const char* fn = "h3q_rmsnorm_adaln_nvfp4_host";
  g_last_error.clear();
  if (int e = check_shape(fn, rows, cols)) return e;
  if (!std::isfinite(eps) || eps < 0.0f) return invalid(fn, "eps must be finite and >= 0");
  if (num_frames < 1) return invalid(fn, "num_frames must be >= 1");
  if (num_frames > (int64_t(1) << 31)) return invalid(fn, "num_frames exceeds 2^31");
  if (chunk_rows <= 0 || chunk_rows % 128 != 0) return invalid(fn, "chunk_rows must be a positive multiple of 128");
  if (chunk_rows > (int64_t(1) << 40) / cols) return invalid(fn, "chunk_rows * cols is too large");
  if (rows == 0) return H3Q_OK;
  if (x_host == nullptr || codes_host == nullptr || scales_host == nullptr)
    return invalid(fn, "x_host, codes_host and scales_host must not be NULL");
  if (int e = check_input(fn, "gamma", gamma, cols, 1, cols)) return e;
  if (int e = check_input(fn, "mod_table", mod_table, cols, 2 * num_frames, cols)) return e;
  if (global_scale == nullptr || !aligned(global_scale, 4))
    return invalid(fn, "global_scale must be a 4-byte aligned pointer");
  if (row_frame != nullptr) {
    if (!aligned(row_frame, 4)) return invalid(fn, "row_frame must be 4-byte aligned");
  } else {
    if (rows_per_frame < 1) return invalid(fn, "rows_per_frame must be >= 1 when row_frame is NULL");
    if ((rows - 1) / rows_per_frame >= num_frames)
      return invalid(fn, "rows / rows_per_frame reaches past the modulation table");
  }
  if (workspace == nullptr || !aligned(workspace, 256)) return invalid(fn, "workspace must be 256-byte aligned");
  if (workspace_bytes < h3q_host_workspace_bytes(chunk_rows, cols, rows, row_frame == nullptr))
    return invalid(fn, "workspace_bytes is below h3q_host_workspace_bytes");
  const Span xs = span(x_host, rows * cols * 2);
  const Span c = span(codes_host, h3q_code_bytes(rows, cols));
  const Span s = span(scales_host, h3q_scale_bytes(rows, cols));
  if (overlap(xs, c) || overlap(xs, s) || overlap(c, s))
    return invalid(fn, "host outputs overlap the input or each other");
  const Span ws = span(workspace, workspace_bytes);
  const Span dev_ins[4] = {span(gamma, cols * 2), span(mod_table, num_frames * 4 * cols),
                           span(global_scale, 4), row_frame ? span(row_frame, rows * 4) : Span{0, 0}};
  for (const Span& in : dev_ins)
    if (overlap(in, ws)) return invalid(fn, "workspace overlaps a device input");
  cudaError_t err = h3q::launch_adaln_host(
      static_cast<const uint16_t*>(x_host), rows, cols, static_cast<const uint16_t*>(gamma),
      static_cast<const uint16_t*>(mod_table), num_frames, row_frame, rows_per_frame, eps, global_scale,
      codes_host, scales_host, static_cast<uint8_t*>(workspace), chunk_rows,
      static_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? H3Q_OK : cuda_failed(fn, err);
}

// --- the paged NVFP4 cache ---------------------------------------------------

namespace {

struct CacheShape {
  uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
  int64_t num_pages, page_size, kv_heads, head_dim;
  Span spans[4];
};

int check_cache(const char* fn, CacheShape& c) {
  if (c.head_dim != 64 && c.head_dim != 128 && c.head_dim != 256)
    return invalid(fn, "head_dim must be 64, 128 or 256");
  if (c.kv_heads < 1) return invalid(fn, "kv_heads must be >= 1");
  if (c.kv_heads > kMaxCols / c.head_dim) return invalid(fn, "kv_heads * head_dim exceeds 2^24");
  if (c.page_size != 16 && c.page_size != 32 && c.page_size != 64 && c.page_size != 128)
    return invalid(fn, "page_size must be 16, 32, 64 or 128");
  if (c.num_pages < 1 || c.num_pages >= (int64_t(1) << 31)) return invalid(fn, "num_pages must be in [1, 2^31)");
  return 0;
}

int check_cache_buffers(const char* fn, CacheShape& c) {
  const uint8_t* p[4] = {c.k_codes, c.k_scales, c.v_codes, c.v_scales};
  const int64_t rows = c.num_pages * c.page_size * c.kv_heads;
  for (int i = 0; i < 4; ++i) {
    if (p[i] == nullptr || !aligned(p[i], 16))
      return invalid(fn, "k_codes, k_scales, v_codes and v_scales must be 16-byte aligned and not NULL");
    c.spans[i] = span(p[i], rows * (c.head_dim / (i % 2 == 0 ? 2 : 16)));
  }
  return 0;
}

int check_lists(const char* fn, const int32_t* cu_rows, const int32_t* kv_len, const int32_t* block_table,
                int64_t batch, int64_t max_pages) {
  if (batch < 0 || batch > kMaxBatch) return invalid(fn, "batch must be in [0, 2^24]");
  if (max_pages < 1) return invalid(fn, "max_pages must be >= 1");
  if (batch > 0 && max_pages > (int64_t(1) << 40) / batch) return invalid(fn, "batch * max_pages exceeds 2^40");
  if (batch == 0) return 0;
  if (cu_rows == nullptr || kv_len == nullptr || block_table == nullptr)
    return invalid(fn, "cu_rows, kv_len and block_table must not be NULL");
  if (!aligned(cu_rows, 4) || !aligned(kv_len, 4) || !aligned(block_table, 4))
    return invalid(fn, "cu_rows, kv_len and block_table must be 4-byte aligned");
  return 0;
}

int check_scales(const char* fn, const float* k_gsf, const float* v_gsf) {
  if (k_gsf == nullptr || v_gsf == nullptr || !aligned(k_gsf, 4) || !aligned(v_gsf, 4))
    return invalid(fn, "k_global_scale and v_global_scale must be 4-byte aligned pointers");
  return 0;
}

// The page of a position is found by a shift.
int page_shift(int64_t page_size) { return page_size == 16 ? 4 : page_size == 32 ? 5 : page_size == 64 ? 6 : 7; }

h3q::PagedCache paged_cache(const CacheShape& c) {
  h3q::PagedCache p{};
  p.codes[0] = c.k_codes;
  p.codes[1] = c.v_codes;
  p.scales[0] = c.k_scales;
  p.scales[1] = c.v_scales;
  p.num_pages = c.num_pages;
  p.kv_heads = static_cast<int>(c.kv_heads);
  p.head_dim = static_cast<int>(c.head_dim);
  p.page_shift = page_shift(c.page_size);
  return p;
}

}  // namespace

int h3q_kv_cache_write_nvfp4(const void* k, int64_t ld_k, const void* v, int64_t ld_v, int64_t rows,
                             const int32_t* cu_rows, const int32_t* kv_len, const int32_t* block_table,
                             int64_t batch, int64_t max_pages, const float* k_global_scale,
                             const float* v_global_scale, uint8_t* k_codes, uint8_t* k_scales,
                             uint8_t* v_codes, uint8_t* v_scales, int64_t num_pages, int64_t page_size,
                             int64_t kv_heads, int64_t head_dim, void* stream) {
  static const char* fn = "h3q_kv_cache_write_nvfp4";
  g_last_error.clear();
  CacheShape c{k_codes, k_scales, v_codes, v_scales, num_pages, page_size, kv_heads, head_dim, {}};
  if (int e = check_cache(fn, c)) return e;
  if (rows < 0) return invalid(fn, "rows must be >= 0");
  if (rows > kMaxRows) return invalid(fn, "rows exceeds 2^40");
  if (int e = check_lists(fn, cu_rows, kv_len, block_table, batch, max_pages)) return e;
  if (rows == 0 || batch == 0) return H3Q_OK;
  const int64_t d = kv_heads * head_dim;
  if (int e = check_input(fn, "k", k, ld_k, rows, d)) return e;
  if (int e = check_input(fn, "v", v, ld_v, rows, d)) return e;
  if (int e = check_cache_buffers(fn, c)) return e;
  if (int e = check_scales(fn, k_global_scale, v_global_scale)) return e;
  const Span ins[] = {span(k, view_bytes(rows, d, ld_k)), span(v, view_bytes(rows, d, ld_v)),
                      span(cu_rows, (batch + 1) * 4), span(kv_len, batch * 4),
                      span(block_table, batch * max_pages * 4), span(k_global_scale, 4), span(v_global_scale, 4)};
  for (int i = 0; i < 4; ++i) {
    for (const Span& in : ins)
      if (overlap(c.spans[i], in)) return invalid(fn, "the cache overlaps an input");
    for (int j = 0; j < i; ++j)
      if (overlap(c.spans[i], c.spans[j])) return invalid(fn, "the cache's buffers overlap each other");
  }
  const uint16_t* x[2] = {static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v)};
  const int64_t ld[2] = {ld_k, ld_v};
  const float* gsf[2] = {k_global_scale, v_global_scale};
  const h3q::PagedRows at{cu_rows, kv_len, block_table, max_pages, static_cast<int>(batch)};
  cudaError_t err = h3q::launch_cache_write(paged_cache(c), at, x, ld, gsf, rows, static_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? H3Q_OK : cuda_failed(fn, err);
}

int h3q_kv_cache_read_nvfp4(const uint8_t* k_codes, const uint8_t* k_scales, const uint8_t* v_codes,
                            const uint8_t* v_scales, int64_t num_pages, int64_t page_size,
                            int64_t kv_heads, int64_t head_dim, const float* k_global_scale,
                            const float* v_global_scale, int64_t rows, const int32_t* cu_rows,
                            const int32_t* kv_len, const int32_t* block_table, int64_t batch,
                            int64_t max_pages, void* k_out, void* v_out, void* stream) {
  static const char* fn = "h3q_kv_cache_read_nvfp4";
  g_last_error.clear();
  CacheShape c{const_cast<uint8_t*>(k_codes), const_cast<uint8_t*>(k_scales), const_cast<uint8_t*>(v_codes),
               const_cast<uint8_t*>(v_scales), num_pages, page_size, kv_heads, head_dim, {}};
  if (int e = check_cache(fn, c)) return e;
  if (rows < 0) return invalid(fn, "rows must be >= 0");
  if (rows > kMaxRows) return invalid(fn, "rows exceeds 2^40");
  if (int e = check_lists(fn, cu_rows, kv_len, block_table, batch, max_pages)) return e;
  if (rows == 0 || batch == 0) return H3Q_OK;
  if (int e = check_cache_buffers(fn, c)) return e;
  if (int e = check_scales(fn, k_global_scale, v_global_scale)) return e;
  if (k_out == nullptr || v_out == nullptr || !aligned(k_out, 32) || !aligned(v_out, 32))
    return invalid(fn, "k_out and v_out must be 32-byte aligned and not NULL");
  const int64_t bytes = rows * kv_heads * head_dim * 2;
  const Span outs[2] = {span(k_out, bytes), span(v_out, bytes)};
  const Span ins[] = {c.spans[0], c.spans[1], c.spans[2], c.spans[3], span(cu_rows, (batch + 1) * 4),
                      span(kv_len, batch * 4), span(block_table, batch * max_pages * 4),
                      span(k_global_scale, 4), span(v_global_scale, 4)};
  for (const Span& o : outs)
    for (const Span& in : ins)
      if (overlap(o, in)) return invalid(fn, "an output overlaps an input");
  if (overlap(outs[0], outs[1])) return invalid(fn, "k_out and v_out overlap");
  uint16_t* out[2] = {static_cast<uint16_t*>(k_out), static_cast<uint16_t*>(v_out)};
  const float* gsf[2] = {k_global_scale, v_global_scale};
  const h3q::PagedRows at{cu_rows, kv_len, block_table, max_pages, static_cast<int>(batch)};
  cudaError_t err = h3q::launch_cache_read(paged_cache(c), at, out, gsf, rows, static_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? H3Q_OK : cuda_failed(fn, err);
}

int h3q_attention_varlen(const void* q, int64_t ld_q, const void* k, int64_t ld_k, const void* v, int64_t ld_v,
                         const int32_t* cu_q, const int32_t* cu_k, int64_t batch, int64_t rows_q, int64_t rows_k,
                         int64_t heads, int64_t kv_heads, int64_t head_dim, int causal, float scale, void* o,
                         float* lse, void* stream) {
  static const char* fn = "h3q_attention_varlen";
  g_last_error.clear();
  constexpr int64_t kMaxPacked = (int64_t(1) << 31) - 512;   // tensor-copy coordinates are 32-bit
  constexpr int64_t kMaxKeys = int64_t(1) << 25;   // a unit of work stays far inside the kernel's bounded waits
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return invalid(fn, "head_dim must be 64, 128 or 256");
  if (kv_heads < 1) return invalid(fn, "kv_heads must be >= 1");
  if (heads < 1 || heads % kv_heads != 0) return invalid(fn, "heads must be a positive multiple of kv_heads");
  if (heads > kMaxCols / head_dim) return invalid(fn, "heads * head_dim exceeds 2^24");
  if (rows_q < 0 || rows_q > kMaxPacked) return invalid(fn, "rows_q must be in [0, 2^31 - 512]");
  if (rows_k < 0 || rows_k > kMaxKeys) return invalid(fn, "rows_k must be in [0, 2^25]");
  if (batch < 0 || batch > kMaxBatch) return invalid(fn, "batch must be in [0, 2^24]");
  if (causal != 0 && causal != 1) return invalid(fn, "causal must be 0 or 1");
  if (!std::isfinite(scale) || !(scale > 0.0f)) return invalid(fn, "scale must be finite and > 0");
  if (rows_q == 0 || batch == 0) return H3Q_OK;
  const int64_t dq = heads * head_dim, dk = kv_heads * head_dim;
  if (int e = check_input(fn, "q", q, ld_q, rows_q, dq)) return e;
  if (rows_k > 0) {
    if (int e = check_input(fn, "k", k, ld_k, rows_k, dk)) return e;
    if (int e = check_input(fn, "v", v, ld_v, rows_k, dk)) return e;
  }
  if (cu_q == nullptr || cu_k == nullptr || !aligned(cu_q, 4) || !aligned(cu_k, 4))
    return invalid(fn, "cu_q and cu_k must be 4-byte aligned and not NULL");
  if (o == nullptr || !aligned(o, 16)) return invalid(fn, "o must be 16-byte aligned and not NULL");
  if (lse != nullptr && !aligned(lse, 4)) return invalid(fn, "lse must be 4-byte aligned");
  const Span outs[2] = {span(o, rows_q * dq * 2), lse ? span(lse, heads * rows_q * 4) : Span{0, 0}};
  const Span ins[] = {span(q, view_bytes(rows_q, dq, ld_q)),
                      rows_k > 0 ? span(k, view_bytes(rows_k, dk, ld_k)) : Span{0, 0},
                      rows_k > 0 ? span(v, view_bytes(rows_k, dk, ld_v)) : Span{0, 0},
                      span(cu_q, (batch + 1) * 4), span(cu_k, (batch + 1) * 4)};
  for (const Span& out : outs)
    for (const Span& in : ins)
      if (overlap(out, in)) return invalid(fn, "an output overlaps an input");
  if (overlap(outs[0], outs[1])) return invalid(fn, "o and lse overlap");
  cudaError_t err = h3q::launch_attention(
      static_cast<const uint16_t*>(q), ld_q, static_cast<const uint16_t*>(k), ld_k, static_cast<const uint16_t*>(v),
      ld_v, cu_q, cu_k, static_cast<int>(batch), rows_q, rows_k, static_cast<int>(heads), static_cast<int>(kv_heads),
      static_cast<int>(head_dim), causal, scale, static_cast<uint16_t*>(o), lse, static_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? H3Q_OK : cuda_failed(fn, err);
}

int h3q_attention_cache_nvfp4(const void* q, int64_t ld_q, int64_t rows, int64_t heads, int64_t max_rows,
                              const int32_t* cu_rows, const int32_t* kv_len, const int32_t* block_table,
                              int64_t batch, int64_t max_pages, const int64_t* tree_mask, const uint8_t* k_codes,
                              const uint8_t* k_scales, const uint8_t* v_codes, const uint8_t* v_scales,
                              int64_t num_pages, int64_t page_size, int64_t kv_heads, int64_t head_dim,
                              const float* k_global_scale, const float* v_global_scale, float scale, void* o,
                              float* lse, void* workspace, int64_t workspace_bytes, void* stream) {
  static const char* fn = "h3q_attention_cache_nvfp4";
  g_last_error.clear();
  CacheShape c{const_cast<uint8_t*>(k_codes), const_cast<uint8_t*>(k_scales), const_cast<uint8_t*>(v_codes),
               const_cast<uint8_t*>(v_scales), num_pages, page_size, kv_heads, head_dim, {}};
  if (int e = check_cache(fn, c)) return e;
  if (rows < 0) return invalid(fn, "rows must be >= 0");
  if (rows > kMaxRows) return invalid(fn, "rows exceeds 2^40");
  if (heads < 1 || heads % kv_heads != 0) return invalid(fn, "heads must be a positive multiple of kv_heads");
  if (heads > kMaxCols / head_dim) return invalid(fn, "heads * head_dim exceeds 2^24");
  if (max_rows < 1 || max_rows > 64) return invalid(fn, "max_rows must be in [1, 64]");
  if (!std::isfinite(scale) || !(scale > 0.0f)) return invalid(fn, "scale must be finite and > 0");
  if (int e = check_lists(fn, cu_rows, kv_len, block_table, batch, max_pages)) return e;
  if (rows == 0 || batch == 0) return H3Q_OK;
  const int64_t d = heads * head_dim;
  if (int e = check_input(fn, "q", q, ld_q, rows, d)) return e;
  if (int e = check_cache_buffers(fn, c)) return e;
  if (int e = check_scales(fn, k_global_scale, v_global_scale)) return e;
  if (tree_mask != nullptr && !aligned(tree_mask, 8)) return invalid(fn, "tree_mask must be 8-byte aligned");
  if (o == nullptr || !aligned(o, 16)) return invalid(fn, "o must be 16-byte aligned and not NULL");
  if (lse != nullptr && !aligned(lse, 4)) return invalid(fn, "lse must be 4-byte aligned");
  if (workspace == nullptr || !aligned(workspace, 256)) return invalid(fn, "workspace must be 256-byte aligned");
  if (workspace_bytes < h3q_attention_cache_workspace_bytes(max_rows, heads, kv_heads, head_dim))
    return invalid(fn, "workspace_bytes is below h3q_attention_cache_workspace_bytes");
  const Span outs[3] = {span(o, rows * d * 2), lse ? span(lse, heads * rows * 4) : Span{0, 0},
                        span(workspace, workspace_bytes)};
  const Span ins[] = {span(q, view_bytes(rows, d, ld_q)), c.spans[0], c.spans[1], c.spans[2], c.spans[3],
                      span(cu_rows, (batch + 1) * 4), span(kv_len, batch * 4),
                      span(block_table, batch * max_pages * 4), span(k_global_scale, 4), span(v_global_scale, 4),
                      tree_mask ? span(tree_mask, rows * 8) : Span{0, 0}};
  for (int i = 0; i < 3; ++i) {
    for (const Span& in : ins)
      if (overlap(outs[i], in)) return invalid(fn, "an output or the workspace overlaps an input");
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i], outs[j])) return invalid(fn, "outputs and workspace overlap each other");
  }
  const h3q::PagedRows at{cu_rows, kv_len, block_table, max_pages, static_cast<int>(batch)};
  cudaError_t err = h3q::launch_cache_attention(
      paged_cache(c), at, static_cast<const uint16_t*>(q), ld_q, rows, static_cast<int>(heads),
      static_cast<int>(max_rows), tree_mask, k_global_scale, v_global_scale, scale, static_cast<uint16_t*>(o), lse,
      static_cast<uint8_t*>(workspace), static_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? H3Q_OK : cuda_failed(fn, err);
}

// --- rotary positions with several axes, norms around a block, attention over blocks --

int h3q_qkv_epilogue_axes(const void* q, int64_t ld_q, const void* k, int64_t ld_k, const void* v, int64_t ld_v,
                          const void* bias_q, const void* bias_k, const void* bias_v, const void* weight_q,
                          const void* weight_k, const int32_t* positions, int64_t axes, const int64_t* axis_dims,
                          const double* theta, const double* scale, int sections, int interleaved, int norm,
                          int64_t rows, int64_t heads, int64_t kv_heads, int64_t head_dim, float eps, void* q_out,
                          void* k_out, void* v_out, void* stream) {
  static const char* fn = "h3q_qkv_epilogue_axes";
  g_last_error.clear();
  if (rows < 0) return invalid(fn, "rows must be >= 0");
  if (rows > kMaxRows) return invalid(fn, "rows exceeds 2^40");
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return invalid(fn, "head_dim must be 64, 128 or 256");
  if (kv_heads < 1) return invalid(fn, "kv_heads must be >= 1");
  if (heads < 1 || heads % kv_heads != 0) return invalid(fn, "heads must be a positive multiple of kv_heads");
  if (heads > kMaxCols / head_dim) return invalid(fn, "heads * head_dim exceeds 2^24");
  if (axes < 1 || axes > 4) return invalid(fn, "axes must be in [1, 4]");
  if (axis_dims == nullptr || theta == nullptr || scale == nullptr)
    return invalid(fn, "axis_dims, theta and scale must not be NULL");
  int64_t rot = 0;
  for (int64_t i = 0; i < axes; ++i) {
    if (axis_dims[i] < 2 || axis_dims[i] % 2 != 0 || axis_dims[i] > head_dim)
      return invalid(fn, "axis_dims must be positive, even and at most head_dim");
    if (!std::isfinite(theta[i]) || !(theta[i] > 0.0)) return invalid(fn, "theta must be finite and > 0");
    if (!std::isfinite(scale[i])) return invalid(fn, "scale must be finite");
    rot += axis_dims[i];
  }
  if (rot % 16 != 0 || rot > head_dim)
    return invalid(fn, "the sum of axis_dims must be a multiple of 16 and at most head_dim");
  for (int flag : {sections, interleaved, norm})
    if (flag != 0 && flag != 1) return invalid(fn, "sections, interleaved and norm must be 0 or 1");
  if (!norm && (weight_q != nullptr || weight_k != nullptr)) return invalid(fn, "weights need the norm");
  if (!std::isfinite(eps) || eps < 0.0f) return invalid(fn, "eps must be finite and >= 0");
  h3q::RopeTurns turns{};
  int64_t j = 0;
  for (int64_t i = 0; i < axes; ++i) {
    // theta^(-2 p / d) as a power of two (half of pow's time, which is a tenth of a small call's)
    const double step = -2.0 * std::log2(theta[sections ? 0 : i]) / static_cast<double>(sections ? rot : axis_dims[i]);
    for (int64_t p = 0; p < axis_dims[i] / 2; ++p, ++j) {
      const double f = scale[i] * std::exp2(step * static_cast<double>(sections ? j : p));
      constexpr double kTurn = 6.283185307179586476925;
      const double t = f / kTurn;
      if (!std::isfinite(t)) return invalid(fn, "theta and scale give a frequency that is not finite");
      const double part = t - std::floor(t);   // of a turn, in [0, 1]
      turns.of_pair[j] = part >= 1.0 ? 0ull : static_cast<unsigned long long>(std::ldexp(part, 64));
      turns.axis[j] = static_cast<uint8_t>(i);
    }
  }
  if (rows == 0) return H3Q_OK;
  const void* xs[3] = {q, k, v};
  const int64_t lds[3] = {ld_q, ld_k, ld_v};
  const int64_t ds[3] = {heads * head_dim, kv_heads * head_dim, kv_heads * head_dim};
  const void* bs[3] = {bias_q, bias_k, bias_v};
  const void* ws[2] = {weight_q, weight_k};
  void* outs[3] = {q_out, k_out, v_out};
  static const char* xn[3] = {"q", "k", "v"};
  static const char* bn[3] = {"bias_q", "bias_k", "bias_v"};
  static const char* wn[2] = {"weight_q", "weight_k"};
  Span ins[9], os[3];
  int n_in = 0;
  for (int i = 0; i < 3; ++i) {
    if (int e = check_input(fn, xn[i], xs[i], lds[i], rows, ds[i])) return e;
    ins[n_in++] = span(xs[i], view_bytes(rows, ds[i], lds[i]));
    if (bs[i] != nullptr) {
      if (int e = check_input(fn, bn[i], bs[i], ds[i], 1, ds[i])) return e;
      ins[n_in++] = span(bs[i], ds[i] * 2);
    }
    if (i < 2 && ws[i] != nullptr) {
      if (int e = check_input(fn, wn[i], ws[i], head_dim, 1, head_dim)) return e;
      ins[n_in++] = span(ws[i], head_dim * 2);
    }
    if (outs[i] == nullptr || !aligned(outs[i], 16))
      return invalid(fn, "q_out, k_out and v_out must be 16-byte aligned and not NULL");
    os[i] = span(outs[i], rows * ds[i] * 2);
  }
  if (positions == nullptr || !aligned(positions, 4))
    return invalid(fn, "positions must be 4-byte aligned and not NULL");
  ins[n_in++] = span(positions, rows * axes * 4);
  for (int i = 0; i < 3; ++i) {
    for (int m = 0; m < n_in; ++m)
      if (overlap(os[i], ins[m])) return invalid(fn, "outputs overlap an input or each other");
    for (int m = i + 1; m < 3; ++m)
      if (overlap(os[i], os[m])) return invalid(fn, "outputs overlap an input or each other");
  }
  const uint16_t* x16[3];
  const uint16_t* b16[3];
  uint16_t* o16[3];
  for (int i = 0; i < 3; ++i) {
    x16[i] = static_cast<const uint16_t*>(xs[i]);
    b16[i] = static_cast<const uint16_t*>(bs[i]);
    o16[i] = static_cast<uint16_t*>(outs[i]);
  }
  const uint16_t* w16[2] = {static_cast<const uint16_t*>(weight_q), static_cast<const uint16_t*>(weight_k)};
  cudaError_t err = h3q::launch_qkv_axes(x16, lds, b16, w16, o16, positions, static_cast<int>(axes), turns,
                                         static_cast<int>(rot), interleaved, norm, rows, static_cast<int>(heads),
                                         static_cast<int>(kv_heads), static_cast<int>(head_dim), eps,
                                         static_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? H3Q_OK : cuda_failed(fn, err);
}

int h3q_postnorm_residual_adaln_nvfp4(float* h, int64_t ld_h, const void* o, int64_t ld_o, const void* bias,
                                      const void* gamma_post, const void* gate_table, float residual_scale,
                                      const void* gamma, const void* mod_table, int64_t num_frames,
                                      const int32_t* row_frame, int64_t rows_per_frame, float eps, int64_t rows,
                                      int64_t cols, const float* global_scale, uint8_t* codes, uint8_t* scales,
                                      float* row_rstd, void* stream) {
  static const char* fn = "h3q_postnorm_residual_adaln_nvfp4";
  g_last_error.clear();
  const bool tables = gate_table != nullptr || mod_table != nullptr;
  if (int e = check_shape(fn, rows, cols)) return e;
  if (cols > 8192) return invalid(fn, "cols exceeds 8,192");
  if (!std::isfinite(eps) || eps < 0.0f) return invalid(fn, "eps must be finite and >= 0");
  if (!std::isfinite(residual_scale)) return invalid(fn, "residual_scale must be finite");
  if (tables) {
    if (num_frames < 1) return invalid(fn, "num_frames must be >= 1");
    if (num_frames > (int64_t(1) << 31)) return invalid(fn, "num_frames exceeds 2^31");
  } else {
    num_frames = 0;
    row_frame = nullptr;
  }
  if (rows == 0) return H3Q_OK;
  if (h == nullptr || !aligned(h, 32)) return invalid(fn, "h must be a 32-byte aligned pointer");
  if (ld_h < cols || ld_h % 8 != 0) return invalid(fn, "ld of h must be >= cols and a multiple of 8");
  if (ld_h > (int64_t(1) << 61) / rows) return invalid(fn, "h: rows * ld overflows");
  if (int e = check_input(fn, "o", o, ld_o, rows, cols)) return e;
  if (bias != nullptr)
    if (int e = check_input(fn, "bias", bias, cols, 1, cols)) return e;
  if (int e = check_input(fn, "gamma_post", gamma_post, cols, 1, cols)) return e;
  if (int e = check_input(fn, "gamma", gamma, cols, 1, cols)) return e;
  if (gate_table != nullptr)
    if (int e = check_input(fn, "gate_table", gate_table, cols, num_frames, cols)) return e;
  if (mod_table != nullptr)
    if (int e = check_input(fn, "mod_table", mod_table, cols, 2 * num_frames, cols)) return e;
  if (int e = check_outputs(fn, codes, scales, global_scale)) return e;
  if (row_frame != nullptr) {
    if (!aligned(row_frame, 4)) return invalid(fn, "row_frame must be 4-byte aligned");
  } else if (tables) {
    if (rows_per_frame < 1) return invalid(fn, "rows_per_frame must be >= 1 when row_frame is NULL");
    if ((rows - 1) / rows_per_frame >= num_frames) return invalid(fn, "rows / rows_per_frame reaches past the tables");
  }
  if (row_rstd != nullptr && !aligned(row_rstd, 4)) return invalid(fn, "row_rstd must be 4-byte aligned");
  const Span none{0, 0};
  const Span outs[4] = {span(h, ((rows - 1) * ld_h + cols) * 4), span(codes, h3q_code_bytes(rows, cols)),
                        span(scales, h3q_scale_bytes(rows, cols)), row_rstd ? span(row_rstd, rows * 4) : none};
  const Span ins[8] = {span(o, view_bytes(rows, cols, ld_o)), bias ? span(bias, cols * 2) : none,
                       span(gamma_post, cols * 2), span(gamma, cols * 2),
                       gate_table ? span(gate_table, num_frames * 2 * cols) : none,
                       mod_table ? span(mod_table, num_frames * 4 * cols) : none,
                       row_frame ? span(row_frame, rows * 4) : none, span(global_scale, 4)};
  for (int i = 0; i < 4; ++i) {
    for (const Span& in : ins)
      if (overlap(outs[i], in)) return invalid(fn, "an output (h, codes, scales, row_rstd) overlaps an input");
    for (int m = i + 1; m < 4; ++m)
      if (overlap(outs[i], outs[m])) return invalid(fn, "outputs overlap each other");
  }
  const h3q::PostnormArgs a{h, ld_h, static_cast<const uint16_t*>(o), ld_o, static_cast<const uint16_t*>(bias),
                            static_cast<const uint16_t*>(gamma_post), static_cast<const uint16_t*>(gate_table),
                            residual_scale, static_cast<const uint16_t*>(gamma),
                            static_cast<const uint16_t*>(mod_table), num_frames, row_frame, rows_per_frame, eps, rows,
                            cols, global_scale, codes, scales, row_rstd};
  cudaError_t err = h3q::launch_postnorm(a, static_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? H3Q_OK : cuda_failed(fn, err);
}

namespace {
constexpr int64_t kMaxPacked = (int64_t(1) << 31) - 512;   // tensor-copy coordinates are 32-bit
constexpr int64_t kMaxKeys = int64_t(1) << 25;
constexpr int64_t kMaxTop = 4096;

// The shapes of the calls that attend over blocks; returns 0 or an error code.
int check_blocks(const char* fn, int64_t batch, int64_t rows_q, int64_t rows_k, int64_t heads, int64_t kv_heads,
                 int64_t head_dim, int64_t block_q, int64_t block_k, int64_t top, int causal) {
  if (head_dim != 64 && head_dim != 128) return invalid(fn, "head_dim must be 64 or 128");
  if (kv_heads < 1) return invalid(fn, "kv_heads must be >= 1");
  if (heads < 1 || heads % kv_heads != 0) return invalid(fn, "heads must be a positive multiple of kv_heads");
  if (heads > kMaxCols / head_dim) return invalid(fn, "heads * head_dim exceeds 2^24");
  if (block_q != 64 && block_q != 128 && block_q != 256) return invalid(fn, "block_q must be 64, 128 or 256");
  if (block_k != 64 && block_k != 128 && block_k != 256) return invalid(fn, "block_k must be 64, 128 or 256");
  if (top < 1 || top > kMaxTop) return invalid(fn, "top must be in [1, 4096]");
  if (rows_q < 0 || rows_q > kMaxPacked) return invalid(fn, "rows_q must be in [0, 2^31 - 512]");
  if (rows_k < 0 || rows_k > kMaxKeys) return invalid(fn, "rows_k must be in [0, 2^25]");
  if (batch < 0 || batch > kMaxBatch) return invalid(fn, "batch must be in [0, 2^24]");
  if (causal != 0 && causal != 1) return invalid(fn, "causal must be 0 or 1");
  return 0;
}

int check_offsets(const char* fn, const int32_t* cu_q, const int32_t* cu_k) {
  if (cu_q == nullptr || cu_k == nullptr || !aligned(cu_q, 4) || !aligned(cu_k, 4))
    return invalid(fn, "cu_q and cu_k must be 4-byte aligned and not NULL");
  return 0;
}

h3q::BlockShape block_shape(const int32_t* cu_q, const int32_t* cu_k, int64_t batch, int64_t rows_q, int64_t rows_k,
                            int64_t heads, int64_t kv_heads, int64_t head_dim, int64_t block_q, int64_t block_k,
                            int64_t top, int causal) {
  return {cu_q, cu_k, static_cast<int>(batch), rows_q, rows_k, static_cast<int>(heads), static_cast<int>(kv_heads),
          static_cast<int>(head_dim), static_cast<int>(block_q), static_cast<int>(block_k), static_cast<int>(top),
          causal};
}
}  // namespace

int h3q_select_blocks(const void* q, int64_t ld_q, const void* k, int64_t ld_k, const int32_t* cu_q,
                      const int32_t* cu_k, int64_t batch, int64_t rows_q, int64_t rows_k, int64_t heads,
                      int64_t kv_heads, int64_t head_dim, int64_t block_q, int64_t block_k, int64_t top, int causal,
                      int64_t first, int32_t* blocks, float* scores, void* workspace, int64_t workspace_bytes,
                      void* stream) {
  static const char* fn = "h3q_select_blocks";
  g_last_error.clear();
  if (int e = check_blocks(fn, batch, rows_q, rows_k, heads, kv_heads, head_dim, block_q, block_k, top, causal)) return e;
  if (first < 0 || first > top) return invalid(fn, "first must be in [0, top]");
  if (causal && top < first + (block_q + block_k - 1) / block_k + 1)
    return invalid(fn, "top leaves no room for the first blocks and the queries' own");
  const int64_t lists = h3q_block_rows(rows_q, batch, block_q);
  if (lists * kv_heads > (int64_t(1) << 31) - 1 || (h3q_block_rows(rows_k, batch, block_k) + lists) * kv_heads >
                                                       (int64_t(1) << 31) - 1)
    return invalid(fn, "too many blocks: batch, rows and kv_heads give 2^31 lists or more");
  if (lists == 0) return H3Q_OK;
  const int64_t dq = heads * head_dim, dk = kv_heads * head_dim;
  if (rows_q > 0)
    if (int e = check_input(fn, "q", q, ld_q, rows_q, dq)) return e;
  if (rows_k > 0)
    if (int e = check_input(fn, "k", k, ld_k, rows_k, dk)) return e;
  if (int e = check_offsets(fn, cu_q, cu_k)) return e;
  if (blocks == nullptr || !aligned(blocks, 4)) return invalid(fn, "blocks must be 4-byte aligned and not NULL");
  if (scores != nullptr && !aligned(scores, 4)) return invalid(fn, "scores must be 4-byte aligned");
  if (workspace == nullptr || !aligned(workspace, 256)) return invalid(fn, "workspace must be 256-byte aligned");
  if (workspace_bytes < h3q_select_blocks_workspace_bytes(rows_q, rows_k, batch, kv_heads, head_dim, block_q, block_k))
    return invalid(fn, rows_k / block_k > h3q::kNearBlocks
                           ? "workspace_bytes is below h3q_select_blocks_workspace_bytes (rows of scores for more than "
                             "16,000 key blocks included)"
                           : "workspace_bytes is below h3q_select_blocks_workspace_bytes");
  const int64_t entries = lists * kv_heads * top;
  const Span outs[3] = {span(blocks, entries * 4), scores ? span(scores, entries * 4) : Span{0, 0},
                        span(workspace, workspace_bytes)};
  const Span ins[] = {rows_q > 0 ? span(q, view_bytes(rows_q, dq, ld_q)) : Span{0, 0},
                      rows_k > 0 ? span(k, view_bytes(rows_k, dk, ld_k)) : Span{0, 0}, span(cu_q, (batch + 1) * 4),
                      span(cu_k, (batch + 1) * 4)};
  for (int i = 0; i < 3; ++i) {
    for (const Span& in : ins)
      if (overlap(outs[i], in)) return invalid(fn, "an output or the workspace overlaps an input");
    for (int m = 0; m < i; ++m)
      if (overlap(outs[i], outs[m])) return invalid(fn, "outputs and workspace overlap each other");
  }
  cudaError_t err = h3q::launch_select_blocks(
      block_shape(cu_q, cu_k, batch, rows_q, rows_k, heads, kv_heads, head_dim, block_q, block_k, top, causal),
      static_cast<const uint16_t*>(q), ld_q, static_cast<const uint16_t*>(k), ld_k, static_cast<int>(first), blocks,
      scores, static_cast<uint8_t*>(workspace), static_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? H3Q_OK : cuda_failed(fn, err);
}

int h3q_attention_blocks(const void* q, int64_t ld_q, const void* k, int64_t ld_k, const void* v, int64_t ld_v,
                         const int32_t* cu_q, const int32_t* cu_k, int64_t batch, int64_t rows_q, int64_t rows_k,
                         int64_t heads, int64_t kv_heads, int64_t head_dim, int64_t block_q, int64_t block_k,
                         const int32_t* blocks, int64_t top, int causal, float scale, void* o, float* lse,
                         void* stream) {
  static const char* fn = "h3q_attention_blocks";
  g_last_error.clear();
  if (int e = check_blocks(fn, batch, rows_q, rows_k, heads, kv_heads, head_dim, block_q, block_k, top, causal)) return e;
  if (!std::isfinite(scale) || !(scale > 0.0f)) return invalid(fn, "scale must be finite and > 0");
  if (rows_q == 0 || batch == 0) return H3Q_OK;
  const h3q::BlockShape shape =
      block_shape(cu_q, cu_k, batch, rows_q, rows_k, heads, kv_heads, head_dim, block_q, block_k, top, causal);
  if (h3q::attention_blocks_units(shape) > (int64_t(1) << 31) - 1)
    return invalid(fn, "too many rows: batch, rows_q and heads give 2^31 pairs of row tiles or more");
  const int64_t dq = heads * head_dim, dk = kv_heads * head_dim;
  if (int e = check_input(fn, "q", q, ld_q, rows_q, dq)) return e;
  if (rows_k > 0) {
    if (int e = check_input(fn, "k", k, ld_k, rows_k, dk)) return e;
    if (int e = check_input(fn, "v", v, ld_v, rows_k, dk)) return e;
  }
  if (int e = check_offsets(fn, cu_q, cu_k)) return e;
  if (blocks == nullptr || !aligned(blocks, 4)) return invalid(fn, "blocks must be 4-byte aligned and not NULL");
  if (o == nullptr || !aligned(o, 16)) return invalid(fn, "o must be 16-byte aligned and not NULL");
  if (lse != nullptr && !aligned(lse, 4)) return invalid(fn, "lse must be 4-byte aligned");
  const Span outs[2] = {span(o, rows_q * dq * 2), lse ? span(lse, heads * rows_q * 4) : Span{0, 0}};
  const Span ins[] = {span(q, view_bytes(rows_q, dq, ld_q)),
                      rows_k > 0 ? span(k, view_bytes(rows_k, dk, ld_k)) : Span{0, 0},
                      rows_k > 0 ? span(v, view_bytes(rows_k, dk, ld_v)) : Span{0, 0},
                      span(cu_q, (batch + 1) * 4), span(cu_k, (batch + 1) * 4),
                      span(blocks, h3q_block_rows(rows_q, batch, block_q) * kv_heads * top * 4)};
  for (const Span& out : outs)
    for (const Span& in : ins)
      if (overlap(out, in)) return invalid(fn, "an output overlaps an input");
  if (overlap(outs[0], outs[1])) return invalid(fn, "o and lse overlap");
  cudaError_t err = h3q::launch_attention_blocks(
      shape, static_cast<const uint16_t*>(q), ld_q, static_cast<const uint16_t*>(k), ld_k, static_cast<const uint16_t*>(v),
      ld_v, blocks, scale, static_cast<uint16_t*>(o), lse, static_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? H3Q_OK : cuda_failed(fn, err);
}

}  // extern "C"
