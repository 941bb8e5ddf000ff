// C-ABI entry points of libfp4.so: host-side argument checks, the gfx950 check
// and dispatch to the kernel launchers.  Nothing here allocates device memory
// or synchronizes.
#include <hip/hip_runtime.h>

#include <atomic>
#include <cstdio>
#include <cstring>

#include "fp4.h"
#include "fp4_internal.h"

namespace {

thread_local char g_last_hip_error[256] = "";

fp4_status hip_fail(hipError_t e, const char* where) {
  std::snprintf(g_last_hip_error, sizeof(g_last_hip_error), "%s: %s", where, hipGetErrorString(e));
  return FP4_ERR_HIP;
}

constexpr int kMaxDevices = 64;
// 0 = unknown, 1 = gfx950, 2 = other architecture
std::atomic<int> g_arch_state[kMaxDevices];

fp4_status check_arch() {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return hip_fail(e, "hipGetDevice");
  if (dev < 0 || dev >= kMaxDevices) return FP4_ERR_ARCH;
  int st = g_arch_state[dev].load(std::memory_order_relaxed);
  if (st == 0) {
    hipDeviceProp_t prop;
    e = hipGetDeviceProperties(&prop, dev);
    if (e != hipSuccess) return hip_fail(e, "hipGetDeviceProperties");
    st = (std::strncmp(prop.gcnArchName, "gfx950", 6) == 0) ? 1 : 2;
    g_arch_state[dev].store(st, std::memory_order_relaxed);
  }
  return st == 1 ? FP4_OK : FP4_ERR_ARCH;
}

bool valid_dtype(fp4_dtype t) { return t == FP4_F32 || t == FP4_BF16; }
bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

#define FP4_TRY_LAUNCH(expr, where)            \
  do {                                         \
    hipError_t _e = (expr);                    \
    if (_e != hipSuccess) return hip_fail(_e, where); \
  } while (0)

// Shared front half of the NVFP4-producing calls.
fp4_status check_quant_args(const void* x, fp4_dtype xt, int64_t rows, int64_t cols,
                            const uint8_t* q, const uint8_t* scales, const float* global_amax,
                            int amax_given, const float* global_scale, const void* workspace,
                            size_t workspace_bytes) {
  if (!valid_dtype(xt)) return FP4_ERR_DTYPE;
  if (rows < 0 || cols < 0) return FP4_ERR_SHAPE;
  if (global_scale == nullptr) return FP4_ERR_NULL;
  if (amax_given && global_amax == nullptr) return FP4_ERR_NULL;
  if (rows == 0 || cols == 0) return FP4_OK;
  if (x == nullptr || q == nullptr || scales == nullptr) return FP4_ERR_NULL;
  if (!amax_given) {
    if (workspace == nullptr || workspace_bytes < FP4_AMAX_WORKSPACE_BYTES) return FP4_ERR_WORKSPACE;
    if (!aligned(workspace, 4)) return FP4_ERR_ALIGN;
  }
  if (!aligned(x, xt == FP4_BF16 ? 2 : 4) || !aligned(global_scale, 4) ||
      (global_amax && !aligned(global_amax, 4)))
    return FP4_ERR_ALIGN;
  return FP4_OK;
}

fp4_status dequantize_blocks(fp4_format fmt, int block, const uint8_t* q,
                                    const uint8_t* scales, const float* global_scale, int64_t rows,
                                    int64_t cols, void* y, fp4_dtype yt, hipStream_t stream) {
  if (fmt != FP4_NVFP4 && fmt != FP4_MXFP4) return FP4_ERR_DTYPE;
  if (!valid_dtype(yt)) return FP4_ERR_DTYPE;
  if (rows < 0 || cols < 0) return FP4_ERR_SHAPE;
  if (fmt == FP4_MXFP4 && global_scale != nullptr) return FP4_ERR_DTYPE;
  if (rows == 0 || cols == 0) return FP4_OK;
  if (q == nullptr || scales == nullptr || y == nullptr) return FP4_ERR_NULL;
  if (fmt == FP4_NVFP4 && global_scale == nullptr) return FP4_ERR_NULL;
  if (!aligned(y, yt == FP4_BF16 ? 2 : 4)) return FP4_ERR_ALIGN;
  fp4_status st = check_arch();
  if (st != FP4_OK) return st;
  FP4_TRY_LAUNCH(fp4impl::launch_dequant(fmt == FP4_MXFP4, q, scales, global_scale, rows, cols, y,
                                         yt == FP4_BF16, stream, block),
                 "fp4_dequantize");
  return FP4_OK;
}

}  // namespace

extern "C" {

const char* fp4_status_string(fp4_status s) {
  switch (s) {
    case FP4_OK: return "ok";
    case FP4_ERR_NULL: return "a required pointer is NULL";
    case FP4_ERR_SHAPE: return "invalid shape";
    case FP4_ERR_DTYPE: return "invalid dtype, format or rounding mode";
    case FP4_ERR_ALIGN: return "pointer misaligned";
    case FP4_ERR_ARCH: return "current device is not gfx950 (MI355X)";
    case FP4_ERR_WORKSPACE: return "workspace missing or too small";
    case FP4_ERR_HIP: return "HIP runtime error";
    case FP4_ERR_ALIAS: return "an output aliases an input it must not alias";
  }
  return "unknown status";
}

const char* fp4_last_hip_error(void) { return g_last_hip_error; }

fp4_status nvfp4_quantize(const void* x, fp4_dtype xt, int64_t rows, int64_t cols, uint8_t* q,
                          uint8_t* scales, float* global_amax, int amax_given, float* global_scale,
                          void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return nvfp4_quantize_ex(x, xt, rows, cols, 16, 0, q, scales, global_amax, amax_given,
                           global_scale, workspace, workspace_bytes, stream);
}

fp4_status nvfp4_quantize_ex(const void* x, fp4_dtype xt, int64_t rows, int64_t cols, int block,
                             int scale_search, uint8_t* q, uint8_t* scales, float* global_amax,
                             int amax_given, float* global_scale, void* workspace,
                             size_t workspace_bytes, hipStream_t stream) {
  if (block != 8 && block != 16 && block != 32) return FP4_ERR_SHAPE;
  if (scale_search < 0 || scale_search > FP4_MAX_SCALE_SEARCH) return FP4_ERR_SHAPE;
  fp4_status st = check_quant_args(x, xt, rows, cols, q, scales, global_amax, amax_given,
                                   global_scale, workspace, workspace_bytes);
  if (st != FP4_OK) return st;
  if ((st = check_arch()) != FP4_OK) return st;
  const bool bf16 = xt == FP4_BF16;
  if (rows == 0 || cols == 0) {
    FP4_TRY_LAUNCH(fp4impl::launch_empty_scales(amax_given ? nullptr : global_amax, global_scale,
                                                stream),
                   "nvfp4_quantize");
    return FP4_OK;
  }
  uint32_t* partials = nullptr;
  int npart = 0;
  if (!amax_given) {
    partials = static_cast<uint32_t*>(workspace);
    FP4_TRY_LAUNCH(fp4impl::launch_amax(x, bf16, rows * cols, partials, &npart, stream),
                   "nvfp4_quantize/amax");
  }
  FP4_TRY_LAUNCH(fp4impl::launch_nv_quant(x, bf16, rows, cols, q, scales,
                                          amax_given ? global_amax : nullptr, partials, npart,
                                          amax_given ? nullptr : global_amax, global_scale, stream,
                                          block, scale_search),
                 "nvfp4_quantize/encode");
  return FP4_OK;
}

fp4_status nvfp4_quantize_no_workspace(const void* x, fp4_dtype xt, int64_t rows, int64_t cols,
                                       uint8_t* q, uint8_t* scales, float* global_amax,
                                       int amax_given, float* global_scale, hipStream_t stream) {
  // the same checks as nvfp4_quantize, with a stand-in for the workspace it
  // does not take (never dereferenced: the library's scratch replaces it)
  fp4_status st = check_quant_args(x, xt, rows, cols, q, scales, global_amax, amax_given,
                                   global_scale, reinterpret_cast<const void*>(FP4_AMAX_WORKSPACE_BYTES),
                                   FP4_AMAX_WORKSPACE_BYTES);
  if (st != FP4_OK) return st;
  if ((st = check_arch()) != FP4_OK) return st;
  const bool bf16 = xt == FP4_BF16;
  if (rows == 0 || cols == 0) {
    FP4_TRY_LAUNCH(fp4impl::launch_empty_scales(amax_given ? nullptr : global_amax, global_scale,
                                                stream),
                   "nvfp4_quantize_no_workspace");
    return FP4_OK;
  }
  uint32_t* partials = nullptr;
  int npart = 0;
  if (!amax_given) {
    FP4_TRY_LAUNCH(fp4impl::amax_scratch(&partials), "nvfp4_quantize_no_workspace/scratch");
    // the amax pass never uses more than kAmaxPartials workgroups, so every
    // size fits the scratch; the first pass writes every partial the second reads
    FP4_TRY_LAUNCH(fp4impl::launch_amax(x, bf16, rows * cols, partials, &npart, stream),
                   "nvfp4_quantize_no_workspace/amax");
  }
  FP4_TRY_LAUNCH(fp4impl::launch_nv_quant(x, bf16, rows, cols, q, scales,
                                          amax_given ? global_amax : nullptr, partials, npart,
                                          amax_given ? nullptr : global_amax, global_scale, stream),
                 "nvfp4_quantize_no_workspace/encode");
  return FP4_OK;
}

fp4_status mxfp4_quantize(const void* x, fp4_dtype xt, int64_t rows, int64_t cols, uint8_t* q,
                          uint8_t* scales, hipStream_t stream) {
  if (!valid_dtype(xt)) return FP4_ERR_DTYPE;
  if (rows < 0 || cols < 0) return FP4_ERR_SHAPE;
  if (rows == 0 || cols == 0) return FP4_OK;
  if (x == nullptr || q == nullptr || scales == nullptr) return FP4_ERR_NULL;
  if (!aligned(x, xt == FP4_BF16 ? 2 : 4)) return FP4_ERR_ALIGN;
  fp4_status st = check_arch();
  if (st != FP4_OK) return st;
  FP4_TRY_LAUNCH(fp4impl::launch_mx_quant(x, xt == FP4_BF16, rows, cols, q, scales, stream),
                 "mxfp4_quantize");
  return FP4_OK;
}

fp4_status fp4_dequantize(fp4_format fmt, const uint8_t* q, const uint8_t* scales,
                          const float* global_scale, int64_t rows, int64_t cols, void* y,
                          fp4_dtype yt, hipStream_t stream) {
  return dequantize_blocks(fmt, 16, q, scales, global_scale, rows, cols, y, yt, stream);
}

fp4_status nvfp4_dequantize_ex(const uint8_t* q, const uint8_t* scales, const float* global_scale,
                               int64_t rows, int64_t cols, int block, void* y, fp4_dtype yt,
                               hipStream_t stream) {
  if (block != 8 && block != 16 && block != 32) return FP4_ERR_SHAPE;
  return dequantize_blocks(FP4_NVFP4, block, q, scales, global_scale, rows, cols, y, yt, stream);
}


fp4_status fp4_scaled_gemm(fp4_format fmt, const uint8_t* A, const uint8_t* a_scales,
                           const float* g_a, const uint8_t* W, const uint8_t* w_scales,
                           const float* g_b, float g_d, int64_t M, int64_t N, int64_t K, void* D,
                           fp4_dtype dt, hipStream_t stream) {
  if (fmt != FP4_NVFP4 && fmt != FP4_MXFP4) return FP4_ERR_DTYPE;
  if (!valid_dtype(dt) && dt != FP4_E4M3) return FP4_ERR_DTYPE;
  const int d_bytes = dt == FP4_F32 ? 4 : dt == FP4_BF16 ? 2 : 1;
  if (M < 0 || N < 0 || K < 0) return FP4_ERR_SHAPE;
  if (K % 32 != 0) return FP4_ERR_SHAPE;
  if (M > FP4_GEMM_MAX_MN || N > FP4_GEMM_MAX_MN || K > FP4_GEMM_MAX_K) return FP4_ERR_SHAPE;
  if (fmt == FP4_MXFP4 && (g_a != nullptr || g_b != nullptr)) return FP4_ERR_DTYPE;
  if (M == 0 || N == 0) return FP4_OK;
  if (K == 0) {   // empty contraction: D = 0, operands are not read
    if (D == nullptr) return FP4_ERR_NULL;
    if (!aligned(D, d_bytes)) return FP4_ERR_ALIGN;
    fp4_status st = check_arch();
    if (st != FP4_OK) return st;
    FP4_TRY_LAUNCH(fp4impl::launch_zero_fill(D, M * N, d_bytes, stream), "fp4_scaled_gemm");
    return FP4_OK;
  }
  if (A == nullptr || a_scales == nullptr || W == nullptr || w_scales == nullptr || D == nullptr)
    return FP4_ERR_NULL;
  if (fmt == FP4_NVFP4 && (g_a == nullptr || g_b == nullptr)) return FP4_ERR_NULL;
  if (!aligned(A, 16) || !aligned(W, 16) || !aligned(D, d_bytes)) return FP4_ERR_ALIGN;
  fp4_status st = check_arch();
  if (st != FP4_OK) return st;
  FP4_TRY_LAUNCH(fp4impl::launch_gemm(fmt == FP4_MXFP4, A, a_scales, g_a, W, w_scales, g_b, g_d, M,
                                      N, K, D, d_bytes, stream),
                 "fp4_scaled_gemm");
  return FP4_OK;
}

fp4_status fp4_scaled_gemm_nvfp4_out(fp4_format fmt, const uint8_t* A, const uint8_t* a_scales,
                                     const float* g_a, const uint8_t* W, const uint8_t* w_scales,
                                     const float* g_b, float g_d, int64_t M, int64_t N, int64_t K,
                                     uint8_t* Dq, uint8_t* d_scales, const float* d_amax,
                                     float* d_global_scale, hipStream_t stream) {
  if (fmt != FP4_NVFP4 && fmt != FP4_MXFP4) return FP4_ERR_DTYPE;
  if (M < 0 || N < 0 || K < 0) return FP4_ERR_SHAPE;
  if (K % 32 != 0) return FP4_ERR_SHAPE;
  if (M > FP4_GEMM_MAX_MN || N > FP4_GEMM_MAX_MN || K > FP4_GEMM_MAX_K) return FP4_ERR_SHAPE;
  if (fmt == FP4_MXFP4 && (g_a != nullptr || g_b != nullptr)) return FP4_ERR_DTYPE;
  if (M == 0 || N == 0) return FP4_OK;
  if (Dq == nullptr || d_scales == nullptr || d_amax == nullptr || d_global_scale == nullptr)
    return FP4_ERR_NULL;
  if (!aligned(d_amax, 4) || !aligned(d_global_scale, 4)) return FP4_ERR_ALIGN;
  // workgroup 0 writes *d_global_scale while the others still read *d_amax
  if (static_cast<const void*>(d_amax) == static_cast<const void*>(d_global_scale))
    return FP4_ERR_ALIAS;
  if (K == 0) {   // empty contraction: D = 0 encodes as codes 0 and scale bytes 0
    fp4_status st = check_arch();
    if (st != FP4_OK) return st;
    FP4_TRY_LAUNCH(fp4impl::launch_zero_fill(Dq, M * ((N + 1) / 2), 1, stream), "fp4_scaled_gemm_nvfp4_out");
    FP4_TRY_LAUNCH(fp4impl::launch_zero_fill(d_scales, M * ((N + 15) / 16), 1, stream),
                   "fp4_scaled_gemm_nvfp4_out");
    FP4_TRY_LAUNCH(fp4impl::launch_nv_global_scale(d_amax, d_global_scale, stream),
                   "fp4_scaled_gemm_nvfp4_out");
    return FP4_OK;
  }
  if (A == nullptr || a_scales == nullptr || W == nullptr || w_scales == nullptr) return FP4_ERR_NULL;
  if (fmt == FP4_NVFP4 && (g_a == nullptr || g_b == nullptr)) return FP4_ERR_NULL;
  if (!aligned(A, 16) || !aligned(W, 16)) return FP4_ERR_ALIGN;
  fp4_status st = check_arch();
  if (st != FP4_OK) return st;
  FP4_TRY_LAUNCH(fp4impl::launch_gemm_nvfp4_out(fmt == FP4_MXFP4, A, a_scales, g_a, W, w_scales, g_b,
                                                g_d, M, N, K, Dq, 0, d_scales, d_amax,
                                                d_global_scale, stream),
                 "fp4_scaled_gemm_nvfp4_out");
  return FP4_OK;
}

fp4_status fp4_grouped_gemm(fp4_format fmt, const uint8_t* A, const uint8_t* a_scales,
                            const float* g_a, const uint8_t* W, const uint8_t* w_scales,
                            const float* g_b, float g_d, int64_t num_groups,
                            const int32_t* offsets, int64_t M_total, int64_t N, int64_t K,
                            void* D, fp4_dtype dt, hipStream_t stream) {
  if (fmt != FP4_NVFP4 && fmt != FP4_MXFP4) return FP4_ERR_DTYPE;
  if (!valid_dtype(dt) && dt != FP4_E4M3) return FP4_ERR_DTYPE;
  const int d_bytes = dt == FP4_F32 ? 4 : dt == FP4_BF16 ? 2 : 1;
  if (num_groups < 1 || M_total < 0 || N < 0 || K < 0 || K % 32 != 0) return FP4_ERR_SHAPE;
  if (M_total > FP4_GEMM_MAX_MN || N > FP4_GEMM_MAX_MN || K > FP4_GEMM_MAX_K ||
      num_groups > FP4_GROUPED_MAX_GROUPS)
    return FP4_ERR_SHAPE;
  if (((M_total + 255) / 256 + num_groups) * ((N + 255) / 256) >= (int64_t)1 << 31) return FP4_ERR_SHAPE;
  if (fmt == FP4_MXFP4 && (g_a != nullptr || g_b != nullptr)) return FP4_ERR_DTYPE;
  if (M_total == 0 || N == 0) return FP4_OK;
  if (D == nullptr) return FP4_ERR_NULL;
  if (!aligned(D, d_bytes)) return FP4_ERR_ALIGN;
  if (K == 0) {   // every group's contraction is empty: D = 0
    fp4_status st = check_arch();
    if (st != FP4_OK) return st;
    FP4_TRY_LAUNCH(fp4impl::launch_zero_fill(D, M_total * N, d_bytes, stream), "fp4_grouped_gemm");
    return FP4_OK;
  }
  if (A == nullptr || a_scales == nullptr || W == nullptr || w_scales == nullptr ||
      offsets == nullptr)
    return FP4_ERR_NULL;
  if (fmt == FP4_NVFP4 && (g_a == nullptr || g_b == nullptr)) return FP4_ERR_NULL;
  if (!aligned(A, 16) || !aligned(W, 16) || !aligned(offsets, 4)) return FP4_ERR_ALIGN;
  fp4_status st = check_arch();
  if (st != FP4_OK) return st;
  FP4_TRY_LAUNCH(fp4impl::launch_grouped_gemm(fmt == FP4_MXFP4, A, a_scales, g_a, W, w_scales, g_b,
                                              g_d, num_groups, offsets, M_total, N, K, D, d_bytes,
                                              stream),
                 "fp4_grouped_gemm");
  return FP4_OK;
}

size_t fp4_gemv_workspace_bytes(int64_t B, int64_t K) {
  if (B < 0 || K < 0) return 0;
  return fp4impl::gemv_workspace_bytes(B, K);
}

fp4_status fp4_gemv_batched(const void* x, fp4_dtype xt, int64_t B, const uint8_t* W,
                            const uint8_t* w_scales, const float* g_w, int64_t N, int64_t K,
                            float g_d, void* y, fp4_dtype yt, void* workspace,
                            size_t workspace_bytes, hipStream_t stream) {
  if (!valid_dtype(xt) || !valid_dtype(yt)) return FP4_ERR_DTYPE;
  if (B < 1 || B > 16 || N < 0 || K < 0 || K % 32 != 0) return FP4_ERR_SHAPE;
  if (N > FP4_GEMV_MAX_N || K > FP4_GEMV_MAX_K) return FP4_ERR_SHAPE;
  if (N == 0) return FP4_OK;
  if (K == 0) {   // empty contraction: y = 0, x, W and the workspace are not read
    if (y == nullptr) return FP4_ERR_NULL;
    if (!aligned(y, yt == FP4_BF16 ? 2 : 4)) return FP4_ERR_ALIGN;
    fp4_status st = check_arch();
    if (st != FP4_OK) return st;
    FP4_TRY_LAUNCH(fp4impl::launch_zero_fill(y, B * N, yt == FP4_BF16 ? 2 : 4, stream), "fp4_gemv_batched");
    return FP4_OK;
  }
  if (x == nullptr || W == nullptr || w_scales == nullptr || g_w == nullptr || y == nullptr)
    return FP4_ERR_NULL;
  if (workspace == nullptr || workspace_bytes < fp4impl::gemv_workspace_bytes(B, K))
    return FP4_ERR_WORKSPACE;
  if (!aligned(x, 16) || !aligned(W, 16) || !aligned(workspace, 16) || !aligned(w_scales, 2) ||
      !aligned(y, yt == FP4_BF16 ? 2 : 4))
    return FP4_ERR_ALIGN;
  fp4_status st = check_arch();
  if (st != FP4_OK) return st;
  FP4_TRY_LAUNCH(fp4impl::launch_gemv(x, xt == FP4_BF16, B, W, w_scales, g_w, N, K, g_d, y,
                                      yt == FP4_BF16, workspace, stream),
                 "fp4_gemv_batched");
  return FP4_OK;
}

fp4_status hadamard_quantize(const void* x, fp4_dtype xt, int64_t rows, int64_t cols, int group,
                             fp4_rounding mode, uint64_t seed, uint8_t* q, uint8_t* scales,
                             float* global_amax, int amax_given, float* global_scale,
                             void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (mode != FP4_RNE && mode != FP4_SR) return FP4_ERR_DTYPE;
  if (group != 128) return FP4_ERR_SHAPE;
  if (cols % group != 0) return FP4_ERR_SHAPE;
  fp4_status st = check_quant_args(x, xt, rows, cols, q, scales, global_amax, amax_given,
                                   global_scale, workspace, workspace_bytes);
  if (st != FP4_OK) return st;
  if (rows != 0 && cols != 0 && (!aligned(x, 16) || !aligned(q, 16) || !aligned(scales, 2)))
    return FP4_ERR_ALIGN;
  if ((st = check_arch()) != FP4_OK) return st;
  const bool bf16 = xt == FP4_BF16;
  if (rows == 0 || cols == 0) {
    FP4_TRY_LAUNCH(fp4impl::launch_empty_scales(amax_given ? nullptr : global_amax, global_scale,
                                                stream),
                   "hadamard_quantize");
    return FP4_OK;
  }
  uint32_t* partials = nullptr;
  int npart = 0;
  if (!amax_given) {
    partials = static_cast<uint32_t*>(workspace);
    FP4_TRY_LAUNCH(fp4impl::launch_hadamard_amax(x, bf16, rows, cols, partials, &npart, stream),
                   "hadamard_quantize/amax");
  }
  FP4_TRY_LAUNCH(fp4impl::launch_hadamard_quant(x, bf16, rows, cols, mode == FP4_SR, seed, q,
                                                scales, amax_given ? global_amax : nullptr,
                                                partials, npart,
                                                amax_given ? nullptr : global_amax, global_scale,
                                                stream),
                 "hadamard_quantize/encode");
  return FP4_OK;
}

fp4_status hadamard_quantize_mx(const void* x, fp4_dtype xt, int64_t rows, int64_t cols, int group,
                                fp4_rounding mode, uint64_t seed, uint8_t* q, uint8_t* scales,
                                hipStream_t stream) {
  if (!valid_dtype(xt)) return FP4_ERR_DTYPE;
  if (mode != FP4_RNE && mode != FP4_SR) return FP4_ERR_DTYPE;
  if (group != 128 || rows < 0 || cols < 0 || cols % group != 0) return FP4_ERR_SHAPE;
  if (rows == 0 || cols == 0) return FP4_OK;
  if (x == nullptr || q == nullptr || scales == nullptr) return FP4_ERR_NULL;
  if (!aligned(x, 16) || !aligned(q, 16)) return FP4_ERR_ALIGN;
  fp4_status st = check_arch();
  if (st != FP4_OK) return st;
  FP4_TRY_LAUNCH(fp4impl::launch_hadamard_quant_mx(x, xt == FP4_BF16, rows, cols, mode == FP4_SR,
                                                   seed, q, scales, stream),
                 "hadamard_quantize_mx");
  return FP4_OK;
}

fp4_status hadamard_rotate(const void* x, fp4_dtype xt, int64_t rows, int64_t cols, int group,
                           void* y, fp4_dtype yt, hipStream_t stream) {
  if (!valid_dtype(xt) || !valid_dtype(yt)) return FP4_ERR_DTYPE;
  if (group != 128 || rows < 0 || cols < 0 || cols % group != 0) return FP4_ERR_SHAPE;
  if (rows == 0 || cols == 0) return FP4_OK;
  if (x == nullptr || y == nullptr) return FP4_ERR_NULL;
  if (!aligned(x, 16) || !aligned(y, 16)) return FP4_ERR_ALIGN;
  fp4_status st = check_arch();
  if (st != FP4_OK) return st;
  FP4_TRY_LAUNCH(fp4impl::launch_hadamard_rotate(x, xt == FP4_BF16, rows, cols, y, yt == FP4_BF16,
                                                 stream),
                 "hadamard_rotate");
  return FP4_OK;
}

}  // extern "C"

namespace {

bool valid_act(fp4_activation a) { return a >= FP4_ACT_NONE && a <= FP4_ACT_GELU_TANH; }
// a pointer aligned to its FP4_F32 / FP4_BF16 element
bool elem_aligned(const void* p, fp4_dtype t) { return aligned(p, t == FP4_BF16 ? 2 : 4); }

// Shared front half of the fused GEMMs (ngroups 0: dense).
fp4_status fused_gemm(fp4_format fmt, const uint8_t* A, const uint8_t* a_scales, const float* g_a,
                      const uint8_t* W, const uint8_t* w_scales, const float* g_b, float g_d,
                      int64_t ngroups, const int32_t* offsets, int64_t M, int64_t N, int64_t K,
                      fp4_activation activation, int gated, const void* bias, fp4_dtype bias_type,
                      const void* residual, fp4_dtype residual_type, void* preact,
                      fp4_dtype preact_type, void* D, fp4_dtype dt, hipStream_t stream,
                      const char* name) {
  if (fmt != FP4_NVFP4 && fmt != FP4_MXFP4) return FP4_ERR_DTYPE;
  if (!valid_dtype(dt) || !valid_act(activation)) return FP4_ERR_DTYPE;
  if (bias != nullptr && !valid_dtype(bias_type)) return FP4_ERR_DTYPE;
  if (residual != nullptr && !valid_dtype(residual_type)) return FP4_ERR_DTYPE;
  if (preact != nullptr && !valid_dtype(preact_type)) return FP4_ERR_DTYPE;
  if (M < 0 || N < 0 || K < 0 || K % 32 != 0) return FP4_ERR_SHAPE;
  if (M > FP4_GEMM_MAX_MN || N > FP4_GEMM_MAX_MN || K > FP4_GEMM_MAX_K) return FP4_ERR_SHAPE;
  if (gated != 0 && (gated != 1 || N % 2 != 0)) return FP4_ERR_SHAPE;
  if (((M + 255) / 256 + ngroups) * ((N + 255) / 256) >= (int64_t)1 << 31) return FP4_ERR_SHAPE;
  if (fmt == FP4_MXFP4 && (g_a != nullptr || g_b != nullptr)) return FP4_ERR_DTYPE;
  if (M == 0 || N == 0) return FP4_OK;
  if (D == nullptr || (ngroups > 0 && offsets == nullptr)) return FP4_ERR_NULL;
  if (K > 0 && (A == nullptr || a_scales == nullptr || W == nullptr || w_scales == nullptr))
    return FP4_ERR_NULL;
  if (K > 0 && fmt == FP4_NVFP4 && (g_a == nullptr || g_b == nullptr)) return FP4_ERR_NULL;
  if (!aligned(A, 16) || !aligned(W, 16) || !elem_aligned(D, dt) || !aligned(offsets, 4) ||
      !aligned(g_a, 4) || !aligned(g_b, 4))
    return FP4_ERR_ALIGN;
  if ((bias && !elem_aligned(bias, bias_type)) || (residual && !elem_aligned(residual, residual_type)) ||
      (preact && !elem_aligned(preact, preact_type)))
    return FP4_ERR_ALIGN;
  // in place only element for element
  if (residual == D && residual_type != dt) return FP4_ERR_ALIAS;
  if (preact == D || (preact != nullptr && preact == residual)) return FP4_ERR_ALIAS;
  fp4_status st = check_arch();
  if (st != FP4_OK) return st;
  const fp4impl::Epilogue ep{activation, gated, bias, bias_type == FP4_BF16, residual,
                             residual_type == FP4_BF16, preact, preact_type == FP4_BF16};
  FP4_TRY_LAUNCH(fp4impl::launch_fused_gemm(fmt == FP4_MXFP4, A, a_scales, g_a, W, w_scales, g_b, g_d,
                                            ngroups, offsets, M, N, K, ep, D, dt == FP4_BF16, stream),
                 name);
  return FP4_OK;
}

// Sizes shared by the routing and dispatch calls.
bool bad_slots(int64_t T, int64_t E, int top_k) {
  return T < 0 || T > FP4_MOE_MAX_TOKENS || E < 1 || E > FP4_MOE_MAX_EXPERTS || top_k < 1 ||
         top_k > FP4_MOE_MAX_TOPK || T * top_k > (int64_t)1 << 30;
}

}  // namespace

extern "C" {

fp4_status fp4_scaled_gemm_fused(fp4_format fmt, const uint8_t* A, const uint8_t* a_scales,
                                 const float* g_a, const uint8_t* W, const uint8_t* w_scales,
                                 const float* g_b, float g_d, int64_t M, int64_t N, int64_t K,
                                 fp4_activation activation, int gated, const void* bias,
                                 fp4_dtype bias_type, const void* residual, fp4_dtype residual_type,
                                 void* preact, fp4_dtype preact_type, void* D, fp4_dtype dt,
                                 hipStream_t stream) {
  return fused_gemm(fmt, A, a_scales, g_a, W, w_scales, g_b, g_d, 0, nullptr, M, N, K, activation, gated,
                    bias, bias_type, residual, residual_type, preact, preact_type, D, dt, stream,
                    "fp4_scaled_gemm_fused");
}

fp4_status fp4_grouped_gemm_fused(fp4_format fmt, const uint8_t* A, const uint8_t* a_scales,
                                  const float* g_a, const uint8_t* W, const uint8_t* w_scales,
                                  const float* g_b, float g_d, int64_t num_groups,
                                  const int32_t* offsets, int64_t M_total, int64_t N, int64_t K,
                                  fp4_activation activation, int gated, const void* bias,
                                  fp4_dtype bias_type, const void* residual,
                                  fp4_dtype residual_type, void* preact, fp4_dtype preact_type,
                                  void* D, fp4_dtype dt, hipStream_t stream) {
  if (num_groups < 1 || num_groups > FP4_GROUPED_MAX_GROUPS) return FP4_ERR_SHAPE;
  return fused_gemm(fmt, A, a_scales, g_a, W, w_scales, g_b, g_d, num_groups, offsets, M_total, N, K,
                    activation, gated, bias, bias_type, residual, residual_type, preact, preact_type, D,
                    dt, stream, "fp4_grouped_gemm_fused");
}

size_t fp4_epilogue_backward_workspace_bytes(int64_t num_groups, int64_t M, int64_t N) {
  if (num_groups < 1 || M < 0 || N < 1) return 0;
  return fp4impl::epilogue_grad_workspace_bytes(num_groups, M, N);
}

fp4_status fp4_epilogue_backward(const void* dD, fp4_dtype dD_type, const void* z, fp4_dtype z_type,
                                 int64_t num_groups, const int32_t* offsets, int64_t M, int64_t N,
                                 fp4_activation activation, int gated, void* dz, fp4_dtype dz_type,
                                 float* dbias, void* workspace, size_t workspace_bytes,
                                 hipStream_t stream) {
  if (!valid_dtype(dD_type) || !valid_dtype(z_type) || !valid_dtype(dz_type) || !valid_act(activation))
    return FP4_ERR_DTYPE;
  if (M < 0 || N < 0 || M > FP4_GEMM_MAX_MN || N > FP4_GEMM_MAX_MN) return FP4_ERR_SHAPE;
  if (gated != 0 && (gated != 1 || N % 2 != 0)) return FP4_ERR_SHAPE;
  if (num_groups < 1 || num_groups > FP4_GROUPED_MAX_GROUPS || (offsets == nullptr && num_groups != 1))
    return FP4_ERR_SHAPE;
  if (num_groups * ((N + 511) / 512) >= (int64_t)1 << 28) return FP4_ERR_SHAPE;
  if (N == 0 || (M == 0 && dbias == nullptr)) return FP4_OK;
  if (M > 0 && (dD == nullptr || z == nullptr || dz == nullptr)) return FP4_ERR_NULL;
  if (dbias != nullptr &&
      (workspace == nullptr || workspace_bytes < fp4_epilogue_backward_workspace_bytes(num_groups, M, N)))
    return FP4_ERR_WORKSPACE;
  if (!elem_aligned(dD, dD_type) || !elem_aligned(z, z_type) || !elem_aligned(dz, dz_type) ||
      !aligned(dbias, 4) || !aligned(offsets, 4) || (dbias != nullptr && !aligned(workspace, 4)))
    return FP4_ERR_ALIGN;
  if (M > 0 && (dz == dD || (dz == z && dz_type != z_type))) return FP4_ERR_ALIAS;
  fp4_status st = check_arch();
  if (st != FP4_OK) return st;
  FP4_TRY_LAUNCH(fp4impl::launch_epilogue_grad(dD, dD_type == FP4_BF16, z, z_type == FP4_BF16, num_groups,
                                               offsets, M, N, activation, gated != 0, dz,
                                               dz_type == FP4_BF16, dbias, workspace, stream),
                 "fp4_epilogue_backward");
  return FP4_OK;
}

fp4_status moe_route(const void* logits, fp4_dtype lt, int64_t T, int64_t E, int top_k,
                     fp4_score score, const float* bias, int num_groups, int top_groups,
                     int group_top, int renormalize, float scale, int32_t* ids, float* weights,
                     hipStream_t stream) {
  if (!valid_dtype(lt) || (score != FP4_SCORE_SOFTMAX && score != FP4_SCORE_SIGMOID)) return FP4_ERR_DTYPE;
  if (bad_slots(T, E, top_k) || top_k > E) return FP4_ERR_SHAPE;
  if (num_groups < 1 || num_groups > FP4_MOE_MAX_GROUPS || E % num_groups != 0 || top_groups < 1 ||
      top_groups > num_groups || group_top < 1 || group_top > 2)
    return FP4_ERR_SHAPE;
  if (T == 0) return FP4_OK;
  if (logits == nullptr || ids == nullptr || weights == nullptr) return FP4_ERR_NULL;
  if (!elem_aligned(logits, lt) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(weights, 4))
    return FP4_ERR_ALIGN;
  fp4_status st = check_arch();
  if (st != FP4_OK) return st;
  const fp4impl::RouteProblem p{logits, lt == FP4_BF16, T, E, top_k, score == FP4_SCORE_SIGMOID,
                                renormalize != 0, scale};
  FP4_TRY_LAUNCH(fp4impl::launch_route(p, bias, num_groups, top_groups, group_top, ids, weights, stream),
                 "moe_route");
  return FP4_OK;
}

fp4_status moe_route_backward(const float* d_weights, const void* logits, fp4_dtype lt,
                              const int32_t* ids, int64_t T, int64_t E, int top_k, fp4_score score,
                              int renormalize, float scale, void* d_logits, fp4_dtype dt,
                              hipStream_t stream) {
  if (!valid_dtype(lt) || !valid_dtype(dt) || (score != FP4_SCORE_SOFTMAX && score != FP4_SCORE_SIGMOID))
    return FP4_ERR_DTYPE;
  if (bad_slots(T, E, top_k) || top_k > E) return FP4_ERR_SHAPE;
  if (T == 0) return FP4_OK;
  if (d_weights == nullptr || logits == nullptr || ids == nullptr || d_logits == nullptr)
    return FP4_ERR_NULL;
  if (!aligned(d_weights, 4) || !elem_aligned(logits, lt) || !aligned(ids, 4) || !elem_aligned(d_logits, dt))
    return FP4_ERR_ALIGN;
  fp4_status st = check_arch();
  if (st != FP4_OK) return st;
  const fp4impl::RouteProblem p{logits, lt == FP4_BF16, T, E, top_k, score == FP4_SCORE_SIGMOID,
                                renormalize != 0, scale};
  FP4_TRY_LAUNCH(fp4impl::launch_route_grad(p, d_weights, ids, d_logits, dt == FP4_BF16, stream),
                 "moe_route_backward");
  return FP4_OK;
}

size_t moe_dispatch_workspace_bytes(int64_t T, int64_t top_k, int64_t E) {
  if (T < 0 || T > FP4_MOE_MAX_TOKENS || top_k < 1 || top_k > FP4_MOE_MAX_TOPK || E < 1 ||
      E > FP4_MOE_MAX_EXPERTS)
    return 0;
  return fp4impl::dispatch_workspace_bytes(T * top_k, E);
}

fp4_status moe_dispatch(fp4_format fmt, const void* x, fp4_dtype xt, int64_t T, int64_t H,
                        const int32_t* ids, int top_k, int64_t E, uint8_t* q, uint8_t* scales,
                        float* global_amax, int amax_given, float* global_scale, int32_t* offsets,
                        int32_t* slot_rows, int32_t* row_slots, void* workspace,
                        size_t workspace_bytes, hipStream_t stream) {
  if (fmt != FP4_NVFP4 && fmt != FP4_MXFP4) return FP4_ERR_DTYPE;
  if (!valid_dtype(xt)) return FP4_ERR_DTYPE;
  if (bad_slots(T, E, top_k) || H < 0 || H > FP4_GEMM_MAX_K || H % 32 != 0) return FP4_ERR_SHAPE;
  const bool mx = fmt == FP4_MXFP4;
  if (mx && (global_amax != nullptr || global_scale != nullptr || amax_given)) return FP4_ERR_DTYPE;
  if (offsets == nullptr) return FP4_ERR_NULL;
  if (!mx && (global_scale == nullptr || (amax_given && global_amax == nullptr))) return FP4_ERR_NULL;
  if (T > 0) {
    if (ids == nullptr || slot_rows == nullptr || row_slots == nullptr) return FP4_ERR_NULL;
    if (H > 0 && (x == nullptr || q == nullptr || scales == nullptr)) return FP4_ERR_NULL;
    if (workspace == nullptr || workspace_bytes < moe_dispatch_workspace_bytes(T, top_k, E))
      return FP4_ERR_WORKSPACE;
  }
  if (!elem_aligned(x, xt) || !aligned(q, 16) || !aligned(ids, 4) || !aligned(offsets, 4) ||
      !aligned(slot_rows, 4) || !aligned(row_slots, 4) || !aligned(workspace, 4) ||
      !aligned(global_amax, 4) || !aligned(global_scale, 4))
    return FP4_ERR_ALIGN;
  // one workgroup writes *global_scale while the others still read *global_amax
  if (global_amax != nullptr && global_amax == global_scale) return FP4_ERR_ALIAS;
  fp4_status st = check_arch();
  if (st != FP4_OK) return st;
  const fp4impl::DispatchProblem p{mx, x, xt == FP4_BF16, T, H, ids, top_k, E, q, scales,
                                   amax_given ? global_amax : nullptr,
                                   amax_given ? nullptr : global_amax, global_scale, offsets, slot_rows,
                                   row_slots, workspace};
  FP4_TRY_LAUNCH(fp4impl::launch_dispatch(p, stream), "moe_dispatch");
  return FP4_OK;
}

fp4_status moe_combine(const void* rows, fp4_dtype rt, int64_t M, int64_t H, const float* weights,
                       const int32_t* slot_rows, int64_t T, int top_k, const void* residual,
                       fp4_dtype residual_type, void* y, fp4_dtype yt, hipStream_t stream) {
  if (!valid_dtype(rt) || !valid_dtype(yt) || (residual != nullptr && !valid_dtype(residual_type)))
    return FP4_ERR_DTYPE;
  if (bad_slots(T, 1, top_k) || M < 0 || M > FP4_GEMM_MAX_MN || H < 0 || H > FP4_GEMM_MAX_K)
    return FP4_ERR_SHAPE;
  if (T * ((H + 255) / 256) >= (int64_t)1 << 31) return FP4_ERR_SHAPE;
  if (T == 0 || H == 0) return FP4_OK;
  if ((M > 0 && rows == nullptr) || weights == nullptr || slot_rows == nullptr || y == nullptr)
    return FP4_ERR_NULL;
  if (!elem_aligned(rows, rt) || !aligned(weights, 4) || !aligned(slot_rows, 4) || !elem_aligned(y, yt) ||
      (residual != nullptr && !elem_aligned(residual, residual_type)))
    return FP4_ERR_ALIGN;
  if (rows == y || (residual == y && residual_type != yt)) return FP4_ERR_ALIAS;
  fp4_status st = check_arch();
  if (st != FP4_OK) return st;
  FP4_TRY_LAUNCH(fp4impl::launch_combine(rows, rt == FP4_BF16, M, H, weights, slot_rows, T, top_k,
                                         residual, residual_type == FP4_BF16, y, yt == FP4_BF16, stream),
                 "moe_combine");
  return FP4_OK;
}

fp4_status moe_combine_backward(const void* dy, fp4_dtype dyt, const void* rows, fp4_dtype rt,
                                const float* weights, const int32_t* slot_rows,
                                const int32_t* row_slots, int64_t T, int top_k, int64_t H,
                                void* d_rows, fp4_dtype drt, float* d_weights, hipStream_t stream) {
  if (!valid_dtype(dyt) || !valid_dtype(rt) || !valid_dtype(drt)) return FP4_ERR_DTYPE;
  if (bad_slots(T, 1, top_k) || H < 0 || H > FP4_GEMM_MAX_K) return FP4_ERR_SHAPE;
  if (T == 0) return FP4_OK;
  if (weights == nullptr || slot_rows == nullptr || row_slots == nullptr || d_weights == nullptr)
    return FP4_ERR_NULL;
  if (H > 0 && (dy == nullptr || rows == nullptr || d_rows == nullptr)) return FP4_ERR_NULL;
  if (!elem_aligned(dy, dyt) || !elem_aligned(rows, rt) || !elem_aligned(d_rows, drt) ||
      !aligned(weights, 4) || !aligned(slot_rows, 4) || !aligned(row_slots, 4) || !aligned(d_weights, 4))
    return FP4_ERR_ALIGN;
  if (H > 0 && (d_rows == dy || d_rows == rows)) return FP4_ERR_ALIAS;
  fp4_status st = check_arch();
  if (st != FP4_OK) return st;
  FP4_TRY_LAUNCH(fp4impl::launch_combine_grad(dy, dyt == FP4_BF16, rows, rt == FP4_BF16, T * top_k, H,
                                              weights, slot_rows, row_slots, T, top_k, d_rows,
                                              drt == FP4_BF16, d_weights, stream),
                 "moe_combine_backward");
  return FP4_OK;
}

}  // extern "C"
