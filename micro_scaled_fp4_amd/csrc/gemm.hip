// Host side of the block-scaled FP4 GEMMs that write alpha * (A @ W^T) as it is:
// picks the kernel (gemm_kernels.h) by format, output type and alignment.
#include "gemm_kernels.h"

namespace {

template <bool MX, int OUT>
hipError_t launch_s(const uint8_t* A, const uint8_t* as, const uint8_t* W, const uint8_t* ws,
                    const float* g_a, const float* g_b, float g_d, int M, int N, int K,
                    const OutArgs& o, hipStream_t stream) {
  const bool vec = K % BK == 0 && (reinterpret_cast<uintptr_t>(as) & 15) == 0 &&
                   (reinterpret_cast<uintptr_t>(ws) & 15) == 0;
  return vec ? launch_t<MX, OUT, true>(A, as, W, ws, g_a, g_b, g_d, M, N, K, o, stream)
             : launch_t<MX, OUT, false>(A, as, W, ws, g_a, g_b, g_d, M, N, K, o, stream);
}

// d_bytes: 4 float32, 2 bf16, 1 E4M3, 0 NVFP4 codes
template <bool MX>
hipError_t launch_o(const uint8_t* A, const uint8_t* as, const uint8_t* W, const uint8_t* ws,
                    const float* g_a, const float* g_b, float g_d, int M, int N, int K,
                    const OutArgs& o, int d_bytes, hipStream_t stream) {
  switch (d_bytes) {
    case 4: return launch_s<MX, 4>(A, as, W, ws, g_a, g_b, g_d, M, N, K, o, stream);
    case 2: return launch_s<MX, 2>(A, as, W, ws, g_a, g_b, g_d, M, N, K, o, stream);
    case 1: return launch_s<MX, 1>(A, as, W, ws, g_a, g_b, g_d, M, N, K, o, stream);
    case 0: return launch_s<MX, 0>(A, as, W, ws, g_a, g_b, g_d, M, N, K, o, stream);
    default: return hipErrorInvalidValue;
  }
}

template <bool MX>
hipError_t launch_grouped_o(const uint8_t* A, const uint8_t* as, const uint8_t* W, const uint8_t* ws,
                            const float* g_a, const float* g_b, float g_d, int M, int N, int K,
                            void* D, int d_bytes, const Groups& gr, hipStream_t stream) {
  const bool vec = K % BK == 0 && (reinterpret_cast<uintptr_t>(as) & 15) == 0 &&
                   (reinterpret_cast<uintptr_t>(ws) & 15) == 0;
  const OutArgs o{D, nullptr, nullptr, nullptr};
#define FP4_GG(OUTV)                                                                          \
  return vec ? launch_t<MX, OUTV, true, true>(A, as, W, ws, g_a, g_b, g_d, M, N, K, o, stream, gr) \
             : launch_t<MX, OUTV, false, true>(A, as, W, ws, g_a, g_b, g_d, M, N, K, o, stream, gr)
  switch (d_bytes) {
    case 4: FP4_GG(4);
    case 2: FP4_GG(2);
    case 1: FP4_GG(1);
    default: return hipErrorInvalidValue;
  }
#undef FP4_GG
}

__global__ void k_global_scale(const float* __restrict__ amax, float* __restrict__ out) {
  if (threadIdx.x == 0) *out = nv_global_scale(*amax);
}

}  // namespace

namespace fp4impl {

hipError_t launch_gemm(bool mx, const uint8_t* A, const uint8_t* a_scales, const float* g_a,
                       const uint8_t* W, const uint8_t* w_scales, const float* g_b, float g_d,
                       int64_t M, int64_t N, int64_t K, void* D, int d_bytes, hipStream_t stream) {
  return launch_gemm_nvfp4_out(mx, A, a_scales, g_a, W, w_scales, g_b, g_d, M, N, K, D, d_bytes,
                               nullptr, nullptr, nullptr, stream);
}

hipError_t launch_gemm_nvfp4_out(bool mx, const uint8_t* A, const uint8_t* a_scales,
                                 const float* g_a, const uint8_t* W, const uint8_t* w_scales,
                                 const float* g_b, float g_d, int64_t M, int64_t N, int64_t K,
                                 void* D, int d_bytes, uint8_t* d_scales, const float* d_amax,
                                 float* d_gscale, hipStream_t stream) {
  // buffer ranges cover one 256-row tile of an operand: 256 * K / 2 < 2^31
  if (M > (1 << 30) || N > (1 << 30) || K >= (1 << 23)) return hipErrorInvalidValue;
  if (d_bytes == 0 && (d_scales == nullptr || d_amax == nullptr || d_gscale == nullptr))
    return hipErrorInvalidValue;
  const OutArgs o{D, d_scales, d_amax, d_gscale};
  return mx ? launch_o<true>(A, a_scales, W, w_scales, g_a, g_b, g_d, (int)M, (int)N, (int)K, o,
                             d_bytes, stream)
            : launch_o<false>(A, a_scales, W, w_scales, g_a, g_b, g_d, (int)M, (int)N, (int)K, o,
                              d_bytes, stream);
}

hipError_t launch_grouped_gemm(bool mx, const uint8_t* A, const uint8_t* a_scales,
                               const float* g_a, const uint8_t* W, const uint8_t* w_scales,
                               const float* g_b, float g_d, int64_t ngroups,
                               const int32_t* offsets, int64_t M, int64_t N, int64_t K, void* D,
                               int d_bytes, hipStream_t stream) {
  // buffer ranges cover one 256-row tile of an operand: 256 * K / 2 < 2^31
  if (M > (1 << 30) || N > (1 << 30) || K >= (1 << 23) || ngroups > (1 << 20))
    return hipErrorInvalidValue;
  if (((M + BM - 1) / BM + ngroups) * ((N + BN - 1) / BN) >= (int64_t)1 << 31) return hipErrorInvalidValue;
  const Groups gr{offsets, (int)ngroups};
  return mx ? launch_grouped_o<true>(A, a_scales, W, w_scales, g_a, g_b, g_d, (int)M, (int)N, (int)K,
                                     D, d_bytes, gr, stream)
            : launch_grouped_o<false>(A, a_scales, W, w_scales, g_a, g_b, g_d, (int)M, (int)N,
                                      (int)K, D, d_bytes, gr, stream);
}

hipError_t launch_nv_global_scale(const float* amax, float* out, hipStream_t stream) {
  hipLaunchKernelGGL(k_global_scale, dim3(1), dim3(64), 0, stream, amax, out);
  return hipGetLastError();
}

}  // namespace fp4impl
