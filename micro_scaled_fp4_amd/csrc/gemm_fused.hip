// Host side of the block-scaled FP4 GEMMs with bias, activation and residual in
// the epilogue: the tile kernels of gemm_kernels.h with their fused outputs.
#include "gemm_kernels.h"

namespace {

// Rows of a grouped output past the last group's (slots that were dropped) hold
// zeros, so that what reads the whole tensor next (a quantizer's amax) sees none
// of the memory's earlier contents.
__global__ void __launch_bounds__(256)
    k_zero_tail(const int32_t* __restrict__ goff, int ngroups, int M, int64_t row_bytes,
                uint8_t* __restrict__ D, int64_t z_row_bytes, uint8_t* __restrict__ z) {
  const int lo = min(max(goff[ngroups], 0), M);
  const int64_t i0 = (int64_t)blockIdx.x * 256 + threadIdx.x, step = (int64_t)gridDim.x * 256;
  // row_bytes and z_row_bytes are even, D and z 2-byte aligned (bf16 or float32 rows)
  for (int64_t i = (int64_t)lo * row_bytes / 2 + i0; i < (int64_t)M * row_bytes / 2; i += step)
    reinterpret_cast<uint16_t*>(D)[i] = 0;
  if (z != nullptr)
    for (int64_t i = (int64_t)lo * z_row_bytes / 2 + i0; i < (int64_t)M * z_row_bytes / 2; i += step)
      reinterpret_cast<uint16_t*>(z)[i] = 0;
}

template <bool MX, bool GROUPED>
hipError_t launch_fused_t(const uint8_t* A, const uint8_t* as, const uint8_t* W, const uint8_t* ws,
                          const float* g_a, const float* g_b, float g_d, int M, int N, int K, void* D,
                          bool out_bf16, const Groups& gr, const FusedArgs& f, hipStream_t stream) {
  const bool vec = K % BK == 0 && (reinterpret_cast<uintptr_t>(as) & 15) == 0 &&
                   (reinterpret_cast<uintptr_t>(ws) & 15) == 0;
  const OutArgs o{D, nullptr, nullptr, nullptr};
#define FP4_LAUNCH(OUTV, VECV) \
  launch_t<MX, OUTV, VECV, GROUPED, true>(A, as, W, ws, g_a, g_b, g_d, M, N, K, o, stream, gr, f)
  if (out_bf16) return vec ? FP4_LAUNCH(2, true) : FP4_LAUNCH(2, false);
  return vec ? FP4_LAUNCH(4, true) : FP4_LAUNCH(4, false);
#undef FP4_LAUNCH
}

}  // namespace

namespace fp4impl {

hipError_t launch_fused_gemm(bool mx, const uint8_t* A, const uint8_t* a_scales, const float* g_a,
                             const uint8_t* W, const uint8_t* w_scales, const float* g_b, float g_d,
                             int64_t ngroups, const int32_t* offsets, int64_t M, int64_t N, int64_t K,
                             const Epilogue& ep, void* D, bool out_bf16, hipStream_t stream) {
  // buffer ranges cover one 256-row tile of an operand: 256 * K / 2 < 2^31
  if (M > (1 << 30) || N > (1 << 30) || K >= (1 << 23) || ngroups > (1 << 20) ||
      ((M + BM - 1) / BM + ngroups) * ((N + BN - 1) / BN) >= (int64_t)1 << 31)
    return hipErrorInvalidValue;
  hipError_t e;
  if (few_rows(mx, ngroups, M, K)) {
    e = launch_few_rows(mx, A, a_scales, g_a, W, w_scales, g_b, g_d, ngroups, offsets, M, N, K, ep, D,
                        out_bf16, stream);
  } else {
    FusedArgs f{ep.bias, ep.residual, ep.preact, ep.bias_bf16, ep.residual_bf16, ep.preact_bf16,
                ep.activation, ep.gated, 0};
    auto ok16 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
    f.vec = N % 16 == 0 && ok16(ep.bias) && ok16(ep.residual) && ok16(ep.preact) && ok16(D);
    const Groups gr{offsets, (int)ngroups};
#define FP4_LAUNCH(MXV, GV)                                                                            \
  launch_fused_t<MXV, GV>(A, a_scales, W, w_scales, g_a, g_b, g_d, (int)M, (int)N, (int)K, D, out_bf16, \
                          gr, f, stream)
    if (ngroups > 0)
      e = mx ? FP4_LAUNCH(true, true) : FP4_LAUNCH(false, true);
    else
      e = mx ? FP4_LAUNCH(true, false) : FP4_LAUNCH(false, false);
#undef FP4_LAUNCH
  }
  if (e != hipSuccess || ngroups == 0) return e;
  const int64_t No = ep.gated ? N / 2 : N;
  hipLaunchKernelGGL(k_zero_tail, dim3(64), dim3(256), 0, stream, offsets, (int)ngroups, (int)M,
                     No * (out_bf16 ? 2 : 4), static_cast<uint8_t*>(D), N * (ep.preact_bf16 ? 2 : 4),
                     static_cast<uint8_t*>(ep.preact));
  return hipGetLastError();
}

}  // namespace fp4impl
