// Host side of the block-scaled FP4 GEMMs with bias, activation and residual in
// the epilogue: the tile kernels of gemm_kernels.h with their fused outputs.
#include "gemm_kernels.h"
#include "product_choice.h"

namespace {

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
  const int rows = choose_rows(mx, ngroups, M, N, K, num_cus());
  if (rows < 128)
    return launch_few_rows(mx, A, a_scales, g_a, W, w_scales, g_b, g_d, ngroups, offsets, M, N, K, ep, D,
                           out_bf16, rows, stream);
  if (rows == 128)
    return launch_mid(mx, A, a_scales, g_a, W, w_scales, g_b, g_d, ngroups, offsets, M, N, K, ep, D, out_bf16,
                      stream);
  FusedArgs f{ep.bias, ep.residual, ep.preact, ep.bias_bf16, ep.residual_bf16, ep.preact_bf16,
              ep.activation, ep.gated, 0};
  auto ok16 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
  f.vec = N % 16 == 0 && ok16(ep.bias) && ok16(ep.residual) && ok16(ep.preact) && ok16(D);
  const Groups gr{offsets, (int)ngroups};
#define FP4_LAUNCH(MXV, GV)                                                                              \
  launch_fused_t<MXV, GV>(A, a_scales, W, w_scales, g_a, g_b, g_d, (int)M, (int)N, (int)K, D, out_bf16, \
                          gr, f, stream)
  if (ngroups > 0) return mx ? FP4_LAUNCH(true, true) : FP4_LAUNCH(false, true);
  return mx ? FP4_LAUNCH(true, false) : FP4_LAUNCH(false, false);
#undef FP4_LAUNCH
}

}  // namespace fp4impl
