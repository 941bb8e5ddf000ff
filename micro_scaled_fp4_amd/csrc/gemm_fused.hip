// Host side of the block-scaled FP4 GEMMs with bias, activation and residual in
// the epilogue: the tile kernels of gemm_kernels.h with their fused outputs.
#include <math.h>

#include "gemm_kernels.h"

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

// Which kernel, as the rows of A that it takes at a time: 16, 32 or 64
// (gemm_few_rows.hip), 128 (gemm_mid.hip) or 256, by the least modelled time.
// Few rows stream W once at memory speed but repeat its unpacking every 16 to 64
// rows; 128 x 128 tiles fill the device from a quarter of the output that 256 x 256
// tiles need, at four fifths of their rate.  Measured at the five (us, NVFP4):
//   128 x 512 x 4096     11 /  14 /  16 /  34 /  93
//   300 x 1000 x 7168    27 /  33 /  23 /  58 / 181
//   128 x 27648 x 5120  126 /  93 /  93 /  47 / 115
//   1021 x 5120 x 7168  222 / 159 / 163 / 105 / 154
//   4096 x 4096 x 4096    - /   - /   - / 134 / 117
//   64 groups of 4096 x 7168: 32 rows each 431 / 292 / 446 / 428 / 661,
//                            256 rows 3255 / 2143 / 2092 / 919 / 771
// Over 56 sizes and formats the chosen kernel takes 3% longer than the best of the
// five in the mean, 1.5 times at worst (23 us).  Groups' sizes are on the device: each is
// taken as the mean, plus a quarter of a tile for their unequal ends.
int choose(bool mx, int64_t ngroups, int64_t M, int64_t N, int64_t K) {
  if (K == 0) return 256;
  const int64_t groups = ngroups > 0 ? ngroups : 1;
  auto tiles = [&](int rows) {
    if (ngroups == 0) return (double)((M + rows - 1) / rows);
    return fmax(1.0, (double)M / groups / rows + 0.25);
  };
  const double stages = (double)((K + BK - 1) / BK);
  const double rounds = ceil(groups * tiles(256) * ((N + BN - 1) / BN) / fp4impl::num_cus());
  int best = 256;
  double us = mx ? 12.3 + 1.95 * rounds * stages : 19.6 + 5.4 * rounds * stages;
  auto offer = [&](int rows, double t) {
    if (t < us) {
      us = t;
      best = rows;
    }
  };
  if (((M + 127) / 128 + (ngroups < M ? ngroups : M)) * ((N + 127) / 128) < (int64_t)1 << 31)   // (a workgroup per tile)
    offer(128, fp4impl::mid_us(mx, groups, tiles(128), N, K));
  for (int rows = 64; rows >= 16; rows /= 2)
    offer(rows, fp4impl::few_rows_us(mx, groups, tiles(rows), N, K, rows));
  return best;
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
  const int rows = choose(mx, ngroups, M, N, K);
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
