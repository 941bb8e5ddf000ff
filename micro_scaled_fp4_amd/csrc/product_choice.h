// Which kernel a fused FP4 product takes, by the least modelled time.  Host code
// without a device: `cus` is the device's compute units.
#pragma once

#include <math.h>
#include <stdint.h>

namespace fp4impl {

inline int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Waves of a few-row workgroup (of 8) that split K: at least two pairs of 128-value
// steps each, so that the partial tiles' exchange is small beside the stream.
inline int few_rows_split(int64_t K) {
  const int64_t P = div_up(K, 256);
  return P >= 16 ? 8 : P >= 8 ? 4 : P >= 4 ? 2 : 1;
}

// gemm_few_rows.hip, `item` (16, 32 or 64) rows of A at a time, `groups` (dense: 1) of
// row_items items each: a fixed part and, per value of K, one strip's time for each of
// the strips that a slot goes through (whole units of S granules, every workgroup
// waiting for the fullest).  Fitted to 28 sizes in each format, dense and grouped.
inline double few_rows_us(bool mx, int64_t groups, double row_items, int64_t N, int64_t K, int item, int cus) {
  const int S = item == 64 ? 2 : 4, slots = 8 / few_rows_split(K);
  const double granules = groups * row_items * div_up(N, 16 * slots);
  const double units = ceil(granules / (cus * S));
  const double strip = mx ? (item == 16 ? 0.33e-3 : item == 32 ? 0.48e-3 : 0.92e-3)
                          : (item == 16 ? 0.45e-3 : item == 32 ? 0.62e-3 : 1.18e-3);
  const double fixed = mx ? (item == 64 ? 6.8 : 5.1) : (item == 16 ? 6.7 : item == 32 ? 7.6 : 8.6);
  return fixed + units * S * slots * K * strip;
}

// gemm_mid.hip, `groups` of row_tiles 128-row tiles each: a fixed part and the fullest
// CU's tiles times stages (two tiles on a CU share its LDS and its MFMA pipes, so each
// takes longer than one alone).
inline double mid_us(bool mx, int64_t groups, double row_tiles, int64_t N, int64_t K, int cus) {
  const double tiles = ceil(groups * row_tiles * div_up(N, 128) / cus);
  const int64_t stages = div_up(K, 256);
  if (tiles <= 1) return mx ? 7.1 + 0.61 * stages : 8.5 + 1.8 * stages;
  return mx ? 7.1 + 0.89 * tiles * stages : 8.5 + 2.0 * tiles * stages;
}

// The kernel, as the rows of A that it takes at a time: 16, 32 or 64
// (gemm_few_rows.hip), 128 (gemm_mid.hip) or 256 (gemm_kernels.h).
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
// five in the mean, 1.5 times at worst: 300 x 1000 x 7168, 32 rows at a time (33 us)
// where 64 take 23, since units are counted whole and the kernel deals granules.
// Groups' sizes are on the device: each is taken as the mean, plus a quarter of a tile
// for their unequal ends.
inline int choose_rows(bool mx, int64_t ngroups, int64_t M, int64_t N, int64_t K, int cus) {
  if (K == 0) return 256;
  const int64_t groups = ngroups > 0 ? ngroups : 1;
  auto tiles = [&](int rows) {
    if (ngroups == 0) return (double)div_up(M, rows);
    return fmax(1.0, (double)M / groups / rows + 0.25);
  };
  const double stages = (double)div_up(K, 256);
  const double rounds = ceil(groups * tiles(256) * div_up(N, 256) / cus);
  int best = 256;
  double us = mx ? 12.3 + 1.95 * rounds * stages : 19.6 + 5.4 * rounds * stages;
  auto offer = [&](int rows, double t) {
    if (t < us) {
      us = t;
      best = rows;
    }
  };
  if ((div_up(M, 128) + (ngroups < M ? ngroups : M)) * div_up(N, 128) < (int64_t)1 << 31)   // (a workgroup per tile)
    offer(128, mid_us(mx, groups, tiles(128), N, K, cus));
  for (int rows = 64; rows >= 16; rows /= 2)
    offer(rows, few_rows_us(mx, groups, tiles(rows), N, K, rows, cus));
  return best;
}

}  // namespace fp4impl
