// What the two attention kernels over a paged FP4 cache share: operands on their way to the
// fp16 MFMAs, query rows, masks, and a row's results.
//
// Mathematics.  Scores are taken as S^T = K Q^T and outputs as O^T = V^T P^T, so a query row is
// a lane (of 16 or 32) in both products: its maximum, sum and factors are per-lane values, and
// the weights leave the first product's accumulators in the order of positions in which the
// second takes them, if V's rows are picked in that order too.  Softmax in base 2 with a running
// maximum m and sum l:
//   x = c s,  c = |scale| log2(e) (factors of q's and k's scaling),  P = 2^(x - m + 11),
// where m follows the maximum only when it has grown by more than 4, so that sums are seldom
// rescaled; P is at most 2^15 then.
//
// Why fp16.  A value of the cache is E2M1 x its block scale.  NVFP4: E2M1 x E4M3 has at most 6
// significant bits and lies in [2^-10, 2688], exact in fp16; the tensor scale joins c and the
// output.  MXFP4: E8M0 scales are taken relative to the largest (2^(byte - ref) 2^13), exact
// down to 2^-36 of it; the reference joins c (keys) and is a running one like m (values).  A row
// of q is scaled by a power of two to a maximum in [2^14, 2^15): bf16 values are exact then
// (down to 2^-29 of the maximum), float32 ones are taken as two fp16 parts (22 bits).  P is
// rounded to fp16, half a step being 2^-12 of a weight, against 2^-8 of the bf16 output; its
// factor 2^11 keeps weights down to 2^-25 of the largest at full precision, which many small
// weights next to one large need.  With float32 operands P is two fp16 parts as well.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "fp4_device.h"
#include "fp4_internal.h"
#include "kv_units.h"
#include "scale_bytes.h"

namespace fp4dev {

using fp4impl::AttendProblem;

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr float kLn2 = 0.6931471805599453f;
constexpr float kWeightBits = 11.0f;            // P is 2^11 at m
constexpr float kGrowth = 4.0f;                 // a maximum within m + kGrowth leaves m as it is
// Up to this |m| a score's exponent is c s - m rounded once: m itself, rounded, is off by 2^-3 at most, and P
// stays below 2^15.2.  Past it the products are rounded as m was and then m is taken off, which is exact for
// the largest (elsewhere P would pass fp16, or be 0, from |m| = 2^28 on).
constexpr float kExactSteps = 0x1p22f;

// The larger of v in lanes l and l ^ 32, or l and l ^ 16.
__device__ __forceinline__ float max_over_halves(float v) {
  const u32x2 r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float max_over_rows(float v) {
  const u32x2 r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float sum_over_halves(float v) {
  const u32x2 r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float sum_over_rows(float v) {
  const u32x2 r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Largest of all lanes' v (v >= 0), the same in all.
__device__ __forceinline__ int wave_max_lanes(int v) {
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false));
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false));
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false));
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false));
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false));
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false));
  return __builtin_amdgcn_readlane(v, 63);
}

// Eight values of one dword of codes.  NVFP4: s is the block's E4M3 value x 2^-8 twice
// (e4m3_h2); MXFP4: fs is a power of two.
__device__ __forceinline__ f16x8 mx8(uint32_t codes, float fs) {
  const f16x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, fs, 0), p1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, fs, 1);
  const f16x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, fs, 2), p3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, fs, 3);
  return f16x8{p0.x, p0.y, p1.x, p1.y, p2.x, p2.y, p3.x, p3.y};
}
// 2^(byte - ref + 13), 2^-126 at the least (a value of at most 6 x that is 0 in fp16).
__device__ __forceinline__ float mx_factor(uint32_t byte, int ref) {
  return __uint_as_float((uint32_t)max((int)byte - ref + 140, 1) << 23);
}

// A descriptor of `bytes` bytes from p on, the same in all lanes by construction (the compiler
// would put a loop around each load otherwise).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t uniform_rsrc(const uint8_t* p, int bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(p);
  const uint64_t u = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(a >> 32)) << 32 |
                     (uint32_t)__builtin_amdgcn_readfirstlane((int)a);
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(u), 0, __builtin_amdgcn_readfirstlane(bytes),
                                           kBufferWord3);
}

// A query row of a tile: token row r of the call and query head h, or none.
struct QueryRow {
  int64_t r;
  int h;
  int first, last;               // positions that it sees: first <= t <= last
};

// Row `rho` (packed) of unit u.  Where there is none (h < 0) no position is masked: the row's q is
// taken as 0 and its results go nowhere.
__device__ __forceinline__ QueryRow query_row(const Unit& u, const UnitPlan& p, int head, int rho, int rows_end, int t1) {
  QueryRow q{0, -1, 0, 0x7fffffff};
  if (rho >= rows_end) return q;
  const int i = rho / p.group;
  q.r = u.begin + i;
  q.h = head * p.group + (rho - i * p.group);
  const int pos = u.length - u.n + i;
  q.first = p.window > 0 ? max(0, pos - p.window + 1) : 0;
  q.last = p.causal ? min(pos, t1 - 1) : t1 - 1;
  if (q.last < q.first) q.first = q.last = 0x7f000000;   // no position is there
  return q;
}

// Whether a row does not see position t.
__device__ __forceinline__ bool hidden(const QueryRow& q, int t) { return (uint32_t)(t - q.first) > (uint32_t)(q.last - q.first); }

// Eight consecutive values of a query row.  (Element alignment is enough for 16-byte accesses to global memory.)
template <bool BF16>
__device__ __forceinline__ void load8(const void* q, int64_t i, float (&v)[8]) {
  if constexpr (BF16) {
    u32x4 w;
    __builtin_memcpy(&w, static_cast<const uint16_t*>(q) + i, 16);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = bf16_lo(w[j]);
      v[2 * j + 1] = bf16_hi(w[j]);
    }
  } else {
    __builtin_memcpy(v, static_cast<const float*>(q) + i, 32);
  }
}

// The power of two that brings a row of maximum `top` into [2^14, 2^15), and the exponent of its inverse.
__device__ __forceinline__ void row_factors(float top, float& f, int& inverse) {
  const int e = max((int)(__float_as_uint(top) >> 23), 15);
  f = __uint_as_float((uint32_t)(268 - e) << 23);
  inverse = e - 141;
}

// A row's factor c is |scale| log2(e) (mantissa 2^exponent in AttendProblem) x the inverse of q's factor x
// the keys' (NVFP4: their tensor scale; MXFP4: a step's reference).  Products of some of them may leave
// float32's range where c does not, so it is put together from exponents and rounded once.

// What a lane keeps of its row's c: c itself, or (MXFP4, where the keys' reference joins in each step) an exponent.
template <bool MX>
using RowScale = std::conditional_t<MX, int, float>;

// c = mantissa 2^exponent, kept from 0 and infinity, whose products with -inf (a masked position) and 0 are
// NaN.  (Scores are sums of fp16 products, below 2^40: c of 1e-37 makes them 0.)
__device__ __forceinline__ float row_factor(float mantissa, int exponent) {
  return fminf(fmaxf(__builtin_amdgcn_ldexpf(mantissa, exponent), 1e-37f), 3e38f);
}
__device__ __forceinline__ float row_factor_nv(const AttendProblem& a, int inverse, float gk) {
  return row_factor(a.mantissa * __builtin_amdgcn_frexp_mantf(gk), a.exponent + inverse + __builtin_amdgcn_frexp_expf(gk));
}

// Two fp16 parts of eight float32 values (hi + lo, 22 bits); lo is left out where !SPLIT.
template <bool SPLIT>
__device__ __forceinline__ void to_f16(const float (&v)[8], f16x8& hi, f16x8& lo) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    hi[j] = (_Float16)v[j];
    if constexpr (SPLIT) lo[j] = (_Float16)(v[j] - (float)hi[j]);
  }
}

// Four consecutive output values.
__device__ __forceinline__ void store4(void* out, bool bf16, int64_t i, f32x4 v) {
  if (bf16) {
    const u32x2 w{bf16_pack2(v[0], v[1]), bf16_pack2(v[2], v[3])};
    __builtin_memcpy(static_cast<uint16_t*>(out) + i, &w, 8);
  } else {
    __builtin_memcpy(static_cast<float*>(out) + i, &v, 16);
  }
}

// 1 / l, by which a row's sums of P v are multiplied before the values' own unit is: P is up to 2^15, so the
// sums times the unit, or the unit / l, may leave float32's range where the result does not.  0 where l is
// (nothing was seen), NaN where l is.
__device__ __forceinline__ float inverse_of(float l) { return l == 0 ? 0.0f : 1.0f / l; }

// A part's results in the workspace: for each of its rows m and l, then the outputs [rows][DP] of
// its positions alone.
__device__ __forceinline__ float* part_of(const UnitPlan& p, int heads, int head, int part, int dp) {
  return p.parts + ((int64_t)part * heads + head) * p.rows * (dp + 2);
}

// The reference of a row's weights after a step whose largest exponent is `top`.  (The difference: m + kGrowth
// may round up to `top` where float32's steps are 8.  Where both are -inf it is NaN, and m stays.)
__device__ __forceinline__ float next_max(float m, float top) { return top - m > kGrowth ? top : m; }

// lse of a row with running maximum m and sum l: -inf where it saw nothing, NaN where l is.
__device__ __forceinline__ float row_lse(float m, float l) {
  return l == 0 ? -INFINITY : (m + __builtin_amdgcn_logf(l) - kWeightBits) * kLn2;
}

// Whether the parts of u's tile have room in the workspace (always, unless offsets decrease).
__device__ __forceinline__ bool has_room(const UnitPlan& p, const Unit& u) {
  return u.count == 1 || (u.part0 >= 0 && u.part0 + u.count <= p.max_parts);
}

// Records unit u's tile for k_join_parts (by the first part), and how many tiles there are.
__device__ __forceinline__ void note_tile(const UnitPlan& p, const Unit& u, int unit, int rows) {
  if (threadIdx.x != 0) return;
  if (unit == 0) static_cast<TileParts*>(p.tiles)[p.max_slots].begin = u.slots;
  if (u.any && u.part == 0 && u.slot >= 0 && u.slot < p.max_slots)
    static_cast<TileParts*>(p.tiles)[u.slot] = {u.begin, u.tile * p.rows, rows, u.part0, u.count, {0, 0, 0}};
}

}  // namespace fp4dev
