// Attention for few query rows per sequence (decoding, drafts): tiles of 16 R packed rows.
//
// The four waves of a workgroup take turns at the part's steps of 64 positions, each for all of
// the tile's rows, and join their results at the end: nothing is waited for in between.  Keys go
// from memory straight into the MFMA's A operand: lane (t = lane % 16, quad) loads a quarter of
// position t's row, and Q's registers hold the channels in the same order.  Values pass through
// LDS as fp16, 32 positions at a time, private to the wave, and come back transposed
// (ds_read_b64_tr_b16), four positions of one channel to a lane.  The next step's bytes are
// loaded while this one is computed.
//
// Bound by HBM bytes where contexts are long: 1000000 positions, 8 heads x 128, 4 query heads
// each: 227 us NVFP4, 214 us MXFP4 with the join of the parts (5.08 and 5.07 TB/s), 64 sequences of
// 16384 with 8 query heads each 247 us (4.9 TB/s).  R = 2 is bound by waits: 25 packed rows of 8 heads x 128
// over 16 sequences of 2500 to 9001 positions 36 us (2.6 TB/s), vector units 39% and matrix units 10%
// busy; its waves, 1.4 a SIMD on average, wait 40% of their cycles.  Short contexts pay the chain of a part:
// 2.6 us until its unit is known, 1.9 the first loads, 2.0 a step, 0.8 the join of the waves (1000
// positions, a step a wave: 9 us).  Unrolling over two steps needs more registers than two waves a SIMD
// leave (32 sequences, 51 -> 61 us).
#pragma once

#include "kv_attention.h"

namespace fp4dev {

// Scale bytes and codes of 64 positions as a lane holds them.
template <int DP>
struct RawStep {
  static constexpr int kDwords = DP / 32, kScales = DP == 256 ? 2 : 1;
  uint32_t k[4][kDwords], v[4][kDwords], ks[4][kScales], vs[4][kScales];
  int holes;                     // bit i: positions 16 i .. 16 i + 15 are in a hole
};

// Byte offsets of a lane's quarter row `part` of position t among 16 rows of codes and scales.
template <int DP, bool MX>
struct QuarterRow {
  static constexpr int kChunks = DP == 256 ? 2 : 1;
  int code[kChunks], scale[kChunks];
  __device__ __forceinline__ QuarterRow(int t, int part, int dim) {
#pragma unroll
    for (int j = 0; j < kChunks; ++j) {
      const int d = part * (DP / 4) + 32 * j;
      code[j] = d < dim ? t * (dim / 2) + d / 2 : kOutOfRange;
      scale[j] = d < dim ? (MX ? t * (dim / 32) + d / 32 : t * (dim / 16) + d / 16) : kOutOfRange;
    }
  }
};

// A lane's quarter row.
template <int DP, bool MX>
__device__ __forceinline__ void load_quarter(__amdgpu_buffer_rsrc_t codes, __amdgpu_buffer_rsrc_t scales,
                                             const QuarterRow<DP, MX>& at, uint32_t (&w)[DP / 32],
                                             uint32_t (&s)[DP == 256 ? 2 : 1]) {
  if constexpr (DP == 64) {
    const u32x2 x = __builtin_amdgcn_raw_buffer_load_b64(codes, at.code[0], 0, 0);
    w[0] = x[0];
    w[1] = x[1];
  } else {
#pragma unroll
    for (int j = 0; j < DP / 128; ++j) {
      const u32x4 x = __builtin_amdgcn_raw_buffer_load_b128(codes, at.code[j], 0, 0);
#pragma unroll
      for (int e = 0; e < 4; ++e) w[4 * j + e] = x[e];
    }
  }
#pragma unroll
  for (int j = 0; j < (DP == 256 ? 2 : 1); ++j) {
    if constexpr (MX || DP == 64) s[j] = __builtin_amdgcn_raw_buffer_load_b8(scales, at.scale[j], 0, 0);
    else s[j] = __builtin_amdgcn_raw_buffer_load_b16(scales, at.scale[j], 0, 0);
  }
}

// Dword i of a quarter row as fp16 (MX: relative to scale byte `ref`).
template <int DP, bool MX>
__device__ __forceinline__ f16x8 quarter8(const uint32_t (&w)[DP / 32], const uint32_t (&s)[DP == 256 ? 2 : 1], int i, int ref) {
  if constexpr (MX) {
    return mx8(w[i], mx_factor(s[DP == 256 ? i / 4 : 0], ref));
  } else {
    const f16x2 h = e4m3_pair_h<false>(s[DP == 256 ? i / 4 : 0]);
    const _Float16 b = (i >> 1) & 1 ? h.y : h.x;
    return dq8(w[i], f16x2{b, b});
  }
}

// Orders a wave's own LDS accesses (which the LDS unit takes in order) for the compiler.
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Granule (32 bytes: 16 channels) of row t of a [.][DP] fp16 tile in LDS: rows that a transposed
// read takes together fall on different granules.  (Stores do conflict: all lanes of one write the same half of
// their granules, so half of the banks.  Conflicts are 35% of the LDS cycles here and 40% in the tiles of
// 128 rows, where waves wait for LDS 7% of their cycles.)
template <int DP>
__device__ __forceinline__ int v_granule(int t, int g) { return DP == 64 ? g ^ ((t >> 1) & 3) : g ^ (t & 7); }

// Where a lane points for a transposed read of granule 0 of rows t .. t + 3 (t a multiple of 4):
// lane i of each 16 at row t + i / 4.  Granule g is at this ^ (32 g), and 8 rows further on the
// same lane's place is 8 rows further on.
template <int DP>
__device__ __forceinline__ int v_address(int t) {
  const int i = threadIdx.x & 15, row = t + (i >> 2);
  return row * (2 * DP) + 32 * v_granule<DP>(row, 0) + 8 * (i & 3);
}

// Four positions of a channel: lane i of each 16 gets channel i of the granule.
__device__ __forceinline__ s16x4 read_v4(const uint8_t* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)p);
}

template <int DP, bool MX, bool QBF, bool SPLIT, int R>
__global__ void __launch_bounds__(256, DP == 256 ? 1 : 2)
    k_attend_few(KvCache c, AttendProblem a, UnitPlan p) {
  constexpr int kDwords = DP / 32, kGranules = DP / 16;
  __shared__ __align__(16) uint8_t tile[4][32 * DP * 2];
  __shared__ float stats[4][16][2];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, quad = lane >> 4;
  const int unit = workgroup() / c.heads, head = workgroup() % c.heads;
  const float gk = MX ? 1.0f : nv_global_scale(*c.k_amax), gv = MX ? 1.0f : nv_global_scale(*c.v_amax);
  const Unit u = unit_of<true>(c, p, unit);
  const int rows_end = min((u.tile + 1) * p.rows, u.n * p.group);
  if (head == 0) note_tile(p, u, unit, rows_end - u.tile * p.rows);
  if (!u.any || !has_room(p, u)) return;
  const Span sp = span_of(p, u, rows_end - u.tile * p.rows);

  const QuarterRow<DP, MX> k_at(r16, quad, c.dim), v_at(lane >> 2, lane & 3, c.dim);
  RawStep<DP> next;
  int t0 = sp.t0 + 64 * wave;
  PageWalk walk(c, u.b, t0);
  auto load = [&](int t0) {
    walk.reach(t0);
    next.holes = walk.holes_at(t0);              // (past the last position: masked anyway)
    const int codes = c.dim / 2, scales = c.dim / (MX ? 32 : 16);
    // 16 positions at a time; pages of 64 and more positions hold the whole step
    const bool whole = c.page_shift >= 6;
    int64_t codes_at = 0, scales_at = 0;
    int page = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = t0 + 16 * i;
      if (i == 0 || !whole) {
        page = walk.at(t);
        const int64_t row = cache_row(c, max(page, 0), head, t);
        codes_at = row * codes;
        scales_at = row * scales;
      } else {
        codes_at += 16 * codes;
        scales_at += 16 * scales;
      }
      const int n = page < 0 ? 0 : min(max(sp.t1 - t, 0), 16);
      load_quarter<DP, MX>(uniform_rsrc(c.k_codes + codes_at, n * codes), uniform_rsrc(c.k_scales + scales_at, n * scales), k_at,
                           next.k[i], next.ks[i]);
      load_quarter<DP, MX>(uniform_rsrc(c.v_codes + codes_at, n * codes), uniform_rsrc(c.v_scales + scales_at, n * scales), v_at,
                           next.v[i], next.vs[i]);
    }
  };
  if (t0 < sp.t1) load(t0);

  f16x8 qh[R][kDwords], ql[R][SPLIT ? kDwords : 1];
  RowScale<MX> factor[R];                       // c: scores -> base-2 exponents (MX: its exponent but for the keys')
  QueryRow row[R];
#pragma unroll
  for (int g = 0; g < R; ++g) {
    row[g] = query_row(u, p, head, u.tile * p.rows + 16 * g + r16, rows_end, sp.t1);
    float v[kDwords][8];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kDwords; ++i) {
      const int d = quad * (DP / 4) + 8 * i;
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0;
      if (row[g].h >= 0 && d < c.dim) load8<QBF>(a.q, row[g].r * a.q_stride + (int64_t)row[g].h * c.dim + d, v[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) top = umax(top, __float_as_uint(v[i][j]) & 0x7fffffffu);
    }
    float f;
    int inverse;
    row_factors(max_over_halves(max_over_rows(__uint_as_float(top))), f, inverse);
    if constexpr (MX) factor[g] = a.exponent + inverse - 140;
    else factor[g] = row_factor_nv(a, inverse, gk);
    if (a.negative) f = -f;
#pragma unroll
    for (int i = 0; i < kDwords; ++i) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] *= f;
      to_f16<SPLIT>(v[i], qh[g][i], ql[g][SPLIT ? i : 0]);
    }
  }

  f32x4 acc[R][kGranules];
  float m[R], l[R];
#pragma unroll
  for (int g = 0; g < R; ++g) {
    m[g] = -INFINITY;
    l[g] = 0;
#pragma unroll
    for (int d = 0; d < kGranules; ++d) acc[g][d] = f32x4{0, 0, 0, 0};
  }
  int v_ref = 0;
  uint8_t* mine = tile[wave];
  const int v_at0 = v_address<DP>(4 * quad);

  for (; t0 < sp.t1; t0 += 256) {
    RawStep<DP> now = next;
    if (t0 + 256 < sp.t1) load(t0 + 256);
    if (t0 < sp.lo) {
      // what no row sees may be anything, a NaN or the largest scale too: scale bytes of 0 make it 0
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < RawStep<DP>::kScales; ++j) {
          now.ks[i][j] = t0 + 16 * i + r16 < sp.lo ? 0 : now.ks[i][j];
          now.vs[i][j] = t0 + 16 * i + (lane >> 2) < sp.lo ? 0 : now.vs[i][j];
        }
    }
    int k_ref = 0, v_top = 0;
    if constexpr (MX) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < RawStep<DP>::kScales; ++j) {
          k_ref = max(k_ref, (int)now.ks[i][j]);
          v_top = max(v_top, (int)now.vs[i][j]);
        }
      k_ref = wave_max_lanes(k_ref);
      v_top = max(wave_max_lanes(v_top), v_ref);
    }
    // scores: S^T[t = 16 i + 4 quad + e][row r16]
    f32x4 s[R][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int g = 0; g < R; ++g) s[g][i] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int w = 0; w < kDwords; ++w) {
        const f16x8 k8 = quarter8<DP, MX>(now.k[i], now.ks[i], w, k_ref);
#pragma unroll
        for (int g = 0; g < R; ++g) {
          s[g][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k8, qh[g][w], s[g][i], 0, 0, 0);
          if constexpr (SPLIT) s[g][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k8, ql[g][w], s[g][i], 0, 0, 0);
        }
      }
    }
    f16x8 ph[R][2], pl[R][SPLIT ? 2 : 1];
#pragma unroll
    for (int g = 0; g < R; ++g) {
      float cf;
      if constexpr (MX) cf = row_factor(a.mantissa, factor[g] + k_ref);
      else cf = factor[g];
      if (now.holes != 0 || __any(t0 + 63 > row[g].last || t0 < row[g].first)) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const bool hide = hidden(row[g], t0 + 16 * i + 4 * quad + e) | (now.holes >> i & 1);
            s[g][i][e] = hide ? -INFINITY : s[g][i][e];
          }
      }
      float top = s[g][0][0];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) top = fmaxf(top, s[g][i][e]);
      top = max_over_halves(max_over_rows(top));
      const float was = m[g];
      m[g] = next_max(was, top * cf);
      const float base = m[g] == -INFINITY ? 0.0f : m[g];
      const float drop = __builtin_amdgcn_exp2f(was - base);
      float shift = kWeightBits - base;
      if (__any(fabsf(base) > kExactSteps)) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[g][i][e] = s[g][i][e] * cf - base;
        cf = 1;
        shift = kWeightBits;
      }
      float sum = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float w = __builtin_amdgcn_exp2f(__builtin_fmaf(s[g][i][e], cf, shift));
          sum += w;
          const _Float16 h = (_Float16)w;
          ph[g][i >> 1][4 * (i & 1) + e] = h;
          if constexpr (SPLIT) pl[g][i >> 1][4 * (i & 1) + e] = (_Float16)(w - (float)h);
        }
      const float keep = MX ? __builtin_amdgcn_ldexpf(drop, v_ref - v_top) : drop;
      if (__any(keep != 1.0f)) {
        l[g] *= drop;
#pragma unroll
        for (int d = 0; d < kGranules; ++d) acc[g][d] *= keep;
      }
      l[g] += sum;
    }
    v_ref = v_top;
    // outputs: O^T[channel][row r16] += V^T P^T, 32 positions at a time
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int t = 16 * i + (lane >> 2);
#pragma unroll
        for (int w = 0; w < kDwords; ++w) {
          const int chunk = (lane & 3) * kDwords + w;
          *reinterpret_cast<f16x8*>(mine + t * (2 * DP) + 32 * v_granule<DP>(t, chunk >> 1) + 16 * (chunk & 1)) =
              quarter8<DP, MX>(now.v[2 * h + i], now.vs[2 * h + i], w, v_ref);
        }
      }
      wave_lds_fence();
#pragma unroll
      for (int d = 0; d < kGranules; ++d) {
        const uint8_t* const from = mine + (v_at0 ^ (32 * d));
        const s16x4 x = read_v4(from), y = read_v4(from + 16 * 2 * DP);
        const f16x8 v8 = __builtin_bit_cast(f16x8, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
#pragma unroll
        for (int g = 0; g < R; ++g) {
          acc[g][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v8, ph[g][h], acc[g][d], 0, 0, 0);
          if constexpr (SPLIT) acc[g][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v8, pl[g][h], acc[g][d], 0, 0, 0);
        }
      }
      wave_lds_fence();
    }
  }

  // the waves' results, joined row group by row group; thread (q, c16) takes channels of row q
  const int q = threadIdx.x >> 4, c16 = threadIdx.x & 15;
#pragma unroll
  for (int g = 0; g < R; ++g) {
    __syncthreads();
    const float sum = sum_over_halves(sum_over_rows(l[g]));
    const float unit_of_v = MX ? __builtin_amdgcn_ldexpf(1.0f, v_ref - 140) : gv;
    const float inverse = inverse_of(sum);
    float* const whole = reinterpret_cast<float*>(&tile[0][0]);        // [wave][16 rows][DP]
#pragma unroll
    for (int d = 0; d < kGranules; ++d)
      *reinterpret_cast<f32x4*>(whole + (wave * 16 + r16) * DP + 4 * ((4 * d + quad) ^ r16)) = acc[g][d] * inverse * unit_of_v;
    if (quad == 0) {
      stats[wave][r16][0] = m[g];
      stats[wave][r16][1] = sum;
    }
    __syncthreads();
    const QueryRow out = query_row(u, p, head, u.tile * p.rows + 16 * g + q, rows_end, sp.t1);
    if (out.h < 0) continue;
    float top = -INFINITY, total = 0, part[4];
#pragma unroll
    for (int w = 0; w < 4; ++w) top = fmaxf(top, stats[w][q][0]);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      part[w] = stats[w][q][1] * __builtin_amdgcn_exp2f(stats[w][q][0] - (top == -INFINITY ? 0.0f : top));
      total += part[w];
    }
    const float of_total = inverse_of(total);
#pragma unroll
    for (int w = 0; w < 4; ++w) part[w] *= of_total;
    float* const left = u.count > 1 ? part_of(p, c.heads, head, u.part0 + u.part, DP) : nullptr;
    const int64_t o = (out.r * a.q_heads + out.h) * c.dim;
#pragma unroll
    for (int j = 0; j < DP / 64; ++j) {
      const int chunk = c16 + 16 * j;
      if (4 * chunk >= c.dim) break;
      f32x4 sumv{0, 0, 0, 0};
#pragma unroll
      for (int w = 0; w < 4; ++w) sumv += *reinterpret_cast<const f32x4*>(whole + (w * 16 + q) * DP + 4 * (chunk ^ q)) * part[w];
      if (left != nullptr) *reinterpret_cast<f32x4*>(left + 2 * p.rows + (16 * g + q) * DP + 4 * chunk) = sumv;
      else store4(a.out, a.out_bf16, o + 4 * chunk, sumv);
    }
    if (c16 == 0) {
      if (left != nullptr) {
        left[2 * (16 * g + q)] = top;
        left[2 * (16 * g + q) + 1] = total;
      } else if (a.lse != nullptr) {
        a.lse[out.r * a.q_heads + out.h] = row_lse(top, total);
      }
    }
  }
}

}  // namespace fp4dev
