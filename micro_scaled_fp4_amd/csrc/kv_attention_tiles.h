// Attention for many query rows per sequence (prompts, prompt chunks): tiles of 128 packed rows.
//
// Each of the four waves holds 32 rows (a row is lane % 32 of the 32x32x16 MFMAs).  A step of 64
// positions is dequantized once for the workgroup into LDS as fp16 (wave w: positions 16 w ..
// 16 w + 15), into two buffers in turn: step n + 1's while step n is computed; one barrier ends a
// step.  Codes are loaded two steps ahead.
//
// Bound by the matrix and the vector instructions together: of a step at 128 channels a wave
// issues 32 MFMAs (about 1040 cycles) and 270 vector instructions (about 1350: half for the
// softmax, a quarter for its share of the dequantizing), and the two waves of a SIMD hardly overlap
// them (matrix units 43%, vector units 57% busy).  Causal prompts of 16384, TFLOP/s:
//                                    bf16: NVFP4  MXFP4   float32: NVFP4  MXFP4
//   32 / 8 heads x 64                    808      802          497      477
//   32 / 8 heads x 128                   957      972          562      591
//   8 / 4 heads x 256                    561      514          370      347
// 256 channels: sums and q fill 192 registers, one wave a SIMD; in float32, whose two parts of q and P make
// twice the MFMAs, 35 to 37 more registers spill.  In an earlier state (985 TFLOP/s at the prompt of
// 128 channels), 64 rows a wave at one wave a SIMD reached 722, eight waves over 256 rows 970, the next
// step's scores beside this step's weights 930, raised wave priorities 2% less.
#pragma once

#include <type_traits>

#include "kv_attention.h"
#include "kv_attention_few.h"

namespace fp4dev {

// Chunk (16 bytes: 8 channels) of row t of the keys' fp16 tile: 16 rows that lanes read together
// fall on different banks.
template <int DP>
__device__ __forceinline__ int k_chunk(int t, int chunk) { return DP == 64 ? chunk ^ ((t >> 1) & 7) : chunk ^ (t & 15); }

template <int DP, bool MX, bool QBF, bool SPLIT>
__global__ void __launch_bounds__(256, DP == 256 ? 1 : 2)
    k_attend_tiles(KvCache c, AttendProblem a, UnitPlan p) {
  constexpr int kDwords = DP / 32, kScales = DP == 256 ? 2 : 1, kSteps = DP / 16, kBlocks = DP / 32;
  // (objects of their own, so that the compiler sees which accesses can change places)
  __shared__ __align__(16) uint8_t k_even[64 * DP * 2], k_odd[64 * DP * 2], v_even[64 * DP * 2], v_odd[64 * DP * 2];
  __shared__ int tops[4][4][2];                 // MX: [round][wave][keys, values]
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r32 = lane & 31, half = lane >> 5;
  const int unit = workgroup() / c.heads, head = workgroup() % c.heads;
  const Unit u = unit_of<false>(c, p, unit);
  const int rows_end = min((u.tile + 1) * p.rows, u.n * p.group);
  const int rows = rows_end - u.tile * p.rows;
  if (head == 0) note_tile(p, u, unit, rows);
  if (!u.any || !has_room(p, u)) return;
  const Span sp = span_of(p, u, rows);

  // This wave's 16 positions of each step, and where they are in the cache.
  const QuarterRow<DP, MX> at(lane >> 2, lane & 3, c.dim);
  const int code_row = c.dim / 2, scale_row = c.dim / (MX ? 32 : 16);
  struct Raw {
    uint32_t kw[kDwords], vw[kDwords], ks[kScales], vs[kScales];
  };
  PageWalk walk(c, u.b, sp.t0);
  uint32_t holes = 0;                           // in a step: four bits of 16 positions each, of it and the next two
  int ahead = sp.t0;                            // the next step to load
  Raw near, far;                                // the next step, and the one after it
  auto load = [&](Raw& raw) {
    const int t = ahead + 16 * wave;
    walk.reach(ahead);
    int n = min(max(sp.t1 - t, 0), 16);
    int page = walk.at(t);
    if (page < 0) n = page = 0;
    const int64_t row = cache_row(c, page, head, t);
    const int codes = n * code_row, scales = n * scale_row;
    // what no row sees may be anything, a NaN or the largest scale too: scale bytes of 0 make it 0
    QuarterRow<DP, MX> seen = at;
#pragma unroll
    for (int j = 0; j < kScales; ++j) seen.scale[j] = t + (lane >> 2) < sp.lo ? kOutOfRange : at.scale[j];
    holes = holes >> 4 | walk.holes_at(ahead) << 8;   // (past the last position: masked anyway)
    load_quarter<DP, MX>(uniform_rsrc(c.k_codes + row * code_row, codes), uniform_rsrc(c.k_scales + row * scale_row, scales), seen,
                         raw.kw, raw.ks);
    load_quarter<DP, MX>(uniform_rsrc(c.v_codes + row * code_row, codes), uniform_rsrc(c.v_scales + row * scale_row, scales), seen,
                         raw.vw, raw.vs);
    ahead += 64;
  };
  // MX: this wave's largest scale bytes of a round, and all waves'
  auto note_tops = [&](const Raw& raw, int round) {
    if constexpr (MX) {
      int k = (int)raw.ks[0], v = (int)raw.vs[0];
      if constexpr (kScales == 2) k = max(k, (int)raw.ks[1]), v = max(v, (int)raw.vs[1]);
      k = wave_max_lanes(k);
      v = wave_max_lanes(v);
      if (lane == 0) {
        tops[round & 3][wave][0] = k;
        tops[round & 3][wave][1] = v;
      }
    }
  };
  int k_ref1 = 0, v_ref = 0, v_ref1 = 0;        // of the next step's keys; of the sums so far and the next step's values
  auto take_tops = [&](int round) {
    if constexpr (MX) {
      int k = 0, v = v_ref1;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        k = max(k, tops[round & 3][w][0]);
        v = max(v, tops[round & 3][w][1]);
      }
      k_ref1 = __builtin_amdgcn_readfirstlane(k);
      v_ref1 = __builtin_amdgcn_readfirstlane(v);
    }
  };
  auto dequantize = [&](const Raw& raw, uint8_t* k_tile, uint8_t* v_tile) {
    const int t = 16 * wave + (lane >> 2);
    uint8_t* const k = k_tile + t * (2 * DP);
    uint8_t* const v = v_tile + t * (2 * DP);
#pragma unroll
    for (int w = 0; w < kDwords; ++w) {
      const int chunk = (lane & 3) * kDwords + w;
      *reinterpret_cast<f16x8*>(k + 16 * k_chunk<DP>(t, chunk)) = quarter8<DP, MX>(raw.kw, raw.ks, w, k_ref1);
      *reinterpret_cast<f16x8*>(v + 32 * v_granule<DP>(t, chunk >> 1) + 16 * (chunk & 1)) = quarter8<DP, MX>(raw.vw, raw.vs, w, v_ref1);
    }
  };

  load(near);
  load(far);

  const float gk = MX ? 1.0f : nv_global_scale(*c.k_amax), gv = MX ? 1.0f : nv_global_scale(*c.v_amax);
  const QueryRow row = query_row(u, p, head, u.tile * p.rows + 32 * wave + r32, rows_end, sp.t1);
  f16x8 qh[kSteps], ql[SPLIT ? kSteps : 1];
  RowScale<MX> factor;                          // c: scores -> base-2 exponents (MX: its exponent but for the keys')
  {
    uint32_t top = 0;
    float v[8];
    auto read = [&](int i) {
      const int d = 16 * i + 8 * half;
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = 0;
      if (row.h >= 0 && d < c.dim) load8<QBF>(a.q, row.r * a.q_stride + (int64_t)row.h * c.dim + d, v);
    };
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      read(i);
#pragma unroll
      for (int j = 0; j < 8; ++j) top = umax(top, __float_as_uint(v[j]) & 0x7fffffffu);
    }
    float f;
    int inverse;
    row_factors(max_over_halves(__uint_as_float(top)), f, inverse);
    if constexpr (MX) factor = a.exponent + inverse - 140;
    else factor = row_factor_nv(a, inverse, gk);
    if (a.negative) f = -f;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      read(i);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= f;
      to_f16<SPLIT>(v, qh[i], ql[SPLIT ? i : 0]);
    }
  }

  // scores of the step in a buffer: S^T[position][row r32]; register e of block b: position
  // 32 b + 8 (e / 4) + 4 half + e % 4
  const int k_place = r32 * (2 * DP) + 16 * k_chunk<DP>(r32, half);   // chunk 2 i + half: ^ (32 i)
  auto scores = [&](const uint8_t* k_tile, f32x16 (&s)[2]) {
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int e = 0; e < 16; ++e) s[b][e] = 0;
#pragma unroll
    for (int i = 0; i < kSteps; ++i)
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const f16x8 k8 = *reinterpret_cast<const f16x8*>(k_tile + 32 * b * (2 * DP) + (k_place ^ (32 * i)));
        s[b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(k8, qh[i], s[b], 0, 0, 0);
        if constexpr (SPLIT) s[b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(k8, ql[i], s[b], 0, 0, 0);
      }
  };

  note_tops(near, 0);
  note_tops(far, 1);
  __syncthreads();
  take_tops(0);
  dequantize(near, k_even, v_even);
  __syncthreads();

  f32x16 acc[kBlocks];
#pragma unroll
  for (int d = 0; d < kBlocks; ++d)
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[d][e] = 0;
  float m = -INFINITY, l = 0;
  const int v_at0 = v_address<DP>(4 * half) ^ (32 * ((lane >> 4) & 1));
  int t0 = sp.t0, round = 2;
  // Step t0; near: the step to dequantize, far: the one to load.
  auto step = [&](auto odd, const Raw& near, Raw& far) {
    uint8_t* const k_now = odd.value ? k_odd : k_even;
    uint8_t* const k_next = odd.value ? k_even : k_odd;
    uint8_t* const v_now = odd.value ? v_odd : v_even;
    uint8_t* const v_next = odd.value ? v_even : v_odd;
    load(far);
    const int k_ref = k_ref1, v_top = v_ref1;
    take_tops(round - 1);
    f32x16 s[2];
    scores(k_now, s);
    float cf;
    if constexpr (MX) cf = row_factor(a.mantissa, factor + k_ref);
    else cf = factor;
    if ((holes & 15u) != 0 || __any(t0 + 63 > row.last || t0 < row.first)) {
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const bool hide = hidden(row, t0 + 32 * b + 8 * (e >> 2) + 4 * half + (e & 3)) | (holes >> (2 * b + (e >> 3)) & 1);
          s[b][e] = hide ? -INFINITY : s[b][e];
        }
    }
    float top = s[0][0];
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int e = 0; e < 16; ++e) top = fmaxf(top, s[b][e]);
    const float was = m;
    m = next_max(was, max_over_halves(top) * cf);
    const float base = m == -INFINITY ? 0.0f : m;
    const float drop = __builtin_amdgcn_exp2f(was - base);
    float shift = kWeightBits - base;
    if (__any(fabsf(base) > kExactSteps)) {
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int e = 0; e < 16; ++e) s[b][e] = s[b][e] * cf - base;
      cf = 1;
      shift = kWeightBits;
    }
    const float keep = MX ? __builtin_amdgcn_ldexpf(drop, v_ref - v_top) : drop;
    if (__any(keep != 1.0f)) {
      l *= drop;
#pragma unroll
      for (int d = 0; d < kBlocks; ++d) acc[d] *= keep;
    }
    v_ref = v_top;
    f16x8 ph[4], pl[SPLIT ? 4 : 1];
    float sum = 0;
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float w = __builtin_amdgcn_exp2f(__builtin_fmaf(s[b][e], cf, shift));
        sum += w;
        const _Float16 h = (_Float16)w;
        ph[2 * b + (e >> 3)][e & 7] = h;
        if constexpr (SPLIT) pl[2 * b + (e >> 3)][e & 7] = (_Float16)(w - (float)h);
      }
    l += sum;
    // O^T += V^T P^T: 16 positions at a time, in the order 4 half + 0 .. 3, 8 + 4 half + 0 .. 3
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int d = 0; d < kBlocks; ++d) {
        const uint8_t* const from = v_now + 16 * i * (2 * DP) + (v_at0 ^ (64 * d));
        const s16x4 x = read_v4(from), y = read_v4(from + 8 * 2 * DP);
        const f16x8 v8 = __builtin_bit_cast(f16x8, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
        acc[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v8, ph[i], acc[d], 0, 0, 0);
        if constexpr (SPLIT) acc[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v8, pl[i], acc[d], 0, 0, 0);
      }
    }
    dequantize(near, k_next, v_next);
    note_tops(far, round);
    t0 += 64;
    ++round;
    __syncthreads();
  };
  while (t0 < sp.t1) {
    step(std::integral_constant<int, 0>{}, far, near);
    if (t0 >= sp.t1) break;
    step(std::integral_constant<int, 1>{}, near, far);
  }

  const float unit_of_v = MX ? __builtin_amdgcn_ldexpf(1.0f, v_ref - 140) : gv;
  // register e of block d: channel 32 d + 8 (e / 4) + 4 half + e % 4 of row r32
  l = sum_over_halves(l);
  if (row.h < 0) return;
  const int q = 32 * wave + r32;
  float* const left = u.count > 1 ? part_of(p, c.heads, head, u.part0 + u.part, DP) : nullptr;
  const float inverse = inverse_of(l);
  const int64_t o = (row.r * a.q_heads + row.h) * c.dim;
#pragma unroll
  for (int d = 0; d < kBlocks; ++d) {
    if (32 * d >= c.dim) break;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const f32x4 v = f32x4{acc[d][4 * e], acc[d][4 * e + 1], acc[d][4 * e + 2], acc[d][4 * e + 3]} * inverse * unit_of_v;
      const int channel = 32 * d + 8 * e + 4 * half;
      if (left != nullptr) *reinterpret_cast<f32x4*>(left + 2 * p.rows + q * DP + channel) = v;
      else store4(a.out, a.out_bf16, o + channel, v);
    }
  }
  if (half != 0) return;
  if (left != nullptr) {
    left[2 * q] = m;
    left[2 * q + 1] = l;
  } else if (a.lse != nullptr) {
    a.lse[row.r * a.q_heads + row.h] = row_lse(m, l);
  }
}

}  // namespace fp4dev
