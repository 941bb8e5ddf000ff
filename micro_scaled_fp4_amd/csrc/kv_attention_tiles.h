// Attention for many query rows per sequence (prompts, prompt chunks): tiles of 128 packed rows.
//
// Each of the four waves holds 32 rows (a row is lane % 32 of the 32x32x16 MFMAs).  A step of 64
// positions is dequantized once for the workgroup into LDS as fp16 (wave w: positions 16 w ..
// 16 w + 15), double-buffered: while a step is computed the next one's codes, already in
// registers, wait; they are dequantized into the other buffer at the step's end, behind which
// stands the loop's only barrier.
#pragma once

#include "kv_attention.h"
#include "kv_attention_few.h"

namespace fp4dev {

// Chunk (16 bytes: 8 channels) of row t of the keys' fp16 tile: 16 rows that lanes read together
// fall on different banks.
template <int DP>
__device__ __forceinline__ int k_chunk(int t, int chunk) { return DP == 64 ? chunk ^ ((t >> 1) & 7) : chunk ^ (t & 15); }

template <int DP>
struct StepBuffer {
  uint8_t k[64 * DP * 2], v[64 * DP * 2];
};

template <int DP, bool MX, bool QBF, bool SPLIT>
__global__ void __launch_bounds__(256, DP == 256 ? 1 : 2)
    k_attend_tiles(KvCache c, AttendProblem a, UnitPlan p, bool q_vec, bool out_vec) {
  constexpr int kDwords = DP / 32, kScales = DP == 256 ? 2 : 1, kSteps = DP / 16, kBlocks = DP / 32;
  __shared__ __align__(16) StepBuffer<DP> buffer[2];
  __shared__ int tops[16];                      // MX: [2][4 waves][keys, values]
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r32 = lane & 31, half = lane >> 5;
  const int unit = workgroup() / c.heads, head = workgroup() % c.heads;
  const Unit u = unit_of(c, p, unit);
  const int rows_end = min((u.tile + 1) * p.rows, u.n * p.group);
  const int rows = rows_end - u.tile * p.rows;
  if (head == 0) note_tile(p, u, unit, rows);
  if (!u.any || !has_room(p, u)) return;
  const Span sp = span_of(p, u, rows);

  // codes of the step after this one, scales of the one after that
  const QuarterRow<DP, MX> at(lane >> 2, lane & 3, c.dim);
  uint32_t kw[kDwords], vw[kDwords], ks[kScales], vs[kScales], ks2[kScales], vs2[kScales];
  int holes = 0, holes_next = 0;                // of 16 positions each
  PageWalk walk(c, u.b, sp.t0), walk2 = walk;   // along the codes, and one step ahead along the scales
  auto load = [&](int t0, bool codes) {
    const int t = t0 + 16 * wave;
    int n = min(max(sp.t1 - t, 0), 16);
    (codes ? walk : walk2).reach(t0);
    int page = (codes ? walk : walk2).at(t);
    if (page < 0) n = page = 0;
    const int64_t row = cache_row(c, page, head, t);
    const int cb = c.dim / 2, sb = c.dim / (MX ? 32 : 16);
    if (codes) {
      const __amdgpu_buffer_rsrc_t rk = uniform_rsrc(c.k_codes + row * cb, n * cb), rv = uniform_rsrc(c.v_codes + row * cb, n * cb);
      if constexpr (DP == 64) {
        const u32x2 x = __builtin_amdgcn_raw_buffer_load_b64(rk, at.code[0], 0, 0), y = __builtin_amdgcn_raw_buffer_load_b64(rv, at.code[0], 0, 0);
        kw[0] = x[0], kw[1] = x[1], vw[0] = y[0], vw[1] = y[1];
      } else {
#pragma unroll
        for (int j = 0; j < DP / 128; ++j) {
          const u32x4 x = __builtin_amdgcn_raw_buffer_load_b128(rk, at.code[j], 0, 0), y = __builtin_amdgcn_raw_buffer_load_b128(rv, at.code[j], 0, 0);
#pragma unroll
          for (int e = 0; e < 4; ++e) kw[4 * j + e] = x[e], vw[4 * j + e] = y[e];
        }
      }
    } else {
      const __amdgpu_buffer_rsrc_t rk = uniform_rsrc(c.k_scales + row * sb, n * sb), rv = uniform_rsrc(c.v_scales + row * sb, n * sb);
#pragma unroll
      for (int j = 0; j < kScales; ++j) {
        if constexpr (MX || DP == 64) {
          ks2[j] = __builtin_amdgcn_raw_buffer_load_b8(rk, at.scale[j], 0, 0);
          vs2[j] = __builtin_amdgcn_raw_buffer_load_b8(rv, at.scale[j], 0, 0);
        } else {
          ks2[j] = __builtin_amdgcn_raw_buffer_load_b16(rk, at.scale[j], 0, 0);
          vs2[j] = __builtin_amdgcn_raw_buffer_load_b16(rv, at.scale[j], 0, 0);
        }
      }
    }
  };
  // of the step whose codes were loaded last (past the last position: masked anyway)
  auto holes_at = [&](int t0) {
    int h = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) h |= walk.at(t0 + 16 * i) < 0 ? 1 << i : 0;
    return h;
  };
  // MX: this wave's largest scale bytes of the step whose scales are in ks2, vs2
  auto note_tops = [&](int parity) {
    if constexpr (MX) {
      int k = (int)ks2[0], v = (int)vs2[0];
      if constexpr (kScales == 2) k = max(k, (int)ks2[1]), v = max(v, (int)vs2[1]);
      k = wave_max_lanes(k);
      v = wave_max_lanes(v);
      if (lane == 0) {
        tops[(parity * 4 + wave) * 2] = k;
        tops[(parity * 4 + wave) * 2 + 1] = v;
      }
    }
  };
  int v_ref = 0, k_ref_next = 0, v_ref_next = 0;
  auto take_tops = [&](int parity) {
    if constexpr (MX) {
      k_ref_next = 0;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        k_ref_next = max(k_ref_next, tops[(parity * 4 + w) * 2]);
        v_ref_next = max(v_ref_next, tops[(parity * 4 + w) * 2 + 1]);
      }
      k_ref_next = __builtin_amdgcn_readfirstlane(k_ref_next);
      v_ref_next = __builtin_amdgcn_readfirstlane(v_ref_next);
    }
  };
  auto scales_arrive = [&]() {
#pragma unroll
    for (int j = 0; j < kScales; ++j) ks[j] = ks2[j], vs[j] = vs2[j];
  };
  auto dequantize = [&](int into) {
    const int t = 16 * wave + (lane >> 2);
    uint8_t* const k = buffer[into].k + t * (2 * DP);
    uint8_t* const v = buffer[into].v + t * (2 * DP);
#pragma unroll
    for (int w = 0; w < kDwords; ++w) {
      const int chunk = (lane & 3) * kDwords + w;
      *reinterpret_cast<f16x8*>(k + 16 * k_chunk<DP>(t, chunk)) = quarter8<DP, MX>(kw, ks, w, k_ref_next);
      *reinterpret_cast<f16x8*>(v + 32 * v_granule<DP>(t, chunk >> 1) + 16 * (chunk & 1)) = quarter8<DP, MX>(vw, vs, w, v_ref_next);
    }
  };

  // first step into buffer 0, its successor's codes and scales on their way
  load(sp.t0, false);
  load(sp.t0, true);

  const float gk = MX ? 1.0f : nv_global_scale(*c.k_amax), gv = MX ? 1.0f : nv_global_scale(*c.v_amax);
  const QueryRow row = query_row(u, p, head, u.tile * p.rows + 32 * wave + r32, rows_end, sp.t1);
  f16x8 qh[kSteps], ql[SPLIT ? kSteps : 1];
  float factor;
  {
    uint32_t top = 0;
    float v[8];
    auto read = [&](int i) {
      const int d = 16 * i + 8 * half;
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = 0;
      if (row.h >= 0 && d < c.dim) load8<QBF>(a.q, row.r * a.q_stride + (int64_t)row.h * c.dim + d, q_vec, v);
    };
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      read(i);
#pragma unroll
      for (int j = 0; j < 8; ++j) top = umax(top, __float_as_uint(v[j]) & 0x7fffffffu);
    }
    float f, inverse;
    row_factors(max_over_halves(__uint_as_float(top)), f, inverse);
    factor = fmaxf(fabsf(a.scale) * kLog2e * inverse * gk, 1e-37f);
    if (a.scale < 0) f = -f;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      read(i);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= f;
      to_f16<SPLIT>(v, qh[i], ql[SPLIT ? i : 0]);
    }
  }

  note_tops(0);
  scales_arrive();
  load(sp.t0 + 64, false);
  __syncthreads();
  take_tops(0);
  dequantize(0);
  holes = holes_at(sp.t0);
  load(sp.t0 + 64, true);
  holes_next = holes_at(sp.t0 + 64);
  note_tops(1);
  __syncthreads();

  f32x16 acc[kBlocks];
#pragma unroll
  for (int d = 0; d < kBlocks; ++d)
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[d][e] = 0;
  float m = -INFINITY, l = 0;

  int now = 0;
  for (int t0 = sp.t0; t0 < sp.t1; t0 += 64, now ^= 1) {
    // k_ref_next, v_ref_next: this step's references; the next step's scales are in ks2, vs2
    const int k_ref = k_ref_next, v_top = v_ref_next;
    const bool more = t0 + 64 < sp.t1;
    scales_arrive();
    if (more) load(t0 + 128, false);
    // a wave whose rows all end before this step only takes part in what the workgroup shares
    if (__any(t0 <= row.last && t0 + 63 >= row.first)) {
      const uint8_t* const kt = buffer[now].k;
      const uint8_t* const vt = buffer[now].v;
      f32x16 s[2];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
#pragma unroll
        for (int e = 0; e < 16; ++e) s[b][e] = 0;
        const int t = 32 * b + r32;
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          const f16x8 k8 = *reinterpret_cast<const f16x8*>(kt + t * (2 * DP) + 16 * k_chunk<DP>(t, 2 * i + half));
          s[b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(k8, qh[i], s[b], 0, 0, 0);
          if constexpr (SPLIT) s[b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(k8, ql[i], s[b], 0, 0, 0);
        }
      }
      const float cf = MX ? fmaxf(__builtin_amdgcn_ldexpf(factor, k_ref - 140), 1e-37f) : factor;
      // register e of block b: position 32 b + 8 (e / 4) + 4 half + e % 4
      if (holes != 0 || __any(t0 + 63 > row.last || t0 < row.first)) {
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int o = 32 * b + 8 * (e >> 2) + 4 * half + (e & 3);
            if (t0 + o > row.last || t0 + o < row.first || (holes >> (2 * b + (e >> 3)) & 1)) s[b][e] = -INFINITY;
          }
      }
      float top = s[0][0];
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int e = 0; e < 16; ++e) top = fmaxf(top, s[b][e]);
      top = max_over_halves(top);
      const float was = m;
      m = next_max(was, top * cf);
      const float base = m == -INFINITY ? 0.0f : m;
      const float drop = __builtin_amdgcn_exp2f(was - base);
      f16x8 ph[4], pl[SPLIT ? 4 : 1];
      float sum = 0;
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float w = __builtin_amdgcn_exp2f(__builtin_fmaf(s[b][e], cf, kWeightBits - base));
          sum += w;
          const _Float16 h = (_Float16)w;
          ph[2 * b + (e >> 3)][e & 7] = h;
          if constexpr (SPLIT) pl[2 * b + (e >> 3)][e & 7] = (_Float16)(w - (float)h);
        }
      const float keep = MX ? __builtin_amdgcn_ldexpf(drop, v_ref - v_top) : drop;
      if (__any(keep != 1.0f)) {
        l *= drop;
#pragma unroll
        for (int d = 0; d < kBlocks; ++d) acc[d] *= keep;
      }
      l += sum;
      v_ref = v_top;
      // O^T += V^T P^T: 16 positions at a time, in the order 4 half + 0 .. 3, 8 + 4 half + 0 .. 3
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int d = 0; d < kBlocks; ++d) {
          const int g = 2 * d + ((lane >> 4) & 1);
          const s16x4 x = read_v4<DP>(vt, 16 * i + 4 * half, g), y = read_v4<DP>(vt, 16 * i + 8 + 4 * half, g);
          const f16x8 v8 = __builtin_bit_cast(f16x8, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
          acc[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v8, ph[i], acc[d], 0, 0, 0);
          if constexpr (SPLIT) acc[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v8, pl[i], acc[d], 0, 0, 0);
        }
      }
    }
    if (more) {
      take_tops(now ^ 1);
      dequantize(now ^ 1);
      load(t0 + 128, true);
      holes = holes_next;
      holes_next = holes_at(t0 + 128);
    }
    // the step after the next one's references, for the end of the next step
    note_tops(now);
    __syncthreads();
  }

  // register e of block d: channel 32 d + 8 (e / 4) + 4 half + e % 4 of row r32
  l = sum_over_halves(l);
  if (row.h < 0) return;
  const float unit_of_v = MX ? __builtin_amdgcn_ldexpf(1.0f, v_ref - 140) : gv;
  if (u.count > 1) {
    float* const left = part_of(p, c.heads, head, u.part0 + u.part, DP);
    const int q = 32 * wave + r32;
#pragma unroll
    for (int d = 0; d < kBlocks; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (32 * d < c.dim)
          *reinterpret_cast<f32x4*>(left + 2 * p.rows + q * DP + 32 * d + 8 * e + 4 * half) =
              f32x4{acc[d][4 * e], acc[d][4 * e + 1], acc[d][4 * e + 2], acc[d][4 * e + 3]} * unit_of_v;
    if (half == 0) {
      left[2 * q] = m;
      left[2 * q + 1] = l;
    }
    return;
  }
  const float inverse = l > 0 ? 1.0f / l : 0.0f;
  const int64_t o = (row.r * a.q_heads + row.h) * c.dim;
#pragma unroll
  for (int d = 0; d < kBlocks; ++d)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (32 * d < c.dim)
        store4(a.out, a.out_bf16, out_vec, o + 32 * d + 8 * e + 4 * half,
               f32x4{acc[d][4 * e], acc[d][4 * e + 1], acc[d][4 * e + 2], acc[d][4 * e + 3]} * unit_of_v * inverse);
  if (half == 0 && a.lse != nullptr) a.lse[row.r * a.q_heads + row.h] = row_lse(m, l);
}

}  // namespace fp4dev
