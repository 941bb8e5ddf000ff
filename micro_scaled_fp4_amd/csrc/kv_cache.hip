// Writing and reading a paged key/value cache in FP4 (include/fp4.h, kv_cache_write
// and kv_cache_read).
//
// A wave takes one row of the call, k and v, all heads: it finds the row's sequence and
// page once, then its lanes take the row's values in order.
//   Write: a lane quantizes 16 values, an NVFP4 block; two lanes share an MXFP4 block and
//   its maximum.  The steps are those of nvfp4_quantize and mxfp4_quantize, bit for bit.
//   Read: a lane dequantizes 8 values (one dword of codes) and stores 16 bytes of bf16.
// Both are bound by HBM bytes (a row of 8 heads x 128 bf16 channels moves 4096 bytes one
// way and 1152 the other).
#include "fp4_device.h"
#include "fp4_internal.h"
#include "grid.h"
#include "kv_cache.h"

using namespace fp4dev;
using fp4impl::KvCache;

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

// N consecutive values from x + i.  VEC: x + i is 16-byte aligned.
template <bool BF16, bool VEC, int N>
__device__ __forceinline__ void load_values(const void* x, int64_t i, float (&v)[N]) {
  if constexpr (BF16) {
    const uint16_t* p = static_cast<const uint16_t*>(x) + i;
    if constexpr (VEC) {
#pragma unroll
      for (int j = 0; j < N / 8; ++j) {
        const u32x4 w = reinterpret_cast<const u32x4*>(p)[j];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[8 * j + 2 * e] = bf16_lo(w[e]);
          v[8 * j + 2 * e + 1] = bf16_hi(w[e]);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j) v[j] = __uint_as_float((uint32_t)p[j] << 16);
    }
  } else {
    const float* p = static_cast<const float*>(x) + i;
    if constexpr (VEC) {
#pragma unroll
      for (int j = 0; j < N / 4; ++j) {
        const f32x4 w = reinterpret_cast<const f32x4*>(p)[j];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[4 * j + e] = w[e];
      }
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j) v[j] = p[j];
    }
  }
}

template <bool MX, bool BF16, bool VEC>
__device__ __forceinline__ void write_row(const KvCache& c, const void* x, int64_t at, uint8_t* codes,
                                          uint8_t* scales, float s_global, int page, int t) {
  const int lane = threadIdx.x & 63, units = c.heads * c.dim >> 4, per_head = c.dim >> 4;
  for (int u0 = 0; u0 < units; u0 += 64) {
    const int u = u0 + lane;                    // units is even: an MXFP4 block's two lanes stay together
    if (u >= units) break;
    const int head = u / per_head, part = u - head * per_head;
    float v[16];
    load_values<BF16, VEC>(x, at + (int64_t)u * 16, v);
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 16; ++j) m = umax(m, __float_as_uint(v[j]) & 0x7fffffffu);
    uint32_t byte;
    float r;
    if constexpr (MX) {
      m = umax(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0xb1, 0xf, 0xf, true));   // lanes 2i and 2i + 1
      byte = e8m0_code(m);
      r = e8m0_inv(byte);
    } else {
      nv_block_scale(__uint_as_float(m), s_global, byte, r);
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] *= r;
    const int64_t row = cache_row(c, page, head, t);
    reinterpret_cast<u32x2*>(codes)[row * per_head + part] = u32x2{e2m1_pack8(v), e2m1_pack8(v + 8)};
    if constexpr (MX) {
      if ((part & 1) == 0) scales[row * (per_head >> 1) + (part >> 1)] = (uint8_t)byte;
    } else {
      scales[row * per_head + part] = (uint8_t)byte;
    }
  }
}

template <bool MX, bool BF16, bool VEC>
__global__ void __launch_bounds__(kThreads) k_kv_write(KvCache c, const void* k, int64_t k_stride, const void* v,
                                                       int64_t v_stride) {
  const int r = (int)(workgroup() * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6));
  if (r >= c.rows) return;
  const int b = seq_of_row(c, r);
  if (b < 0) return;
  const int begin = seq_begin(c, b), end = seq_end(c, b, begin);
  const int t = seq_length(c, b) - (end - r);
  if (r >= end || t < 0) return;
  const int page = page_of(c, b, t);
  if (page < 0) return;
  const float gk = MX ? 1.0f : nv_global_scale(*c.k_amax), gv = MX ? 1.0f : nv_global_scale(*c.v_amax);
  write_row<MX, BF16, VEC>(c, k, r * k_stride, c.k_codes, c.k_scales, gk, page, t);
  write_row<MX, BF16, VEC>(c, v, r * v_stride, c.v_codes, c.v_scales, gv, page, t);
}

// Eight values of codes and their scale as fp4_dequantize gives them.
template <bool MX>
__device__ __forceinline__ void dequant8_f32(uint32_t codes, uint32_t byte, float s_global, float (&v)[8]) {
  const float s = MX ? e8m0_value(byte) : s_global * e4m3_value(byte);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = s * e2m1_value((codes >> (4 * j)) & 15u);
}

template <bool MX, bool BF16, bool VEC>
__device__ __forceinline__ void read_row(const KvCache& c, void* y, int64_t at, const uint8_t* codes,
                                         const uint8_t* scales, float s_global, int page, int t) {
  const int lane = threadIdx.x & 63, units = c.heads * c.dim >> 3, per_head = c.dim >> 3;
  constexpr int kShift = MX ? 2 : 1;            // units of a scale
  for (int u = lane; u < units; u += 64) {
    const int head = u / per_head, part = u - head * per_head;
    uint32_t w = 0, byte = 0;
    if (page >= 0) {
      const int64_t row = cache_row(c, page, head, t);
      w = reinterpret_cast<const uint32_t*>(codes)[row * per_head + part];
      byte = scales[row * (per_head >> kShift) + (part >> kShift)];
    }
    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (page >= 0) dequant8_f32<MX>(w, byte, s_global, v);
    const int64_t i = at + (int64_t)u * 8;
    if constexpr (BF16) {
      uint16_t* p = static_cast<uint16_t*>(y) + i;
      const u32x4 o{bf16_pack2(v[0], v[1]), bf16_pack2(v[2], v[3]), bf16_pack2(v[4], v[5]), bf16_pack2(v[6], v[7])};
      if constexpr (VEC) {
        *reinterpret_cast<u32x4*>(p) = o;
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) p[j] = (uint16_t)(o[j >> 1] >> (16 * (j & 1)));
      }
    } else {
      float* p = static_cast<float*>(y) + i;
      if constexpr (VEC) {
        reinterpret_cast<f32x4*>(p)[0] = f32x4{v[0], v[1], v[2], v[3]};
        reinterpret_cast<f32x4*>(p)[1] = f32x4{v[4], v[5], v[6], v[7]};
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) p[j] = v[j];
      }
    }
  }
}

template <bool MX, bool BF16, bool VEC>
__global__ void __launch_bounds__(kThreads) k_kv_read(KvCache c, const int32_t* starts, void* k, void* v) {
  const int r = (int)(workgroup() * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6));
  if (r >= c.rows) return;
  const int b = seq_of_row(c, r);
  if (b < 0) return;
  const int begin = seq_begin(c, b), end = seq_end(c, b, begin);
  if (r >= end) return;
  const int length = seq_length(c, b);
  const int64_t t = starts != nullptr ? (int64_t)starts[b] + (r - begin) : length - (end - r);
  const int page = t >= 0 && t < length ? page_of(c, b, (int)t) : -1;
  const float gk = MX ? 1.0f : nv_global_scale(*c.k_amax), gv = MX ? 1.0f : nv_global_scale(*c.v_amax);
  const int64_t at = (int64_t)r * c.heads * c.dim;
  read_row<MX, BF16, VEC>(c, k, at, c.k_codes, c.k_scales, gk, page, (int)t);
  read_row<MX, BF16, VEC>(c, v, at, c.v_codes, c.v_scales, gv, page, (int)t);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// f(MX, BF16, VEC) with the three as compile-time constants.
template <typename F>
void select3(bool a, bool b, bool c, F f) {
  auto with = [&](auto x, auto y) { c ? f(x, y, std::true_type{}) : f(x, y, std::false_type{}); };
  auto next = [&](auto x) { b ? with(x, std::true_type{}) : with(x, std::false_type{}); };
  a ? next(std::true_type{}) : next(std::false_type{});
}

}  // namespace

namespace fp4impl {

hipError_t launch_kv_write(const KvCache& c, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                           bool bf16, hipStream_t stream) {
  const int64_t e = bf16 ? 2 : 4;
  const bool vec = aligned16(k) && aligned16(v) && k_stride * e % 16 == 0 && v_stride * e % 16 == 0;
  select3(c.mx, bf16, vec, [&](auto mx, auto bf, auto al) {
    k_kv_write<mx.value, bf.value, al.value><<<grid_of((c.rows + kWaves - 1) / kWaves), kThreads, 0, stream>>>(
        c, k, k_stride, v, v_stride);
  });
  return hipGetLastError();
}

hipError_t launch_kv_read(const KvCache& c, const int32_t* starts, void* k, void* v, bool bf16,
                          hipStream_t stream) {
  select3(c.mx, bf16, aligned16(k) && aligned16(v), [&](auto mx, auto bf, auto al) {
    k_kv_read<mx.value, bf.value, al.value><<<grid_of((c.rows + kWaves - 1) / kWaves), kThreads, 0, stream>>>(
        c, starts, k, v);
  });
  return hipGetLastError();
}

}  // namespace fp4impl
