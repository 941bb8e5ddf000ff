// Writing and reading a paged key/value cache in FP4 (include/fp4.h, kv_cache_write
// and kv_cache_read).
//
// A wave takes one row of the call, k and v, all heads: it finds the row's sequence and
// page once, then its lanes take the row's values in order.
//   Write: a lane quantizes 16 values, an NVFP4 block; two lanes share an MXFP4 block and
//   its maximum.  The steps are those of nvfp4_quantize and mxfp4_quantize, bit for bit.
//   Read: a lane dequantizes 8 values (one dword of codes) and stores 16 bytes of bf16, past
//   the caches: what is read back is larger than they are.
// Both are bound by HBM bytes (a row of 8 heads x 128 bf16 channels moves 4096 bytes one
// way and 1152 or 1088 the other).  Measured at that row: written, 32 rows 4.3 us (the chain of
// loads that finds a row's page), 16384 rows 18.5 us (4.6 TB/s); read, 32 rows 4.0 us, 4096 rows
// 7.0, 16384 rows 15 and 65536 rows 54 (6.3 TB/s).  Four rows a wave read no faster (8.1 us at
// 1024 rows, 54 at 65536).
#include <type_traits>

#include "fp4_device.h"
#include "fp4_internal.h"
#include "grid.h"
#include "kv_cache.h"

using namespace fp4dev;
using fp4impl::KvCache;

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

// Sixteen consecutive values from x + i.  (Element alignment is enough for 16-byte accesses to global memory.)
template <bool BF16>
__device__ __forceinline__ void load16(const void* x, int64_t i, float (&v)[16]) {
  if constexpr (BF16) {
    u32x4 w[2];
    __builtin_memcpy(w, static_cast<const uint16_t*>(x) + i, 32);
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[8 * j + 2 * e] = bf16_lo(w[j][e]);
        v[8 * j + 2 * e + 1] = bf16_hi(w[j][e]);
      }
  } else {
    __builtin_memcpy(v, static_cast<const float*>(x) + i, 64);
  }
}

template <bool MX, bool BF16>
__device__ __forceinline__ void write_row(const KvCache& c, const void* x, int64_t at, uint8_t* codes,
                                          uint8_t* scales, float s_global, int page, int t) {
  const int lane = threadIdx.x & 63, units = c.heads * c.dim >> 4, per_head = c.dim >> 4;
  for (int u0 = 0; u0 < units; u0 += 64) {
    const int u = u0 + lane;                    // units is even: an MXFP4 block's two lanes stay together
    if (u >= units) break;
    const int head = u / per_head, part = u - head * per_head;
    float v[16];
    load16<BF16>(x, at + (int64_t)u * 16, v);
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

template <bool MX, bool BF16>
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
  write_row<MX, BF16>(c, k, r * k_stride, c.k_codes, c.k_scales, gk, page, t);
  write_row<MX, BF16>(c, v, r * v_stride, c.v_codes, c.v_scales, gv, page, t);
}

// Eight values of codes and their scale as fp4_dequantize gives them.
template <bool MX>
__device__ __forceinline__ void dequant8_f32(uint32_t codes, uint32_t byte, float s_global, float (&v)[8]) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  const float s = MX ? e8m0_value(byte) : s_global * __builtin_amdgcn_cvt_f32_fp8((int)byte, 0);
  const f32x2 p[4] = {
      __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 0), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 1),
      __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 2), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 3)};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = s * p[j][0];
    v[2 * j + 1] = s * p[j][1];
  }
}

// A lane takes units of 8 values of the wave's row, keys first, then values; kUnits at a time, so that
// their loads are on their way together.
template <bool MX, bool BF16>
__global__ void __launch_bounds__(kThreads) k_kv_read(KvCache c, const int32_t* starts, void* k, void* v) {
  const int r = (int)(workgroup() * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6));
  if (r >= c.rows) return;
  const int b = seq_of_row(c, r);
  if (b < 0) return;
  const int begin = seq_begin(c, b), end = seq_end(c, b, begin);
  if (r >= end) return;
  const int length = seq_length(c, b);
  const int64_t at = (int64_t)(starts != nullptr ? starts[b] : length - (end - begin)) + (r - begin);
  const int t = at >= 0 && at < length ? (int)at : 0;
  const int page = at >= 0 && at < length ? page_of(c, b, t) : -1;     // (-1: zeros)
  const float gk = MX ? 1.0f : nv_global_scale(*c.k_amax), gv = MX ? 1.0f : nv_global_scale(*c.v_amax);
  const int lane = threadIdx.x & 63, units = c.heads * c.dim >> 3, per_head = c.dim >> 3;
  constexpr int kShift = MX ? 2 : 1;            // units of a scale
  constexpr int kUnits = 4;
  for (int u0 = 0; u0 < 2 * units; u0 += 64 * kUnits) {
    uint32_t w[kUnits], byte[kUnits];
#pragma unroll
    for (int j = 0; j < kUnits; ++j) {
      const int u = u0 + 64 * j + lane;
      const bool value = u >= units;
      const int x = value ? u - units : u, head = x / per_head, part = x - head * per_head;
      w[j] = byte[j] = 0;
      if (u < 2 * units && page >= 0) {
        const int64_t row = cache_row(c, page, head, t);
        w[j] = reinterpret_cast<const uint32_t*>(value ? c.v_codes : c.k_codes)[row * per_head + part];
        byte[j] = (value ? c.v_scales : c.k_scales)[row * (per_head >> kShift) + (part >> kShift)];
      }
    }
#pragma unroll
    for (int j = 0; j < kUnits; ++j) {
      const int u = u0 + 64 * j + lane;
      if (u >= 2 * units) continue;
      const bool value = u >= units;
      const int64_t o = (int64_t)r * c.heads * c.dim + (value ? u - units : u) * 8;
      float x[8];
      dequant8_f32<MX>(w[j], byte[j], value ? gv : gk, x);
      if constexpr (BF16) {
        typedef u32x4 any __attribute__((aligned(2)));
        const u32x4 y{bf16_pack2(x[0], x[1]), bf16_pack2(x[2], x[3]), bf16_pack2(x[4], x[5]), bf16_pack2(x[6], x[7])};
        __builtin_nontemporal_store(y, reinterpret_cast<any*>(static_cast<uint16_t*>(value ? v : k) + o));
      } else {
        typedef f32x4 any __attribute__((aligned(4)));
        any* const p = reinterpret_cast<any*>(static_cast<float*>(value ? v : k) + o);
        __builtin_nontemporal_store(f32x4{x[0], x[1], x[2], x[3]}, p);
        __builtin_nontemporal_store(f32x4{x[4], x[5], x[6], x[7]}, p + 1);
      }
    }
  }
}

// f(MX, BF16) with the two as compile-time constants.
template <typename F>
void select2(bool a, bool b, F f) {
  auto with = [&](auto x) { b ? f(x, std::true_type{}) : f(x, std::false_type{}); };
  a ? with(std::true_type{}) : with(std::false_type{});
}

}  // namespace

namespace fp4impl {

hipError_t launch_kv_write(const KvCache& c, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                           bool bf16, hipStream_t stream) {
  select2(c.mx, bf16, [&](auto mx, auto bf) {
    k_kv_write<mx.value, bf.value><<<grid_of((c.rows + kWaves - 1) / kWaves), kThreads, 0, stream>>>(
        c, k, k_stride, v, v_stride);
  });
  return hipGetLastError();
}

hipError_t launch_kv_read(const KvCache& c, const int32_t* starts, void* k, void* v, bool bf16,
                          hipStream_t stream) {
  select2(c.mx, bf16, [&](auto mx, auto bf) {
    k_kv_read<mx.value, bf.value><<<grid_of((c.rows + kWaves - 1) / kWaves), kThreads, 0, stream>>>(c, starts, k, v);
  });
  return hipGetLastError();
}

}  // namespace fp4impl
