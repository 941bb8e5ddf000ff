// Attention over a paged key/value cache in FP4 (include/fp4.h, kv_cache_attention).
//
// One wave per query row and head, in float32: 64 positions at a time, a lane per
// position for the scores, a lane per channel for the weighted sum, with the running
// maximum and sum of the softmax.
#include "fp4_device.h"
#include "fp4_internal.h"
#include "grid.h"
#include "kv_cache.h"

using namespace fp4dev;
using fp4impl::AttendProblem;
using fp4impl::KvCache;

namespace {

__device__ __forceinline__ float block_value(bool mx, uint32_t byte, float s_global) {
  return mx ? e8m0_value(byte) : s_global * e4m3_value(byte);
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v = fmaxf(v, __shfl_xor(v, off, 64));
  return v;
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

__global__ void __launch_bounds__(64) k_attend(KvCache c, AttendProblem a) {
  __shared__ float q[256];
  const int lane = threadIdx.x;
  const int r = workgroup() / a.q_heads, h = workgroup() % a.q_heads;
  if (r >= c.rows) return;
  const int b = seq_of_row(c, r);
  if (b < 0) return;
  const int begin = seq_begin(c, b), end = seq_end(c, b, begin), length = seq_length(c, b);
  if (r >= end) return;
  const int pos = length - (end - r);
  const int hi = a.causal ? min(length, pos + 1) : length, lo = a.window > 0 ? max(0, pos - a.window + 1) : 0;
  const int head = h / (a.q_heads / c.heads), bs = c.mx ? 32 : 16;
  const float gk = c.mx ? 1.0f : nv_global_scale(*c.k_amax), gv = c.mx ? 1.0f : nv_global_scale(*c.v_amax);
  for (int d = lane; d < c.dim; d += 64) {
    const int64_t i = r * a.q_stride + (int64_t)h * c.dim + d;
    q[d] = a.q_bf16 ? __uint_as_float((uint32_t) static_cast<const uint16_t*>(a.q)[i] << 16)
                    : static_cast<const float*>(a.q)[i];
  }
  __syncthreads();
  float acc[4] = {0, 0, 0, 0}, m = -INFINITY, l = 0;
  for (int t0 = lo; t0 < hi; t0 += 64) {
    const int t = t0 + lane, page = t < hi ? page_of(c, b, t) : -1;
    float s = -INFINITY;
    if (page >= 0) {
      const int64_t row = cache_row(c, page, head, t);
      float sum = 0;
      for (int w = 0; w < c.dim / 8; ++w) {
        const uint32_t codes = reinterpret_cast<const uint32_t*>(c.k_codes)[row * (c.dim / 8) + w];
        const float sb = block_value(c.mx, c.k_scales[row * (c.dim / bs) + w * 8 / bs], gk);
        float part = 0;
        for (int j = 0; j < 8; ++j) part += q[8 * w + j] * e2m1_value((codes >> (4 * j)) & 15u);
        sum += part * sb;
      }
      s = a.scale * sum;
    }
    const float now = fmaxf(m, wave_max(s));
    const float base = now == -INFINITY ? 0.0f : now;
    const float p = __expf(s - base), drop = __expf(m - base);
    l = l * drop + wave_sum(p);
    m = now;
    for (int j = 0; j < 4; ++j) acc[j] *= drop;
    for (int i = 0; i < 64 && t0 + i < hi; ++i) {
      const float pi = __shfl(p, i, 64);
      const int pg = __shfl(page, i, 64);
      if (pg < 0) continue;
      const int64_t row = cache_row(c, pg, head, t0 + i);
      for (int j = 0; j < 4; ++j) {
        const int d = lane + 64 * j;
        if (d < c.dim)
          acc[j] += pi * block_value(c.mx, c.v_scales[row * (c.dim / bs) + d / bs], gv) *
                    e2m1_value((c.v_codes[row * (c.dim / 2) + d / 2] >> (4 * (d & 1))) & 15u);
      }
    }
  }
  for (int j = 0; j < 4; ++j) {
    const int d = lane + 64 * j;
    if (d >= c.dim) continue;
    const int64_t i = ((int64_t)r * a.q_heads + h) * c.dim + d;
    const float o = l > 0 ? acc[j] / l : 0.0f;
    if (a.out_bf16) static_cast<uint16_t*>(a.out)[i] = (uint16_t)f32_to_bf16(o);
    else static_cast<float*>(a.out)[i] = o;
  }
  if (a.lse != nullptr && lane == 0) a.lse[(int64_t)r * a.q_heads + h] = l > 0 ? m + logf(l) : -INFINITY;
}

}  // namespace

namespace fp4impl {

size_t kv_attention_workspace_bytes(int64_t, int64_t, int, int, int) { return 16; }

hipError_t launch_kv_attention(const KvCache& c, const AttendProblem& p, hipStream_t stream) {
  k_attend<<<grid_of((int64_t)c.rows * p.q_heads), 64, 0, stream>>>(c, p);
  return hipGetLastError();
}

}  // namespace fp4impl
