// Backward pass of the fused epilogues: dz from dD and the pre-activations, and
// the bias gradient (column sums of dz, per group in the grouped form).
//
//   D = act(z) + residual          dz = dD act'(z)
//   D = act(g) u + residual        dg = dD u act'(g),  du = dD act(g)   (z: g, u alternate)
//
// The residual's gradient is dD itself.
#include "epilogue.h"
#include "fp4_internal.h"
#include "grid.h"

using namespace fp4dev;

namespace {

struct GradArgs {
  const void* dD;
  const void* z;
  void* dz;
  float* partials;            // [groups * splits][N], or NULL: no bias gradient
  const int32_t* offsets;     // grouped, else NULL
  int dD_bf16, z_bf16, dz_bf16;
  int64_t M;
  int N, groups, splits, gated, activation, col_wgs;
};

constexpr int kGradThreads = 256;
constexpr int kGradWaves = kGradThreads / 64;

// 16 bytes that are read or written once
__device__ __forceinline__ u32x4 stream_load(const void* p) {
  return __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
}

// Values [c, c + V) of row `row`; V 4 or 8: whole accesses, V 1 or 2: any size
// (zeros past N).
template <int V>
__device__ __forceinline__ void load_cols(const void* p, int64_t row, int c, int N, bool bf16, float (&v)[V]) {
  const int64_t i = row * N + c;
  if constexpr (V == 4) {
    const f32x4 w = load4(p, i, bf16);
    v[0] = w.x; v[1] = w.y; v[2] = w.z; v[3] = w.w;
  } else if constexpr (V == 8) {
    if (bf16) {
      const uint16_t* q = reinterpret_cast<const uint16_t*>(p) + i;
#pragma unroll
      for (int k = 0; k < V / 8; ++k) {
        const u32x4 w = stream_load(q + 8 * k);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[8 * k + 2 * e] = bf16_lo(w[e]);
          v[8 * k + 2 * e + 1] = bf16_hi(w[e]);
        }
      }
    } else {
      const float* q = reinterpret_cast<const float*>(p) + i;
#pragma unroll
      for (int k = 0; k < V / 4; ++k) {
        const u32x4 w = stream_load(q + 4 * k);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[4 * k + e] = __uint_as_float(w[e]);
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k) v[k] = c + k < N ? load1(p, i + k, bf16) : 0.0f;
  }
}
template <int V>
__device__ __forceinline__ void store_cols(void* p, int64_t row, int c, int N, bool bf16, const float (&v)[V]) {
  const int64_t i = row * N + c;
  if constexpr (V == 8) {
    if (bf16) {
      u32x4* q = reinterpret_cast<u32x4*>(reinterpret_cast<uint16_t*>(p) + i);
#pragma unroll
      for (int k = 0; k < V / 8; ++k)
        __builtin_nontemporal_store(u32x4{bf16_pack2(v[8 * k], v[8 * k + 1]), bf16_pack2(v[8 * k + 2], v[8 * k + 3]),
                                          bf16_pack2(v[8 * k + 4], v[8 * k + 5]), bf16_pack2(v[8 * k + 6], v[8 * k + 7])},
                                    q + k);
    } else {
      f32x4* q = reinterpret_cast<f32x4*>(reinterpret_cast<float*>(p) + i);
#pragma unroll
      for (int k = 0; k < V / 4; ++k)
        __builtin_nontemporal_store(f32x4{v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]}, q + k);
    }
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k)
      if (c + k < N) store1(p, i + k, bf16, v[k]);
  }
}

// dz of the rows past the last group's (slots that were dropped): zeros, as the
// forward writes them in D and preact, so that a quantizer of all of dz sees none of
// the memory's earlier contents.  Every thread of the launch takes a share, in 16-byte
// pieces where rows are whole pieces (V 8).
template <int V>
__device__ __forceinline__ void zero_past_groups(const GradArgs& a) {
  const int64_t lo = min(max((int64_t)a.offsets[a.groups], (int64_t)0), a.M);
  if (lo == a.M) return;
  const int64_t first = (int64_t)workgroup() * kGradThreads + threadIdx.x, step = (int64_t)workgroups() * kGradThreads;
  if constexpr (V == 8) {
    const int per = a.dz_bf16 ? 8 : 4;             // values of a piece
    u32x4* q = reinterpret_cast<u32x4*>(a.dz);
    for (int64_t i = lo * a.N / per + first; i < a.M * a.N / per; i += step)
      __builtin_nontemporal_store(u32x4{0, 0, 0, 0}, q + i);
  } else {
    for (int64_t i = lo * a.N + first; i < a.M * a.N; i += step) store1(a.dz, i, a.dz_bf16, 0.0f);
  }
}

// A workgroup takes 64 V columns and one split of a group's rows, its waves
// every kGradWaves-th row of it, so a lane keeps its columns' sums in registers.
// Bias partials: the waves' sums added in wave order, one row per split.
// V 8: 16-byte accesses (N a multiple of 16, aligned pointers), contiguous over the
// lanes; V 2: any size.  HBM bound: everything is read or written once.  Gated bf16
// 8192 x 28672, 1.17 GB: 236 us, 5.0 TB/s, a large copy's rate (the same tensors
// again and again: 200; with 16 columns a lane, half lines per access, 327; through
// the caches, in 8-byte accesses, 258).
template <int V>
__global__ void __launch_bounds__(kGradThreads) k_epilogue_grad(GradArgs a) {
  __shared__ float red[kGradWaves][64 * V];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint32_t wg = workgroup();
  const int part = wg / (uint32_t)a.col_wgs, col_wg = wg - (uint32_t)part * a.col_wgs;
  const int c = (col_wg * 64 + lane) * V;
  const int e = part / a.splits, s = part - e * a.splits;
  int64_t lo = 0, hi = a.M;
  if (a.offsets != nullptr) zero_past_groups<V>(a);
  if (e >= a.groups) return;                       // (a grid's last row runs past the count)
  if (a.offsets != nullptr) {
    lo = min(max((int64_t)a.offsets[e], (int64_t)0), a.M);
    hi = min(max((int64_t)a.offsets[e + 1], lo), a.M);
  }
  const int64_t per = (hi - lo + a.splits - 1) / a.splits;
  const int64_t r0 = min(lo + s * per, hi), r1 = min(r0 + per, hi);
  float sum[V];
#pragma unroll
  for (int k = 0; k < V; ++k) sum[k] = 0.0f;
  const int No = a.gated ? a.N / 2 : a.N;
  if (c < a.N) {
    with_act(a.activation, [&](auto act) {
      constexpr int ACT = decltype(act)::value;
      for (int64_t r = r0 + wave; r < r1; r += kGradWaves) {
        float z[V], dz[V];
        load_cols<V>(a.z, r, c, a.N, a.z_bf16, z);
        if (a.gated) {
          float d[V / 2];
          load_cols<V / 2>(a.dD, r, c / 2, No, a.dD_bf16, d);
#pragma unroll
          for (int k = 0; k < V / 2; ++k) {
            float v, g;
            act_both<ACT>(z[2 * k], v, g);
            dz[2 * k] = d[k] * z[2 * k + 1] * g;
            dz[2 * k + 1] = d[k] * v;
          }
        } else {
          float d[V];
          load_cols<V>(a.dD, r, c, a.N, a.dD_bf16, d);
#pragma unroll
          for (int k = 0; k < V; ++k) {
            float v, g;
            act_both<ACT>(z[k], v, g);
            dz[k] = d[k] * g;
          }
        }
#pragma unroll
        for (int k = 0; k < V; ++k) sum[k] += dz[k];
        store_cols<V>(a.dz, r, c, a.N, a.dz_bf16, dz);
      }
    });
  }
  if (a.partials == nullptr) return;
#pragma unroll
  for (int k = 0; k < V; ++k) red[wave][lane * V + k] = sum[k];
  __syncthreads();
  const int c0 = col_wg * 64 * V;
  for (int i = threadIdx.x; i < 64 * V && c0 + i < a.N; i += kGradThreads) {
    float t = red[0][i];
#pragma unroll
    for (int w = 1; w < kGradWaves; ++w) t += red[w][i];
    a.partials[(int64_t)part * a.N + c0 + i] = t;
  }
}

// dbias[e][c] = sum of the splits' partials: 64 columns a workgroup, wave w the
// splits w, w + 4, ... in order, then the waves in order
__global__ void __launch_bounds__(kGradThreads)
    k_bias_grad(const float* __restrict__ partials, int splits, int64_t cols, int N, float* __restrict__ dbias) {
  __shared__ float red[kGradWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t i = (int64_t)workgroup() * 64 + lane;
  float s = 0.0f;
  if (i < cols) {
    const int64_t e = i / N, c = i - e * N;
    const float* p = partials + e * splits * N + c;
#pragma unroll 8
    for (int k = wave; k < splits; k += kGradWaves) s += p[(int64_t)k * N];
  }
  red[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && i < cols) dbias[i] = ((red[0][lane] + red[1][lane]) + red[2][lane]) + red[3][lane];
}

// Row splits: enough workgroups to fill the device several times over at the
// vector form's 512 columns each, at least 64 rows a split.
int64_t grad_splits(int64_t groups, int64_t M, int64_t N) {
  const int64_t cols = (N + 511) / 512, want = 4096;
  const int64_t by_wgs = (want + cols * groups - 1) / (cols * groups);
  const int64_t by_rows = M / groups / 64;
  const int64_t s = by_wgs < by_rows ? by_wgs : by_rows;
  return s < 1 ? 1 : s;
}

}  // namespace

namespace fp4impl {

size_t epilogue_grad_workspace_bytes(int64_t groups, int64_t M, int64_t N) {
  return (size_t)(groups * grad_splits(groups, M, N) * N) * 4;
}

hipError_t launch_epilogue_grad(const void* dD, bool dD_bf16, const void* z, bool z_bf16, int64_t groups,
                                const int32_t* offsets, int64_t M, int64_t N, int activation, bool gated,
                                void* dz, bool dz_bf16, float* dbias, void* workspace, hipStream_t stream) {
  auto ok16 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
  const bool vec = N % 16 == 0 && ok16(dD) && ok16(z) && ok16(dz);
  const int64_t splits = grad_splits(groups, M, N);
  const int64_t per = 64 * (vec ? 8 : 2), col_wgs = (N + per - 1) / per;
  if (groups * splits * col_wgs >= (int64_t)1 << 31) return hipErrorInvalidValue;
  // (one split: its sums are the gradient)
  float* partials = dbias == nullptr ? nullptr : splits == 1 ? dbias : static_cast<float*>(workspace);
  const GradArgs a{dD, z, dz, partials, offsets, dD_bf16, z_bf16, dz_bf16, M, (int)N, (int)groups,
                   (int)splits, gated, activation, (int)col_wgs};
  const dim3 grid = grid_of(groups * splits * col_wgs);
  if (vec)
    hipLaunchKernelGGL((k_epilogue_grad<8>), grid, dim3(kGradThreads), 0, stream, a);
  else
    hipLaunchKernelGGL((k_epilogue_grad<2>), grid, dim3(kGradThreads), 0, stream, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || dbias == nullptr || splits == 1) return e;
  const int64_t cols = groups * N;
  hipLaunchKernelGGL(k_bias_grad, grid_of((cols + 63) / 64),
                     dim3(kGradThreads), 0, stream, partials, (int)splits, cols, (int)N, dbias);
  return hipGetLastError();
}

}  // namespace fp4impl
