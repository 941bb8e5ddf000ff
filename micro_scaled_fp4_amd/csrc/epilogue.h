// Device side of the fused epilogues: activations, their derivatives and the
// row pieces that a lane turns from accumulators into outputs.
//
//   z = alpha * acc + bias;  D = act(z) + residual, or, gated (W rows hold gate
//   and up projections alternately), D[:, j] = act(z[:, 2j]) * z[:, 2j + 1] + residual.
//
// Everything is float32 until the one rounding to the output type.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp4_device.h"
#include "grid.h"

namespace fp4dev {

// LDS traffic between the lanes of one wave: LDS operations of a wave complete
// in order, so only the compiler has to keep them in order.
__device__ __forceinline__ void wave_lds_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// values of fp4_activation
constexpr int kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActGeluTanh = 4;

// Optional parts of an epilogue (NULL: absent).  vec: N and every pointer allow
// whole 16-column pieces (16-byte accesses), so a piece is inside N or past it.
struct FusedArgs {
  const void* bias;       // [N], grouped [groups, N]
  const void* residual;   // [M, No], No = N, or N / 2 when gated; may be D itself
  void* preact;           // out: z [M, N]
  int bias_bf16, residual_bf16, preact_bf16;   // 1: bf16, 0: float32
  int activation, gated, vec;
};

// 1 / (1 + e^-x) on the transcendental unit (v_exp_f32, v_rcp_f32: 1 ulp each);
// the rounding of x * log2 e adds |x| 2^-24, so the relative error is below
// 4e-7 (1 + |x| / 4).  x -> -inf gives 1 / inf = 0.
__device__ __forceinline__ float sigmoid_fast(float x) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x * -0x1.715476p+0f));
}

// Upper tail Q(t) = (1 - Phi)(t) of the normal distribution, t >= 0, and
// e = exp(-t^2 / 2): Q = e * u * P(u), u = 1 / (1 + 0.3 t), P the degree-7
// minimax polynomial of exp(t^2 / 2) Q(t) / u on t in [0, 14] (relative error
// 1.5e-7, fitted in float64).  One exponential serves Q and the density.
__device__ __forceinline__ float normal_tail(float t, float& e) {
  e = __builtin_amdgcn_exp2f(t * t * -0x1.715476p-1f);
  const float u = __builtin_amdgcn_rcpf(fmaf(0.3f, t, 1.0f));
  float p = 0x1.243f6cp-5f;
  p = fmaf(p, u, -0x1.41f3b0p-3f);
  p = fmaf(p, u, 0x1.a69caap-3f);
  p = fmaf(p, u, -0x1.b7c6c2p-5f);
  p = fmaf(p, u, 0x1.074b52p-3f);
  p = fmaf(p, u, 0x1.993ee4p-4f);
  p = fmaf(p, u, 0x1.ee9bb4p-4f);
  p = fmaf(p, u, 0x1.ea006ap-4f);
  return p * u * e;
}

constexpr float kGeluC = 0x1.988454p-1f;   // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

template <int ACT>
__device__ __forceinline__ float act_value(float x) {
  if constexpr (ACT == kActRelu) return x < 0.0f ? 0.0f : x;
  if constexpr (ACT == kActSilu) return x * sigmoid_fast(x);
  if constexpr (ACT == kActGelu) {
    float e;
    const float q = normal_tail(fabsf(x), e);
    return x * (x < 0.0f ? q : 1.0f - q);
  }
  // 0.5 (1 + tanh u) = sigmoid(2 u)
  if constexpr (ACT == kActGeluTanh) return x * sigmoid_fast(2.0f * kGeluC * fmaf(kGeluA * x * x, x, x));
  return x;
}

// act(x) and act'(x)
template <int ACT>
__device__ __forceinline__ void act_both(float x, float& v, float& d) {
  if constexpr (ACT == kActNone) {
    v = x;
    d = 1.0f;
  } else if constexpr (ACT == kActRelu) {
    v = x < 0.0f ? 0.0f : x;
    d = x > 0.0f ? 1.0f : 0.0f;
  } else if constexpr (ACT == kActSilu) {
    const float s = sigmoid_fast(x);
    v = x * s;
    d = fmaf(v, 1.0f - s, s);
  } else if constexpr (ACT == kActGelu) {
    float e;
    const float q = normal_tail(fabsf(x), e);
    const float phi = x < 0.0f ? q : 1.0f - q;
    v = x * phi;
    d = fmaf(x * e, 0x1.988454p-2f, phi);   // + x * density, 1 / sqrt(2 pi)
  } else {
    const float s = sigmoid_fast(2.0f * kGeluC * fmaf(kGeluA * x * x, x, x));
    v = x * s;
    // (|x| >= 16: s is 0 or 1 and the first product 0, whose other factor must stay finite)
    const float y = __builtin_amdgcn_fmed3f(x, -16.0f, 16.0f);
    d = fmaf(v * (1.0f - s), 2.0f * kGeluC * fmaf(3.0f * kGeluA * y, y, 1.0f), s);
  }
}

// f(std::integral_constant-like tag) for the runtime activation; the switch is
// uniform over a launch.
template <int ACT>
struct ActTag {
  static constexpr int value = ACT;
};
template <typename F>
__device__ __forceinline__ void with_act(int act, F&& f) {
  switch (act) {
    case kActRelu: f(ActTag<kActRelu>{}); break;
    case kActSilu: f(ActTag<kActSilu>{}); break;
    case kActGelu: f(ActTag<kActGelu>{}); break;
    case kActGeluTanh: f(ActTag<kActGeluTanh>{}); break;
    default: f(ActTag<kActNone>{}); break;
  }
}

// ------------------------------------------------- vectors of 4 values --
// 4 consecutive values as float32, from bf16 (8 bytes) or float32 (16 bytes)
__device__ __forceinline__ f32x4 load4(const void* p, int64_t i, bool bf16) {
  if (bf16) {
    const u32x2 h = *reinterpret_cast<const u32x2*>(reinterpret_cast<const uint16_t*>(p) + i);
    return f32x4{bf16_lo(h.x), bf16_hi(h.x), bf16_lo(h.y), bf16_hi(h.y)};
  }
  return *reinterpret_cast<const f32x4*>(reinterpret_cast<const float*>(p) + i);
}
__device__ __forceinline__ float load1(const void* p, int64_t i, bool bf16) {
  return bf16 ? __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(p)[i] << 16)
              : reinterpret_cast<const float*>(p)[i];
}
__device__ __forceinline__ void store1(void* p, int64_t i, bool bf16, float v) {
  if (bf16)
    reinterpret_cast<uint16_t*>(p)[i] = (uint16_t)bf16_pack2(v, v);
  else
    reinterpret_cast<float*>(p)[i] = v;
}
// NV values (a multiple of 8) as 16-byte stores
template <int NV>
__device__ __forceinline__ void store_vec(void* p, int64_t i, bool bf16, const float (&v)[NV]) {
  if (bf16) {
    u32x4* q = reinterpret_cast<u32x4*>(reinterpret_cast<uint16_t*>(p) + i);
#pragma unroll
    for (int k = 0; k < NV / 8; ++k)
      q[k] = u32x4{bf16_pack2(v[8 * k], v[8 * k + 1]), bf16_pack2(v[8 * k + 2], v[8 * k + 3]),
                   bf16_pack2(v[8 * k + 4], v[8 * k + 5]), bf16_pack2(v[8 * k + 6], v[8 * k + 7])};
  } else {
    f32x4* q = reinterpret_cast<f32x4*>(reinterpret_cast<float*>(p) + i);
#pragma unroll
    for (int k = 0; k < NV / 4; ++k)
      q[k] = f32x4{v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]};
  }
}

// A lane's residual values for one 16-column piece (16, or 8 when gated), as
// loaded: at most 64 bytes.
struct ResidualRaw {
  u32x4 v[4];
};
__device__ __forceinline__ void load_residual(ResidualRaw& r, const FusedArgs& f, int64_t row, int n,
                                              int No) {
  const int no = f.gated ? n / 2 : n;
  const int n16 = (f.gated ? 1 : 2) * (f.residual_bf16 ? 1 : 2);   // 16-byte vectors: 1, 2 or 4
  const u32x4* p = reinterpret_cast<const u32x4*>(reinterpret_cast<const uint8_t*>(f.residual) +
                                                  (row * No + no) * (f.residual_bf16 ? 2 : 4));
  r.v[0] = p[0];
  if (n16 > 1) r.v[1] = p[1];
  if (n16 > 2) {
    r.v[2] = p[2];
    r.v[3] = p[3];
  }
}
template <int NV>
__device__ __forceinline__ void add_residual(float (&d)[NV], const ResidualRaw& r, bool bf16) {
  if (bf16) {
#pragma unroll
    for (int k = 0; k < NV / 8; ++k)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        d[8 * k + 2 * q] += bf16_lo(r.v[k][q]);
        d[8 * k + 2 * q + 1] += bf16_hi(r.v[k][q]);
      }
  } else {
#pragma unroll
    for (int k = 0; k < NV / 4; ++k)
#pragma unroll
      for (int q = 0; q < 4; ++q) d[4 * k + q] += __uint_as_float(r.v[k][q]);
  }
}

// One lane's 16 columns n .. n + 15 of row `row` (D's row; z = the accumulators
// times alpha plus bias), whole (vec launches): preact, activation, residual
// and store.  n is a multiple of 16.  `used` is called once r has been read.
template <bool OUT_BF16, typename F>
__device__ __forceinline__ void finish_piece(float (&z)[16], const FusedArgs& f, const ResidualRaw& r,
                                             int64_t row, int n, int N, void* D, F&& used) {
  if (f.preact != nullptr) store_vec<16>(f.preact, row * N + n, f.preact_bf16, z);
  if (f.gated) {
    float d[8];
    with_act(f.activation, [&](auto a) {
#pragma unroll
      for (int q = 0; q < 8; ++q) d[q] = act_value<decltype(a)::value>(z[2 * q]) * z[2 * q + 1];
    });
    if (f.residual != nullptr) {
      add_residual<8>(d, r, f.residual_bf16);
      used();
    }
    store_vec<8>(D, row * (N / 2) + n / 2, OUT_BF16, d);
  } else {
    with_act(f.activation, [&](auto a) {
#pragma unroll
      for (int q = 0; q < 16; ++q) z[q] = act_value<decltype(a)::value>(z[q]);
    });
    if (f.residual != nullptr) {
      add_residual<16>(z, r, f.residual_bf16);
      used();
    }
    store_vec<16>(D, row * N + n, OUT_BF16, z);
  }
}

// The same for sizes and alignments that take no whole pieces: a wave's ROWS
// rows of 64 columns, the accumulators in LDS rows of kStripRow floats; a lane takes
// one column (gated: one pair of columns) of each row, so every access of a row
// is contiguous across the lanes.  Rows row0 .. row0 + ROWS - 1 below m_rows (given as
// their count), columns n0 .. n0 + 63 below N; bias: of the lane's column(s).
constexpr int kStripRow = 68;                  // 64 columns, rows 4 banks apart
template <bool OUT_BF16, int ROWS>
__device__ __forceinline__ void finish_strip(const float* strip, float alpha, const FusedArgs& f, float b0, float b1,
                                             int64_t row0, int rows, int n0, int N, void* D) {
  const int lane = threadIdx.x & 63;
  if (f.gated) {   // 32 pairs, 2 rows at a time
    const int n = n0 + 2 * (lane & 31);
    if (n >= N) return;
    const int64_t No = N / 2;
    float r[ROWS / 2];
#pragma unroll
    for (int i = 0; i < ROWS / 2; ++i) {
      const int m = 2 * i + (lane >> 5);
      r[i] = f.residual != nullptr && m < rows
                 ? load1(f.residual, (row0 + m) * No + n / 2, f.residual_bf16) : 0.0f;
    }
    with_act(f.activation, [&](auto a) {
#pragma unroll
      for (int i = 0; i < ROWS / 2; ++i) {
        const int m = 2 * i + (lane >> 5);
        if (m >= rows) continue;
        const float z0 = fmaf(strip[m * kStripRow + (n - n0)], alpha, b0);
        const float z1 = fmaf(strip[m * kStripRow + (n - n0) + 1], alpha, b1);
        if (f.preact != nullptr) {
          store1(f.preact, (row0 + m) * N + n, f.preact_bf16, z0);
          store1(f.preact, (row0 + m) * N + n + 1, f.preact_bf16, z1);
        }
        store1(D, (row0 + m) * No + n / 2, OUT_BF16, act_value<decltype(a)::value>(z0) * z1 + r[i]);
      }
    });
  } else {
    const int n = n0 + lane;
    if (n >= N) return;
    float r[ROWS];
#pragma unroll
    for (int m = 0; m < ROWS; ++m)
      r[m] = f.residual != nullptr && m < rows
                 ? load1(f.residual, (row0 + m) * N + n, f.residual_bf16) : 0.0f;
    with_act(f.activation, [&](auto a) {
#pragma unroll
      for (int m = 0; m < ROWS; ++m) {
        if (m >= rows) continue;
        const float z = fmaf(strip[m * kStripRow + lane], alpha, b0);
        if (f.preact != nullptr) store1(f.preact, (row0 + m) * N + n, f.preact_bf16, z);
        store1(D, (row0 + m) * N + n, OUT_BF16, act_value<decltype(a)::value>(z) + r[m]);
      }
    });
  }
}

// Bias of 16 columns from n < N on (vec launches; zero without one).  base: the
// group's first element.
__device__ __forceinline__ void load_bias(float (&b)[16], const FusedArgs& f, int64_t base, int n) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const f32x4 v = f.bias != nullptr ? load4(f.bias, base + n + 4 * k, f.bias_bf16) : f32x4{0, 0, 0, 0};
    b[4 * k] = v.x; b[4 * k + 1] = v.y; b[4 * k + 2] = v.z; b[4 * k + 3] = v.w;
  }
}

// Rows of a grouped output (and its preact) past the last group's -- slots that
// were dropped -- hold zeros, so that what reads the whole tensor next (a
// quantizer's amax) sees none of the memory's earlier contents.  Every thread of
// the launch takes a share; usually there are none.
__device__ __forceinline__ void zero_tail(const int32_t* __restrict__ offsets, int groups, int M, int N,
                                          const FusedArgs& f, bool out_bf16, void* D) {
  const int lo = min(max(offsets[groups], 0), M);
  if (lo == M) return;
  const int64_t first = (int64_t)workgroup() * blockDim.x + threadIdx.x;
  const int64_t step = (int64_t)workgroups() * blockDim.x;
  const int64_t No = f.gated ? N / 2 : N;
  for (int64_t i = lo * No + first; i < M * No; i += step) store1(D, i, out_bf16, 0.0f);
  if (f.preact != nullptr)
    for (int64_t i = lo * (int64_t)N + first; i < M * (int64_t)N; i += step)
      store1(f.preact, i, f.preact_bf16, 0.0f);
}

}  // namespace fp4dev
