// Block-scaled FP4 products through the fused epilogue on 128 x 128 tiles, two
// workgroups per CU, dense and grouped: for outputs that 256 x 256 tiles leave most
// of the device without work.
//
// Work.  A workgroup's 2 x 2 waves own 4 x 4 tiles of 16 x 16 each; K advances 256
// values per stage through two LDS buffers that direct-to-LDS loads fill (operand
// swizzle and edges as in gemm_kernels.h).  A stage's operands go to registers at
// once (64 of them), so its buffer is free again before its MFMAs and the loads of
// the stage after next run under two stages of them.  The wait for the next stage
// counts the loads in flight instead of draining them.  The other workgroup of the
// CU computes meanwhile: two of 68 (MXFP4) or 72 KB (NVFP4) fit its LDS, and 256
// registers a wave.  MXFP4 multiplies the codes under their E8M0 bytes; NVFP4
// dequantizes both operands to fp16 (exact), each value twice per workgroup, where
// the 256 x 256 tiles do it twice per four times the outputs.
//
// Bound: the latency of a stage with one tile per CU (MXFP4 0.84, NVFP4 2.2 us), LDS
// reads (MXFP4) or dequantizing beside the MFMAs (NVFP4) with more (0.92 and 2.07 us
// a tile and stage).  Measured: 1021 x 5120 x 7168 NVFP4 108 us (256 x 256 tiles
// 154), MXFP4 42 (57); 128 x 27648 x 5120 55 (115) and 26 (43); 64 groups of 128
// rows x 4096 x 7168 508 (694) and 279 (326).  8192 x 8192 x 8192, where the larger
// tiles fill the device: 953 (782) and 405 (319).  Eight waves that split a stage's
// K: 7 to 12% faster with a tile or less per CU, slower everywhere else.
#include <math.h>

#include <atomic>

#include "gemm_kernels.h"

namespace {

constexpr int kTile = 128;                      // rows of A and of W per workgroup
constexpr int kT = 4;                           // 16-row MFMA tiles of a wave (2 x 2 waves), per operand
constexpr int kTileBytes = kTile * kRowBytes;   // 16 KB
constexpr int kStripRows = 16;
constexpr int kStrip = kStripRows * kStripRow * 4;   // a wave's strip, bytes

template <bool MX>
struct MidCfg {
  static constexpr int kScales = kTile * (MX ? BK / 32 : BK / 16);   // of an operand's stage
  static constexpr int kLds = 2 * 2 * (kTileBytes + kScales);        // 68 KB (MX) / 72 KB (NV)
};

// A barrier that waits for nothing but the waves: what has to be complete is waited
// on before it (__syncthreads would also wait for the loads in flight).
__device__ __forceinline__ void wave_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
}

struct MidArgs {
  const uint8_t* A;
  const uint8_t* as;
  const uint8_t* W;
  const uint8_t* ws;
  const float* g_a;
  const float* g_b;
  float g_d;
  int M, N, K, tiles_m, tiles_n;
  const int32_t* offsets;                       // grouped, else NULL
  int groups;
  void* D;
  FusedArgs f;
};

template <bool MX, bool SVEC, bool OUT_BF16, bool GROUPED>
__global__ void __launch_bounds__(kThreads, 2) k_gemm_mid(MidArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  static_assert(4 * kStrip <= MidCfg<MX>::kLds, "the strips reuse the tiles");
  const int M = a.M, N = a.N, K = a.K;
  const int T = GROUPED ? group_row_tiles<kTile>(a.offsets, a.groups, M) * a.tiles_n : a.tiles_m * a.tiles_n;
  if constexpr (GROUPED) zero_tail(a.offsets, a.groups, M, N, a.f, OUT_BF16, a.D);
  if ((int)blockIdx.x >= T) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int r16 = lane & 15, g = lane >> 4;
  const int rowb = K / 2, nsc = K / (MX ? 32 : 16);

  // ---- this workgroup's tile
  int tm = 0, tn = 0, lo = 0, m_rows = M, e = 0;
  if constexpr (GROUPED) {
    int t, hi = 0;
    xcd_tile(blockIdx.x, T, t);
    group_tile_of<kTile>(a.offsets, a.groups, M, t / a.tiles_n, e, tm, lo, hi);
    tn = t % a.tiles_n;
    m_rows = hi - lo;
    e = __builtin_amdgcn_readfirstlane(e);
    tm = __builtin_amdgcn_readfirstlane(tm);
    lo = __builtin_amdgcn_readfirstlane(lo);
    m_rows = __builtin_amdgcn_readfirstlane(m_rows);
  } else {
    tile_of(blockIdx.x, a.tiles_m, a.tiles_n, tm, tn);
  }
  const int m0 = tm * kTile, n0 = tn * kTile;
  const int64_t a_row = (int64_t)lo + m0, w_row = (int64_t)e * N + n0;
  const int rows_a = min(kTile, m_rows - m0), rows_w = min(kTile, N - n0);
  const uint8_t* pa = a.A + a_row * rowb;
  const uint8_t* pw = a.W + w_row * rowb;
  // thread t holds scale row t % 128 of A (t < 128) or W
  const bool of_a = wave < 2;
  const int srow = threadIdx.x & 127;
  const uint8_t* psc = of_a ? a.as + a_row * nsc : a.ws + w_row * nsc;
  const int sc_bytes = (of_a ? rows_a : rows_w) * nsc;

  // LDS: A tiles 0, 1 | W tiles 0, 1 | A scales 0, 1 | W scales 0, 1
  constexpr int kSc = MidCfg<MX>::kScales;
  auto tile_a = [&](int b) { return smem + b * kTileBytes; };
  auto tile_w = [&](int b) { return smem + (2 + b) * kTileBytes; };
  auto sc_a = [&](int b) { return smem + 4 * kTileBytes + b * kSc; };
  auto sc_w = [&](int b) { return smem + 4 * kTileBytes + (2 + b) * kSc; };

  const int nk = (K + BK - 1) / BK;
  constexpr int kBlocks = kTileBytes / 1024 / 4;   // 1 KB blocks per wave and operand
  using Scales = StageScales<MX, SVEC>;
  // stage kt's loads into buffer b; past the last stage through empty ranges
  auto load = [&](Scales& s, int kt, int b) {
    const bool live = kt < nk;
    const ScaleRange rs = scale_range<SVEC>(psc, live ? sc_bytes : 0);
    load_scales<MX, SVEC>(s, rs, srow, nsc, kt * BK);
    const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t*>(pa), 0, live ? rows_a * rowb : 0, kBufferWord3);
    const __amdgpu_buffer_rsrc_t rw = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t*>(pw), 0, live ? rows_w * rowb : 0, kBufferWord3);
#pragma unroll
    for (int q = 0; q < kBlocks; ++q) {
      dma_block<SVEC>(ra, tile_a(b), rowb, K, kt * BK, q);
      dma_block<SVEC>(rw, tile_w(b), rowb, K, kt * BK, q);
    }
  };
  // load instructions of a stage per wave, at least (the compiler may join the scale
  // bytes' dwords into one): that many in flight leave no earlier stage's
  constexpr int kLoads = 2 * kBlocks + 1;
  static_assert(kLoads < 16, "one field of the wait's count");
  // scale entry (h, g, r16, i): the bytes that lane (r16, g) of wave half h needs
  // for its tile i, the 4 tiles' contiguous
  auto store_sc = [&](const Scales& s, int b) {
    uint32_t v[MX ? 2 : 4];
    placed_scales<MX, SVEC>(v, s, srow, nsc);
    uint8_t* sc = of_a ? sc_a(b) : sc_w(b);
    const int h = srow >> 6, i = (srow >> 4) & 3;
#pragma unroll
    for (int gg = 0; gg < 4; ++gg) {
      const int at = ((h * 4 + gg) * 16 + (srow & 15)) * 4 + i;
      if (MX)
        reinterpret_cast<uint16_t*>(sc)[at] = (uint16_t)(v[gg >> 1] >> (16 * (gg & 1)));
      else
        reinterpret_cast<uint32_t*>(sc)[at] = v[gg];
    }
  };

  v4f acc[kT][kT];                              // [W tile][A tile]
#pragma unroll
  for (int i = 0; i < kT; ++i)
#pragma unroll
    for (int j = 0; j < kT; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

  const int ra0 = wm * 16 * kT + r16, rw0 = wn * 16 * kT + r16;
  auto frag = [&](const uint8_t* tile, int row, int chunk) {
    return *reinterpret_cast<const u32x4*>(tile + swz(row, chunk));
  };
  auto stage = [&](Scales& cur, Scales& next, int kt, int b) {
    // stage kt is in buffer b; its operands to registers
    u32x4 fa[2][kT], fw[2][kT];
#pragma unroll
    for (int st = 0; st < 2; ++st)
#pragma unroll
      for (int i = 0; i < kT; ++i) {
        fa[st][i] = frag(tile_a(b), ra0 + 16 * i, 2 * g + st);
        fw[st][i] = frag(tile_w(b), rw0 + 16 * i, 2 * g + st);
      }
    constexpr int kDw = MX ? 2 : 4;
    uint32_t sa[kDw], sw[kDw];
    const uint32_t* lsa = reinterpret_cast<const uint32_t*>(sc_a(b)) + ((wm * 4 + g) * 16 + r16) * kDw;
    const uint32_t* lsw = reinterpret_cast<const uint32_t*>(sc_w(b)) + ((wn * 4 + g) * 16 + r16) * kDw;
#pragma unroll
    for (int q = 0; q < kDw; ++q) {
      sa[q] = lsa[q];
      sw[q] = lsw[q];
    }
    wait_lgkm();
    wave_barrier();                             // buffer b is free
    load(cur, kt + 2, b);
    __builtin_amdgcn_sched_barrier(0);          // issued before the MFMAs, waited on after them
    if constexpr (MX) {
      static_for<2>([&](auto st_c) {
        constexpr int st = decltype(st_c)::value;
        static_for<kT>([&](auto i_c) {
          constexpr int i = decltype(i_c)::value;
          const u32x4 w = fw[st][i];
          const v8i wo = {(int)w.x, (int)w.y, (int)w.z, (int)w.w, 0, 0, 0, 0};
          static_for<kT>([&](auto j_c) {
            constexpr int j = decltype(j_c)::value;
            const u32x4 x = fa[st][j];
            const v8i xo = {(int)x.x, (int)x.y, (int)x.z, (int)x.w, 0, 0, 0, 0};
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                wo, xo, acc[i][j], 4, 4, 2 * (i & 1) + st, sw[i >> 1], 2 * (j & 1) + st, sa[j >> 1]);
          });
        });
      });
    } else {
      static_for<2>([&](auto st_c) {
        constexpr int st = decltype(st_c)::value;
        v8h da[kT][4];
        auto dequant = [&](v8h (&q)[4], const u32x4& codes, uint32_t scale) {
          const v2h p = e4m3_pair_h<st == 1>(scale);
          const v2h h0 = v2h{p.x, p.x}, h1 = v2h{p.y, p.y};
          q[0] = dq8(codes.x, h0);
          q[1] = dq8(codes.y, h0);
          q[2] = dq8(codes.z, h1);
          q[3] = dq8(codes.w, h1);
        };
#pragma unroll
        for (int j = 0; j < kT; ++j) dequant(da[j], fa[st][j], sa[j]);
#pragma unroll
        for (int i = 0; i < kT; ++i) {
          v8h dw[4];
          dequant(dw, fw[st][i], sw[i]);
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int j = 0; j < kT; ++j)
              acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(dw[k], da[j][k], acc[i][j], 0, 0, 0);
        }
      });
    }
    __builtin_amdgcn_sched_barrier(0);
    store_sc(next, b ^ 1);
    __builtin_amdgcn_s_waitcnt(0x0F70 | kLoads);   // stage kt + 1 has landed; kt + 2 may be in flight
    wait_lgkm();
    wave_barrier();
  };

  Scales s0, s1;
  load(s0, 0, 0);
  load(s1, 1, 1);
  store_sc(s0, 0);
  __builtin_amdgcn_s_waitcnt(0x0F70 | kLoads);
  wait_lgkm();
  wave_barrier();
  // two stages an iteration; an odd count runs one past the end (zeros)
  for (int kt = 0; kt < nk; kt += 2) {
    stage(s0, s1, kt, 0);
    stage(s1, s0, kt + 1, 1);
  }
  wait_dma();                                   // the empty loads' zeros have landed: LDS is free
  __syncthreads();
  float alpha = a.g_d;
  if (!MX) alpha = ((*a.g_a) * a.g_b[e]) * a.g_d;
  store_fused<OUT_BF16, kT, kT, kStripRows>(acc, alpha, a.f, a_row - m0, m0 + wm * 16 * kT, m_rows,
                                            n0 + wn * 16 * kT, N, (int64_t)e * N, a.D, smem + wave * kStrip,
                                            r16, g);
}

template <bool MX, bool SVEC, bool OUT_BF16, bool GROUPED>
hipError_t launch_mid_t(const MidArgs& a, hipStream_t stream) {
  static std::atomic<uint64_t> lds_set{0};
  const hipError_t e = fp4impl::set_lds_limit_once(
      lds_set, reinterpret_cast<const void*>(&k_gemm_mid<MX, SVEC, OUT_BF16, GROUPED>), MidCfg<MX>::kLds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((k_gemm_mid<MX, SVEC, OUT_BF16, GROUPED>), dim3(a.tiles_m * a.tiles_n), dim3(kThreads),
                     MidCfg<MX>::kLds, stream, a);
  return hipGetLastError();
}

template <bool MX, bool GROUPED>
hipError_t launch_mid_m(const MidArgs& a, bool svec, bool out_bf16, hipStream_t stream) {
  if (svec)
    return out_bf16 ? launch_mid_t<MX, true, true, GROUPED>(a, stream)
                    : launch_mid_t<MX, true, false, GROUPED>(a, stream);
  return out_bf16 ? launch_mid_t<MX, false, true, GROUPED>(a, stream)
                  : launch_mid_t<MX, false, false, GROUPED>(a, stream);
}

}  // namespace

namespace fp4impl {

// Modelled time: a fixed part and the fullest CU's tiles times stages.  A lone tile
// takes longer than half a pair: nothing runs while it waits.
double mid_us(bool mx, int64_t groups, double row_tiles, int64_t N, int64_t K) {
  const double tiles = ceil(groups * row_tiles * ((N + kTile - 1) / kTile) / num_cus());
  const int64_t stages = (K + BK - 1) / BK;
  if (tiles <= 1) return mx ? 7.2 + 0.84 * stages : 8.6 + 2.2 * stages;
  return mx ? 7.2 + 0.92 * tiles * stages : 8.6 + 2.07 * tiles * stages;
}

hipError_t launch_mid(bool mx, const uint8_t* A, const uint8_t* a_scales, const float* g_a, const uint8_t* W,
                      const uint8_t* w_scales, const float* g_b, float g_d, int64_t ngroups,
                      const int32_t* offsets, int64_t M, int64_t N, int64_t K, const Epilogue& ep, void* D,
                      bool out_bf16, hipStream_t stream) {
  FusedArgs f{ep.bias, ep.residual, ep.preact, ep.bias_bf16, ep.residual_bf16, ep.preact_bf16,
              ep.activation, ep.gated, 0};
  auto ok16 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
  f.vec = N % 16 == 0 && ok16(ep.bias) && ok16(ep.residual) && ok16(ep.preact) && ok16(D);
  const bool svec = K % BK == 0 && ok16(a_scales) && ok16(w_scales);
  const int64_t tiles_m = (M + kTile - 1) / kTile + ngroups, tiles_n = (N + kTile - 1) / kTile;
  if (tiles_m * tiles_n >= (int64_t)1 << 31) return hipErrorInvalidValue;
  const MidArgs a{A, a_scales, W, w_scales, g_a, g_b, g_d, (int)M, (int)N, (int)K, (int)tiles_m, (int)tiles_n,
                  offsets, (int)ngroups, D, f};
  if (ngroups > 0)
    return mx ? launch_mid_m<true, true>(a, svec, out_bf16, stream)
              : launch_mid_m<false, true>(a, svec, out_bf16, stream);
  return mx ? launch_mid_m<true, false>(a, svec, out_bf16, stream)
            : launch_mid_m<false, false>(a, svec, out_bf16, stream);
}

}  // namespace fp4impl
