// Block-scaled FP4 products through the fused epilogue on 128 x 128 tiles, two
// workgroups per CU, dense and grouped: for outputs that 256 x 256 tiles leave most
// of the device without work.
//
// Work.  A workgroup's 2 x 2 waves own 4 x 4 tiles of 16 x 16 each; K advances 256
// values per stage, in two steps, through two LDS buffers that direct-to-LDS loads
// fill (operand swizzle and edges as in gemm_kernels.h).  The second step's operands
// are read while the first one's MFMAs run; then one barrier, after which the stage's
// buffer is free and the next stage has landed: its first operands are read and the
// stage after next is loaded between the second step's MFMAs.  The other workgroup of
// the CU computes meanwhile: two of 68 (MXFP4) or 72 KB (NVFP4) fit its LDS, and 256
// registers a wave.  MXFP4 multiplies the codes under their E8M0 bytes; NVFP4
// dequantizes both operands to fp16 (exact), each value twice per workgroup, where
// the 256 x 256 tiles do it twice per four times the outputs.
//
// Bound.  NVFP4: the vector issue.  A wave's MFMA takes 17 cycles alone or with 2
// other vector instructions behind it, 29 with 4 (a loop of them); here it has 4.3, and
// the counters give 34 cycles per MFMA, MFMA busy 46% (256 x 256 tiles, 2.3: 26
// cycles, 63%).  MXFP4: LDS and the barriers, MFMA busy a quarter of the time.  Per
// stage 1.8 (NVFP4) and 0.61 us (MXFP4) with a tile per CU, 2.0 and 0.89 us a tile
// with more.  Measured: 1021 x 5120
// x 7168 NVFP4 105 us (256 x 256 tiles 154), MXFP4 41 (57); 128 x 27648 x 5120 47
// (115) and 24 (43); 64 groups of 128 rows x 4096 x 7168 490 (694) and 284 (326).
// 4096 x 4096 x 4096, where the larger tiles fill the device: 134 (117) and 57 (48).
// All operands of a stage read at once, two barriers, loads two stages ahead: 108, 42;
// 55, 26; and eight waves that split a stage's K were slower than these.
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

// A point that no memory access moves across, in either direction: for waits that
// count the loads issued after it.  (The comment marks it in the assembly.)
__device__ __forceinline__ void order_point() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("; order point" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
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
  const int bid = (int)workgroup();
  if (workgroup() >= (uint32_t)T) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int r16 = lane & 15, g = lane >> 4;
  const int rowb = K / 2, nsc = K / (MX ? 32 : 16);

  // ---- this workgroup's tile
  int tm = 0, tn = 0, lo = 0, m_rows = M, e = 0;
  if constexpr (GROUPED) {
    int t, hi = 0;
    xcd_tile(bid, T, t);
    group_tile_of<kTile>(a.offsets, a.groups, M, t / a.tiles_n, e, tm, lo, hi);
    tn = t % a.tiles_n;                         // (uniform too, which the compiler does not see:
                                                // W's loads are in loops that run once)
    m_rows = hi - lo;
    e = __builtin_amdgcn_readfirstlane(e);
    tm = __builtin_amdgcn_readfirstlane(tm);
    lo = __builtin_amdgcn_readfirstlane(lo);
    m_rows = __builtin_amdgcn_readfirstlane(m_rows);
  } else {
    tile_of(bid, a.tiles_m, a.tiles_n, tm, tn);
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
  // stage kt's source ranges; past the last stage empty (zeros, no memory touched)
  auto range_a = [&](int kt) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(pa), 0, kt < nk ? rows_a * rowb : 0, kBufferWord3);
  };
  auto range_w = [&](int kt) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(pw), 0, kt < nk ? rows_w * rowb : 0, kBufferWord3);
  };
  auto load_sc = [&](Scales& s, int kt) {
    load_scales<MX, SVEC>(s, scale_range<SVEC>(psc, kt < nk ? sc_bytes : 0), srow, nsc, kt * BK);
  };
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
  u32x4 f[2][2 * kT];                           // operands of a stage's two steps: A tiles, then W's
  auto read_frag = [&](int b, int st, int x) {
    const uint8_t* tile = x < kT ? tile_a(b) : tile_w(b);
    const int row = x < kT ? ra0 + 16 * x : rw0 + 16 * (x - kT);
    f[st][x] = *reinterpret_cast<const u32x4*>(tile + swz(row, 2 * g + st));
  };
  constexpr int kDw = MX ? 2 : 4;
  auto read_sc = [&](int b, uint32_t (&s)[2][kDw]) {
    const uint32_t* la = reinterpret_cast<const uint32_t*>(sc_a(b)) + ((wm * 4 + g) * 16 + r16) * kDw;
    const uint32_t* lw = reinterpret_cast<const uint32_t*>(sc_w(b)) + ((wn * 4 + g) * 16 + r16) * kDw;
#pragma unroll
    for (int q = 0; q < kDw; ++q) {
      s[0][q] = la[q];
      s[1][q] = lw[q];
    }
  };
  // NVFP4: fp16 operands of the current and the next sub-step, block scale pairs of
  // the two steps
  v8h d[2][2 * kT];
  v2h pair[2][2 * kT];
  auto part = [&](int p, int x, uint32_t codes, const v2h& h, auto k_c, int u) {
    constexpr int k = decltype(k_c)::value;
    const v2h v = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 256.0f, k);
    const v2h r = v * ((u & 2) ? v2h{h.y, h.y} : v2h{h.x, h.x});
    d[p][x][2 * k] = r.x;
    d[p][x][2 * k + 1] = r.y;
  };

  Scales s;
  uint32_t sc[2][kDw];
  load_sc(s, 0);
#pragma unroll
  for (int q = 0; q < kBlocks; ++q) {
    dma_block<SVEC>(range_a(0), tile_a(0), rowb, K, 0, q);
    dma_block<SVEC>(range_w(0), tile_w(0), rowb, K, 0, q);
  }
  order_point();                                // the wait below counts what comes after
  store_sc(s, 0);
  load_sc(s, 1);
#pragma unroll
  for (int q = 0; q < kBlocks; ++q) {
    dma_block<SVEC>(range_a(1), tile_a(1), rowb, K, BK, q);
    dma_block<SVEC>(range_w(1), tile_w(1), rowb, K, BK, q);
  }
  order_point();
  // stage 0 has landed when no more than stage 1's loads, those between the two order
  // points, are in flight (at least 2 kBlocks + 1 instructions: the compiler may join
  // the scale bytes' dwords)
  __builtin_amdgcn_s_waitcnt(0x0F70 | (2 * kBlocks + 1));
  wait_lgkm();
  wave_barrier();
  read_sc(0, sc);
#pragma unroll
  for (int x = 0; x < 2 * kT; ++x) read_frag(0, 0, x);
  if constexpr (!MX) {
    static_for<2 * kT>([&](auto x_c) {
      constexpr int x = decltype(x_c)::value;
      pair[0][x] = e4m3_pair_h<false>(sc[x / kT][x % kT]);
      static_for<4>([&](auto k_c) { part(0, x, f[0][x].x, pair[0][x], k_c, 0); });
    });
  }

  // Stage kt in buffer cb.  Its first step multiplies while the second's operands
  // are read; then the next stage has to have landed, and this stage's buffer is
  // free: its loads (stage kt + 2) and the next stage's first operands go between
  // the second step's MFMAs, each MFMA in a slot of its own with its share of the
  // other work.
  auto stage = [&](int kt, auto cb_c) {
    constexpr int cb = decltype(cb_c)::value, nb = cb ^ 1;
    auto turn = [&] {
      store_sc(s, nb);
      wait_dma();
      wait_lgkm();
      wave_barrier();
      load_sc(s, kt + 2);
    };
    const int k_ld = (kt + 2) * BK;
    auto dma = [&](auto q_c) {
      constexpr int q = decltype(q_c)::value;
      if constexpr (q % 2 == 0) dma_block<SVEC>(range_a(kt + 2), tile_a(cb), rowb, K, k_ld, q / 2);
      else dma_block<SVEC>(range_w(kt + 2), tile_w(cb), rowb, K, k_ld, q / 2);
    };
    if constexpr (MX) {
      uint32_t sn[2][kDw];
      static_for<2>([&](auto st_c) {
        constexpr int st = decltype(st_c)::value;
        static_for<16>([&](auto s_c) {
          constexpr int sl = decltype(s_c)::value, i = sl >> 2, j = sl & 3;
          const u32x4 w = f[st][kT + i], x = f[st][j];
          const v8i wo = {(int)w.x, (int)w.y, (int)w.z, (int)w.w, 0, 0, 0, 0};
          const v8i xo = {(int)x.x, (int)x.y, (int)x.z, (int)x.w, 0, 0, 0, 0};
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              wo, xo, acc[i][j], 4, 4, 2 * (i & 1) + st, sc[1][i >> 1], 2 * (j & 1) + st, sc[0][j >> 1]);
          if constexpr (st == 0 && sl < 2 * kT) read_frag(cb, 1, sl);
          if constexpr (st == 1 && sl < 2 * kBlocks) dma(s_c);
          if constexpr (st == 1 && sl >= 4 && sl < 4 + 2 * kT) read_frag(nb, 0, sl - 4);
          if constexpr (st == 1 && sl == 2) read_sc(nb, sn);
          __builtin_amdgcn_sched_barrier(0);
        });
        if constexpr (st == 0) turn();
      });
#pragma unroll
      for (int q = 0; q < kDw; ++q) {
        sc[0][q] = sn[0][q];
        sc[1][q] = sn[1][q];
      }
    } else {
      // 8 sub-steps of one code dword per tile row, the next one's dequantized meanwhile
      static_for<8>([&](auto u_c) {
        constexpr int u = decltype(u_c)::value, p = u & 1, un = (u + 1) & 7, st = un >> 2;
        if constexpr (u == 4) turn();
        static_for<16>([&](auto s_c) {
          constexpr int sl = decltype(s_c)::value, i = sl >> 2, j = sl & 3, x = sl >> 1;
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(d[p][kT + i], d[p][j], acc[i][j], 0, 0, 0);
          using K0 = std::integral_constant<int, 2 * (sl & 1)>;
          using K1 = std::integral_constant<int, 2 * (sl & 1) + 1>;
          part(p ^ 1, x, f[st][x][un & 3], pair[st][x], K0{}, un);
          part(p ^ 1, x, f[st][x][un & 3], pair[st][x], K1{}, un);
          if constexpr (u == 0 && sl % 2 == 0) read_frag(cb, 1, x);
          if constexpr (u == 1 && sl % 2 == 0) pair[1][x] = e4m3_pair_h<true>(sc[x / kT][x % kT]);
          if constexpr (u == 4 && sl % 2 == 0) dma(std::integral_constant<int, x>{});
          if constexpr (u == 5 && sl % 2 == 0) read_frag(nb, 0, x);
          if constexpr (u == 5 && sl == 1) read_sc(nb, sc);
          if constexpr (u == 6 && sl % 2 == 0) pair[0][x] = e4m3_pair_h<false>(sc[x / kT][x % kT]);
          __builtin_amdgcn_sched_barrier(0);
        });
      });
    }
  };
  // two stages an iteration; an odd count runs one past the end (zeros)
  for (int kt = 0; kt < nk; kt += 2) {
    stage(kt, std::integral_constant<int, 0>{});
    stage(kt + 1, std::integral_constant<int, 1>{});
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
  hipLaunchKernelGGL((k_gemm_mid<MX, SVEC, OUT_BF16, GROUPED>), fp4impl::grid_of((int64_t)a.tiles_m * a.tiles_n), dim3(kThreads),
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

hipError_t launch_mid(bool mx, const uint8_t* A, const uint8_t* a_scales, const float* g_a, const uint8_t* W,
                      const uint8_t* w_scales, const float* g_b, float g_d, int64_t ngroups,
                      const int32_t* offsets, int64_t M, int64_t N, int64_t K, const Epilogue& ep, void* D,
                      bool out_bf16, hipStream_t stream) {
  FusedArgs f{ep.bias, ep.residual, ep.preact, ep.bias_bf16, ep.residual_bf16, ep.preact_bf16,
              ep.activation, ep.gated, 0};
  auto ok16 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
  f.vec = N % 16 == 0 && ok16(ep.bias) && ok16(ep.residual) && ok16(ep.preact) && ok16(D);
  const bool svec = K % BK == 0 && ok16(a_scales) && ok16(w_scales);
  const int64_t tiles_m = (M + kTile - 1) / kTile + (ngroups < M ? ngroups : M), tiles_n = (N + kTile - 1) / kTile;
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
