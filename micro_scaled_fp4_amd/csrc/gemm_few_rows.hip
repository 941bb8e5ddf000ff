// Block-scaled FP4 products of few rows (decode), dense and grouped, through the
// fused epilogue: D = act(alpha A W^T + bias) + residual with at most a few tens
// of rows per group, where W is read once and everything else is small.
//
// Work.  Of a workgroup's 8 waves (one workgroup per CU), KS split K and 8 / KS
// take different 16-row strips of W.  A granule is 16 RT rows of one group
// against 8 / KS strips; the granules of all groups are numbered in a row
// (group, row chunk, strips) and each workgroup takes an equal, contiguous part
// of them, so empty groups cost nothing, full ones spread over the device, and
// the parts differ by one granule at most.  A unit is up to S granules of one
// group: a wave adds its K range for S strips at once, and the KS partial tiles
// meet in LDS once per unit, in wave order.
//
// A wave's K range goes by pairs of 128-value steps.  W is loaded 8 rows x 128
// bytes per instruction (full lines) and turned to the MFMA's operand layout
// through a wave-private XOR-swizzled LDS tile; a pair's loads for all S strips
// are in flight in registers while the pair before it computes, across units
// (72 KB per CU in flight; two pairs ahead ran slower for want of registers).  A's
// codes are read from L2 per pair, in the operand layout, and dequantized once for the
// S strips.
// NVFP4: both operands to fp16 exactly (E2M1 x E4M3 has 6 significant bits),
// v_mfma_f32_16x16x32_f16.  MXFP4: codes and E8M0 bytes straight into
// v_mfma_scale_f32_16x16x128_f8f6f4.  W is the MFMA's first operand, so a lane
// ends with 4 consecutive columns of one row.
//
// Bound: HBM, W's bytes.  1 x 27648 x 5120 NVFP4 20 us, 4.0 TB/s; 16 tokens to 8
// of 64 experts of 4096 x 7168, 0.90 GB of them used, 154 to 160 us, 5.7 TB/s, near
// the card's read rate.  From about 24 rows on the instructions bound it, the unpacking
// of W once per 16 to 64 rows and the loops around the loads (64 experts of 32 rows
// each: 292 us, 213 at the copy's rate).
#include <atomic>

#include "epilogue.h"
#include "fp4_device.h"
#include "fp4_internal.h"
#include "product_choice.h"
#include "scale_bytes.h"

using namespace fp4dev;

namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / 64;
constexpr int kGroup = 4;                       // pairs per group of W scale bytes
constexpr int kLoadNT = 2;                      // buffer load cache policy: nontemporal

struct FewArgs {
  const uint8_t* A;
  const uint8_t* as;
  const uint8_t* W;
  const uint8_t* ws;
  const float* g_a;
  const float* g_b;
  float g_d;
  int M, N, K, ks;                              // ks: waves that split K (1, 2, 4, 8)
  const int32_t* offsets;                       // grouped, else NULL
  int groups;
  void* D;
  FusedArgs f;
};

// LDS: transpose tiles [8 waves][S] x 2 KB | W scale groups [8 waves][S][16 rows]
// x (MXFP4 8, NVFP4 16) kGroup | partial tiles [buffers][8 waves][S][RT] x 1 KB,
// two buffers (alternating by unit) where they fit
constexpr int lds_fixed(bool mx, int S) { return kWaves * S * (2048 + 16 * (mx ? 8 : 16) * kGroup); }
constexpr int red_buffers(bool mx, int RT, int S) {
  return lds_fixed(mx, S) + 2 * kWaves * S * RT * 1024 <= 160 * 1024 ? 2 : 1;
}

// SVEC: scale rows are 16-byte aligned and K is a multiple of 256; else scale
// bytes are read as the aligned dwords that hold them and shifted into place,
// with those past K as zeros.
template <bool MX, int RT, int S, bool SVEC, bool OUT_BF16>
__global__ void __launch_bounds__(kThreads, 1) k_few_rows(FewArgs a) {
  constexpr int kRows = 16 * RT;                // rows of an item
  constexpr int kBufs = red_buffers(MX, RT, S);
  constexpr int kSB = MX ? 8 : 16;              // scale bytes of a row per pair
  constexpr int kSG = kSB * kGroup;             // of a row per group of pairs
  constexpr int kGD = kSG / 16;                 // dwords per lane of a group (MXFP4 2, NVFP4 4)
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  const int r8 = lane >> 3, c8 = lane & 7;
  const int KS = a.ks, slots = kWaves / KS, lslots = 31 - __builtin_clz(slots);
  const int part = wave % KS, slot = wave / KS;
  const int N = a.N, K = a.K;
  const int wrow = K / 2, srow = K / (MX ? 32 : 16);
  const int gran = 16 * slots;                  // W rows per granule
  const int gn = (N + gran - 1) / gran;         // granules per item
  uint8_t* tile = lds + wave * (S * 2048);
  uint8_t* sgl = lds + kWaves * S * 2048 + wave * (S * 16 * kSG);
  v4f* red = reinterpret_cast<v4f*>(lds + lds_fixed(MX, S));

  // ---- this workgroup's units
  const bool grouped = a.offsets != nullptr;
  if (grouped) zero_tail(a.offsets, a.groups, a.M, N, a.f, OUT_BF16, a.D);
  // rows and row chunks of groups c .. c + 63, one per lane
  auto chunk_of = [&](int c, int& lo, int& n, int& inc) {
    const int e = c + lane;
    lo = n = 0;
    if (e < a.groups) {
      lo = min(max(a.offsets[e], 0), a.M);
      n = min(max(a.offsets[e + 1], lo), a.M) - lo;
    }
    inc = (n + kRows - 1) / kRows;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(inc, d, 64);
      if (lane >= d) inc += v;
    }
  };
  int items = (a.M + kRows - 1) / kRows;
  if (grouped) {
    items = 0;
    for (int c = 0; c < a.groups; c += 64) {
      int lo, n, inc;
      chunk_of(c, lo, n, inc);
      items += __shfl(inc, 63, 64);
    }
  }
  const int64_t U = (int64_t)items * gn;
  const int64_t u0 = U * blockIdx.x / gridDim.x, u1 = U * (blockIdx.x + 1) / gridDim.x;
  if (u0 == u1) return;                         // (the whole workgroup)

  // An item: kRows rows of a group.  row0: its first row, rows: how many, e: the
  // group.  Granule u is item u / gn, W rows from (u % gn) gran on.
  struct Item {
    int row0, rows, e;
  };
  auto item_of = [&](int it) {
    Item r{it * kRows, 0, 0};
    if (!grouped) {
      r.rows = min(kRows, a.M - r.row0);
      return r;
    }
    int base = 0;
    for (int c = 0; c < a.groups; c += 64) {
      int lo, n, inc;
      chunk_of(c, lo, n, inc);
      const int mine = (n + kRows - 1) / kRows, start = base + inc - mine;
      const uint64_t hit = __ballot(it >= start && it < start + mine);
      if (hit) {
        const int src = __ffsll((unsigned long long)hit) - 1;
        const int in = (it - __shfl(start, src, 64)) * kRows;
        r.e = c + src;
        r.row0 = __shfl(lo, src, 64) + in;
        r.rows = min(kRows, __shfl(n, src, 64) - in);
        break;
      }
      base += __shfl(inc, 63, 64);
    }
    r.e = __builtin_amdgcn_readfirstlane(r.e);
    r.row0 = __builtin_amdgcn_readfirstlane(r.row0);
    r.rows = __builtin_amdgcn_readfirstlane(r.rows);
    return r;
  };

  // A unit: an item, the first of its W rows and its granules.  next_unit walks
  // this workgroup's units.
  struct Unit {
    Item item;
    int n0, size;
  };
  int64_t left = u1 - u0;
  int at_item = (int)(u0 / gn), at_gran = (int)(u0 - (int64_t)at_item * gn);
  Item item = item_of(at_item);
  auto next_unit = [&]() {
    if (at_gran == gn) {
      at_gran = 0;
      item = item_of(++at_item);
    }
    const Unit u{item, at_gran * gran, (int)min((int64_t)min(S, gn - at_gran), left)};
    at_gran += u.size;
    left -= u.size;
    return u;
  };

  // ---- this wave's pairs [pbeg, pbeg + E): dealt evenly, the longer parts first (E > 0:
  // K > 0, and there are no more waves to split it than pairs)
  const int P = (K + 255) / 256;
  const int pbase = P / KS, prem = P % KS;
  const int pbeg = part * pbase + min(part, prem), E = pbase + (part < prem ? 1 : 0);

  // ---- loads.  Through descriptors whose range is the rows that exist: rows
  // past N or past the item read zeros.  K past the end: only without SVEC,
  // where W reads run into the next row (finite, against A = 0) or off the range.
  struct Elem {
    u32x4 w[S][2];
    u32x4 x[RT][2];
    uint32_t xs[RT][SVEC ? 1 : 2];
    uint32_t sg[S][kGD + (SVEC ? 0 : 1)];       // W scale bytes of the group that starts here
    int xs_first, sg_first;                     // !SVEC: row 0's first byte in the ranges
  };
  Elem el;                                      // the element in flight
  const int w_lane = r8 * wrow + 16 * c8;

  Unit lun{item, 0, 0};                         // its unit
  int le = 0;                                   // next element to load: pair pbeg + le of lun
  bool live = false;                            // el holds an element
  auto load_elem = [&]() {
    // past the last unit: empty ranges, not a branch.  (Units come from the groups' counts
    // by lane shuffles, so the compiler does not see that the ranges are the same in all
    // lanes and puts each load in a loop over the distinct ones, which runs once.)
    if (le == 0) {
      live = left > 0;
      if (live) lun = next_unit();
    }
    const int p = pbeg + le;
    // rows of the unit that exist, from this slot's first on; strip s lies s gran
    // rows further
    const int rows_w = live ? max(0, min(lun.size * gran, N - lun.n0) - 16 * slot) : 0;
    const int rows_a = live ? lun.item.rows : 0;
    const int64_t wr0 = (int64_t)lun.item.e * N + lun.n0 + 16 * slot;
    const __amdgpu_buffer_rsrc_t rw = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t*>(a.W) + wr0 * wrow, 0, rows_w * wrow, kBufferWord3);
    const ScaleRange rs = scale_range<SVEC>(a.ws + wr0 * srow, rows_w * srow);
    const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t*>(a.A) + (int64_t)lun.item.row0 * wrow, 0, rows_a * wrow, kBufferWord3);
    const ScaleRange rsa = scale_range<SVEC>(a.as + (int64_t)lun.item.row0 * srow, rows_a * srow);
    if (le % kGroup == 0) {
      // lane (r16, g): the scale bytes of pair p + g of row r16 of each strip
      // (those past this wave's last pair are never used)
      el.sg_first = rs.lead + kSB * p;
#pragma unroll
      for (int s = 0; s < S; ++s) {
        const int off = (s * gran + r16) * srow + kSB * g;
        if constexpr (!SVEC) {
          const int at = (off + el.sg_first) & ~3;
#pragma unroll
          for (int i = 0; i <= kGD; ++i) el.sg[s][i] = __builtin_amdgcn_raw_buffer_load_b32(rs.rsrc, at + 4 * i, 0, 0);
        } else if constexpr (MX) {
          const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(rs.rsrc, off, kSB * p, 0);
          el.sg[s][0] = v.x;
          el.sg[s][1] = v.y;
        } else {
          const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(rs.rsrc, off, kSB * p, 0);
#pragma unroll
          for (int i = 0; i < 4; ++i) el.sg[s][i] = v[i];
        }
      }
    }
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const int row = 16 * t + r16;
      const int k0 = 256 * p + 64 * g;          // this lane's 64 values of the pair
      el.x[t][0] = __builtin_amdgcn_raw_buffer_load_b128(ra, SVEC || k0 < K ? row * wrow + k0 / 2 : kOutOfRange, 0, 0);
      el.x[t][1] = __builtin_amdgcn_raw_buffer_load_b128(
          ra, SVEC || k0 + 32 < K ? row * wrow + k0 / 2 + 16 : kOutOfRange, 0, 0);
      const int b0 = row * srow + (kSB / 4) * g;
      if constexpr (!SVEC) {
        el.xs_first = rsa.lead + kSB * p;
        const int at = (b0 + el.xs_first) & ~3;
        el.xs[t][0] = __builtin_amdgcn_raw_buffer_load_b32(rsa.rsrc, at, 0, 0);
        el.xs[t][1] = __builtin_amdgcn_raw_buffer_load_b32(rsa.rsrc, at + 4, 0, 0);
      } else if constexpr (MX) {
        el.xs[t][0] = __builtin_amdgcn_raw_buffer_load_b16(rsa.rsrc, b0, kSB * p, 0);
      } else {
        el.xs[t][0] = __builtin_amdgcn_raw_buffer_load_b32(rsa.rsrc, b0, kSB * p, 0);
      }
    }
#pragma unroll
    for (int s = 0; s < S; ++s) {
      el.w[s][0] = __builtin_amdgcn_raw_buffer_load_b128(rw, w_lane + s * gran * wrow, 128 * p, kLoadNT);
      el.w[s][1] = __builtin_amdgcn_raw_buffer_load_b128(rw, w_lane + (s * gran + 8) * wrow, 128 * p, kLoadNT);
    }
    if (++le == E) le = 0;
  };

  v4f acc[S][RT];
  auto clear = [&]() {
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
      for (int t = 0; t < RT; ++t) acc[s][t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  };

  // ---- end of unit cun: partial tiles to LDS, then outputs by all threads, two
  // columns each
  Unit cun = lun;                               // unit being computed
  int parity = 0;
  const int cap = 31 - __builtin_clz(S * gran / 2);   // column pairs of a full unit: 1 << cap
  auto finish = [&]() {
    if (kBufs == 1) __syncthreads();            // the previous unit's tiles have been read
    v4f* buf = red + parity * kWaves * S * RT * 64;
    if (kBufs == 2) parity ^= 1;
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
      for (int t = 0; t < RT; ++t) buf[((wave * S + s) * RT + t) * 64 + lane] = acc[s][t];
    float alpha = a.g_d;
    if (!MX) alpha = ((*a.g_a) * a.g_b[cun.item.e]) * a.g_d;
    __syncthreads();
    const int cols = min(cun.size * gran, N - cun.n0);
    for (int i = threadIdx.x; i < cun.item.rows << cap; i += kThreads) {
      const int m = i >> cap, c = 2 * (i - (m << cap));          // row and first column inside the unit
      const int n = cun.n0 + c;
      if (c >= cols) continue;
      // (gran and the slots are powers of two)
      const int s = c >> (4 + lslots), sl = (c >> 4) & (slots - 1), q = c & 3, gg = (c & 15) >> 2;
      // lane (m % 16, gg), elements q and q + 1 of tile (s, m / 16) of the slot's waves
      const float* v = reinterpret_cast<const float*>(buf) +
                       (((sl * KS * S + s) * RT + m / 16) * 64 + gg * 16 + (m & 15)) * 4 + q;
      float z0 = v[0], z1 = v[1];
      for (int k = 1; k < KS; ++k) {
        z0 += v[k * S * RT * 256];
        z1 += v[k * S * RT * 256 + 1];
      }
      const int64_t row = cun.item.row0 + m;
      const int64_t b0 = (int64_t)cun.item.e * N + n;
      const bool both = n + 1 < N;
      z0 = fmaf(z0, alpha, a.f.bias != nullptr ? load1(a.f.bias, b0, a.f.bias_bf16) : 0.0f);
      z1 = fmaf(z1, alpha, a.f.bias != nullptr && both ? load1(a.f.bias, b0 + 1, a.f.bias_bf16) : 0.0f);
      if (a.f.preact != nullptr) {
        store1(a.f.preact, row * N + n, a.f.preact_bf16, z0);
        if (both) store1(a.f.preact, row * N + n + 1, a.f.preact_bf16, z1);
      }
      with_act(a.f.activation, [&](auto act) {
        constexpr int ACT = decltype(act)::value;
        if (a.f.gated) {
          const int64_t o = row * (N / 2) + n / 2;
          float d = act_value<ACT>(z0) * z1;
          if (a.f.residual != nullptr) d += load1(a.f.residual, o, a.f.residual_bf16);
          store1(a.D, o, OUT_BF16, d);
        } else {
          const int64_t o = row * N + n;
          float d0 = act_value<ACT>(z0), d1 = act_value<ACT>(z1);
          if (a.f.residual != nullptr) d0 += load1(a.f.residual, o, a.f.residual_bf16);
          if (a.f.residual != nullptr && both) d1 += load1(a.f.residual, o + 1, a.f.residual_bf16);
          store1(a.D, o, OUT_BF16, d0);
          if (both) store1(a.D, o + 1, OUT_BF16, d1);
        }
      });
    }
  };

  // ---- one element: the group's scale bytes to LDS, strip by strip through the
  // tile, the ring slot refilled once its registers are in LDS
  const int wsw = (r8 ^ c8) << 4;
  const int rd = r16 * 128;
  int ce = 0;                                   // pair being computed
  // 32 values of step st (two 16-value blocks; scale: the pair's 4 bytes) to fp16
  auto dequant = [&](v8h (&q)[4], const u32x4& codes, uint32_t scale, int st) {
    const v2h p = st ? e4m3_pair_h<true>(scale) : e4m3_pair_h<false>(scale);
    const v2h h0 = v2h{p.x, p.x}, h1 = v2h{p.y, p.y};
    q[0] = dq8(codes.x, h0);
    q[1] = dq8(codes.y, h0);
    q[2] = dq8(codes.z, h1);
    q[3] = dq8(codes.w, h1);
  };
  auto elem = [&]() {
    if (ce == 0) cun = lun;                     // el is its first pair
    if (ce % kGroup == 0) {
#pragma unroll
      for (int s = 0; s < S; ++s) {
        uint32_t v[kGD];
        if constexpr (SVEC) {
#pragma unroll
          for (int i = 0; i < kGD; ++i) v[i] = el.sg[s][i];
        } else {
          place_bytes<kGD>(v, el.sg[s], ((16 * s + r16) * srow + kSB * g + el.sg_first) & 3,
                           srow - kSB * (pbeg + ce + g));
        }
        uint8_t* dst = sgl + (16 * s + r16) * kSG + kSB * g;
        if constexpr (MX)
          *reinterpret_cast<u32x2*>(dst) = u32x2{v[0], v[1]};
        else
          *reinterpret_cast<u32x4*>(dst) = u32x4{v[0], v[1], v[2], v[3]};
      }
    }
    // W's codes through the tiles, all strips at once: one LDS round trip per element
#pragma unroll
    for (int s = 0; s < S; ++s) {
      uint8_t* tb = tile + s * 2048;
      *reinterpret_cast<u32x4*>(tb + r8 * 128 + wsw) = el.w[s][0];
      *reinterpret_cast<u32x4*>(tb + (8 + r8) * 128 + (wsw ^ 64)) = el.w[s][1];
    }
    u32x4 codes[S][2];
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
      for (int st = 0; st < 2; ++st) {
        const int c = 2 * g + st;
        codes[s][st] = *reinterpret_cast<const u32x4*>(
            tile + s * 2048 + rd + ((c ^ (r16 & 7) ^ ((r16 >> 3) << 2)) << 4));
      }
    u32x4 xc[RT][2];
    uint32_t xs[RT], wsb[S];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      xc[t][0] = el.x[t][0];
      xc[t][1] = el.x[t][1];
      if constexpr (SVEC) {
        xs[t] = el.xs[t][0];
      } else {
        uint32_t v[1];
        place_bytes<1>(v, el.xs[t], ((16 * t + r16) * srow + (kSB / 4) * g + el.xs_first) & 3,
                       srow - kSB * (pbeg + ce) - (kSB / 4) * g);
        xs[t] = v[0];
      }
    }
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const uint8_t* src = sgl + (16 * s + r16) * kSG + kSB * (ce % kGroup) + (kSB / 4) * g;
      wsb[s] = MX ? (uint32_t)*reinterpret_cast<const uint16_t*>(src) : *reinterpret_cast<const uint32_t*>(src);
    }
    load_elem();                                // el's registers are in use no more
#pragma unroll
    for (int st = 0; st < 2; ++st) {
      if constexpr (MX) {
#pragma unroll
        for (int s = 0; s < S; ++s) {
          const u32x4 c = codes[s][st];
          const v8i wo = {(int)c.x, (int)c.y, (int)c.z, (int)c.w, 0, 0, 0, 0};
#pragma unroll
          for (int t = 0; t < RT; ++t) {
            const u32x4 x = xc[t][st];
            const v8i xo = {(int)x.x, (int)x.y, (int)x.z, (int)x.w, 0, 0, 0, 0};
            acc[s][t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                wo, xo, acc[s][t], 4, 4, 0, st ? wsb[s] >> 8 : wsb[s], 0, st ? xs[t] >> 8 : xs[t]);
          }
        }
      } else {
        // the operand with fewer 16-row tiles stays dequantized, the other passes by
        constexpr bool kHoldX = RT <= S;
        constexpr int H = kHoldX ? RT : S, O = kHoldX ? S : RT;
        v8h hold[H][4];
#pragma unroll
        for (int h = 0; h < H; ++h) dequant(hold[h], kHoldX ? xc[h][st] : codes[h][st], kHoldX ? xs[h] : wsb[h], st);
#pragma unroll
        for (int o = 0; o < O; ++o) {
          v8h pass[4];
          dequant(pass, kHoldX ? codes[o][st] : xc[o][st], kHoldX ? wsb[o] : xs[o], st);
#pragma unroll
          for (int h = 0; h < H; ++h)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              v4f& c = kHoldX ? acc[o][h] : acc[h][o];
              c = __builtin_amdgcn_mfma_f32_16x16x32_f16(kHoldX ? pass[k] : hold[h][k],
                                                         kHoldX ? hold[h][k] : pass[k], c, 0, 0, 0);
            }
        }
      }
    }
    if (++ce == E) {
      ce = 0;
      finish();
      clear();
    }
  };

  clear();
  load_elem();
  while (live) elem();
}

template <bool MX, int RT, int S, bool SVEC, bool OUT_BF16>
hipError_t launch_t(const FewArgs& a, hipStream_t stream) {
  constexpr int lds = lds_fixed(MX, S) + red_buffers(MX, RT, S) * kWaves * S * RT * 1024;
  static_assert(lds <= 160 * 1024, "LDS");
  static std::atomic<uint64_t> lds_set{0};
  const hipError_t e = fp4impl::set_lds_limit_once(
      lds_set, reinterpret_cast<const void*>(&k_few_rows<MX, RT, S, SVEC, OUT_BF16>), lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((k_few_rows<MX, RT, S, SVEC, OUT_BF16>), dim3(fp4impl::num_cus()), dim3(kThreads),
                     lds, stream, a);
  return hipGetLastError();
}

template <bool MX, int RT, int S>
hipError_t launch_s(const FewArgs& a, bool svec, bool out_bf16, hipStream_t stream) {
  if (svec) return out_bf16 ? launch_t<MX, RT, S, true, true>(a, stream) : launch_t<MX, RT, S, true, false>(a, stream);
  return out_bf16 ? launch_t<MX, RT, S, false, true>(a, stream) : launch_t<MX, RT, S, false, false>(a, stream);
}

template <bool MX>
hipError_t launch_m(const FewArgs& a, int item, bool svec, bool out_bf16, hipStream_t stream) {
  if (item == 16) return launch_s<MX, 1, 4>(a, svec, out_bf16, stream);
  if (item == 32) return launch_s<MX, 2, 4>(a, svec, out_bf16, stream);
  return launch_s<MX, 4, 2>(a, svec, out_bf16, stream);
}

}  // namespace

namespace fp4impl {

hipError_t launch_few_rows(bool mx, const uint8_t* A, const uint8_t* a_scales, const float* g_a,
                           const uint8_t* W, const uint8_t* w_scales, const float* g_b, float g_d,
                           int64_t ngroups, const int32_t* offsets, int64_t M, int64_t N, int64_t K,
                           const Epilogue& ep, void* D, bool out_bf16, int item, hipStream_t stream) {
  const FusedArgs f{ep.bias, ep.residual, ep.preact, ep.bias_bf16, ep.residual_bf16, ep.preact_bf16,
                    ep.activation, ep.gated, 0};
  const FewArgs a{A, a_scales, W, w_scales, g_a, g_b, g_d, (int)M, (int)N, (int)K, few_rows_split(K), offsets,
                  (int)ngroups, D, f};
  const bool svec = K % 256 == 0 && (reinterpret_cast<uintptr_t>(a_scales) & 15) == 0 &&
                    (reinterpret_cast<uintptr_t>(w_scales) & 15) == 0;
  return mx ? launch_m<true>(a, item, svec, out_bf16, stream)
            : launch_m<false>(a, item, svec, out_bf16, stream);
}

}  // namespace fp4impl
