// Attention over a paged key/value cache in FP4 (include/fp4.h, kv_cache_attention): the
// choice of kernel, and the kernel that joins the parts of long contexts.
#include <algorithm>
#include <type_traits>

#include "fp4_device.h"
#include "fp4_internal.h"
#include "grid.h"
#include "kv_attention.h"
#include "kv_attention_few.h"
#include "kv_attention_tiles.h"

using namespace fp4dev;
using fp4impl::AttendProblem;
using fp4impl::KvCache;
using fp4impl::TileParts;
using fp4impl::UnitPlan;

namespace {

// Joins the parts of four rows of a tile that was cut: the mean of their outputs by their shares of the
// row's sum.  Wave w finds the shares of row w's parts; then each wave sums every fourth part's four
// rows, a lane DP / 64 channels, and the waves' sums meet in LDS.  The order of the parts is fixed, so the same call gives the same bits.
// Bound by its launch and two chains of loads for few parts (4.6 us), by the bytes of many (113 MB of
// parts read and 17 written in 39 us: 3.3 TB/s); holding all of a part's loads in registers halves the
// waves (5 -> 12 us for 256 tiles of 4 parts).
template <int DP>
__global__ void __launch_bounds__(256) k_join_parts(KvCache c, AttendProblem a, UnitPlan p, int groups) {
  constexpr int kChunk = 256, kPer = DP / 64;
  typedef float fv __attribute__((ext_vector_type(kPer)));
  __shared__ float weight[4][kChunk];
  __shared__ __align__(16) float sums[4][4][DP];
  const TileParts* tiles = static_cast<const TileParts*>(p.tiles);
  const int at = workgroup() / groups, group = workgroup() % groups;     // `groups` workgroups a tile
  const int slot = at / c.heads, head = at % c.heads;
  if (slot >= p.max_slots) return;
  const int slots = tiles[p.max_slots].begin;
  const TileParts t = tiles[slot];
  if (slot >= slots || slots > p.max_slots || t.count <= 1 || t.part0 < 0 || t.part0 + t.count > p.max_parts) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const float* const first = part_of(p, c.heads, head, t.part0, DP);
  const int64_t stride = part_of(p, c.heads, head, t.part0 + 1, DP) - first;
  for (int q0 = 4 * group; q0 < t.rows; q0 += 4 * groups) {
    // the row's maximum and sum, and of these each part's share
    const float* const stats = first + 2 * (q0 + wave);
    float mine = -INFINITY, l = 0;
    for (int k = lane; k < t.count; k += 64) {
      const float m = stats[k * stride], was = mine;
      mine = fmaxf(was, m);
      const float base = mine == -INFINITY ? 0.0f : mine;
      l = l * __builtin_amdgcn_exp2f(was - base) + stats[k * stride + 1] * __builtin_amdgcn_exp2f(m - base);
    }
    float top = mine;
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, 64));
    const float base = top == -INFINITY ? 0.0f : top;
    l *= __builtin_amdgcn_exp2f(mine - base);
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) l += __shfl_xor(l, off, 64);
    const float inverse = inverse_of(l);
    fv sum[4] = {};
    for (int k0 = 0; k0 < t.count; k0 += kChunk) {
      const int n = min(kChunk, t.count - k0);
      __syncthreads();
      for (int k = lane; k < n; k += 64) {
        const float* const left = stats + (k0 + k) * stride;
        weight[wave][k] = left[1] * __builtin_amdgcn_exp2f(left[0] - base) * inverse;
      }
      __syncthreads();
      const float* const from = first + k0 * stride + 2 * p.rows + q0 * DP + lane * kPer;
#pragma unroll 6
      for (int k = wave; k < n; k += 4) {
#pragma unroll
        for (int r = 0; r < 4; ++r) sum[r] += *reinterpret_cast<const fv*>(from + k * stride + r * DP) * weight[r][k];
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) *reinterpret_cast<fv*>(&sums[wave][r][lane * kPer]) = sum[r];
    __syncthreads();
    const int q = q0 + wave, rho = t.first_row + q, i = rho / p.group;
    if (q < t.rows) {
      const int64_t row = (int64_t)(t.begin + i) * a.q_heads + head * p.group + (rho - i * p.group);
      if (4 * lane < c.dim) {
        f32x4 v{0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < 4; ++w) v += *reinterpret_cast<const f32x4*>(&sums[w][wave][4 * lane]);
        store4(a.out, a.out_bf16, row * c.dim + 4 * lane, v);
      }
      if (lane == 0 && a.lse != nullptr) a.lse[row] = row_lse(top, l);
    }
    __syncthreads();
  }
}

// Lays more than kLaneSeqs sequences out, for unit_of: one workgroup, each thread a run of them.  Bound by
// its launch and chains of loads; with it one token each of 65, 128, 256, 512 and 4096 sequences of 1000
// positions (8 heads x 128) takes 39, 50, 85, 154 and 1046 us, laid out by every wave for itself, in an
// earlier state, 34, 48, 88, 208 and 5704.  (So both cost the same near 128; a lane for each sequence
// ends at 64.)
constexpr int kLayOutThreads = 1024, kLayOutWaves = kLayOutThreads / 64;
__global__ void __launch_bounds__(kLayOutThreads) k_lay_out(KvCache c, UnitPlan p) {
  __shared__ float sums[kLayOutWaves];
  __shared__ int scans[3][kLayOutWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int run = (c.seqs + kLayOutThreads - 1) / kLayOutThreads;
  const int b0 = min((int)threadIdx.x * run, c.seqs), b1 = min(b0 + run, c.seqs);
  const SeqSize mine = b0 < b1 ? seq_size(c, p, b0) : SeqSize{0, 0, 0, 0, 1};
  auto each = [&](auto f) {
    if (b0 < b1) f(b0, mine);
    for (int b = b0 + 1; b < b1; ++b) f(b, seq_size(c, p, b));
  };
  // over all threads, the same in all
  auto joined = [&](float v, auto f) {
    __syncthreads();
    if (lane == 0) sums[wave] = v;
    __syncthreads();
    float r = sums[0];
    for (int w = 1; w < kLayOutWaves; ++w) r = f(r, sums[w]);
    return r;
  };
  auto sum = [&](float v) { return joined(sum_lanes(v), [](float x, float y) { return x + y; }); };
  Totals all{0, 0, 0};
  float seen = 0;
  each([&](int, const SeqSize& s) {
    all.work += (float)s.tiles * (float)s.steps;
    seen += seen_steps(p, s);
    all.tiles += (float)s.tiles;
    all.longest = fmaxf(all.longest, s.tiles > 0 ? (float)s.steps : 0.0f);
  });
  all = {sum(all.work), sum(all.tiles), joined(max_lanes(all.longest), [](float x, float y) { return fmaxf(x, y); })};
  if (!fits(p, all)) {
    if (threadIdx.x == 0) p.layout[c.seqs] = {0, 0, fp4impl::kNoLayout, 1};
    return;
  }
  const float whole = p.turn > 1 ? whole_time(p, all) : whole_time(p, all, sum(seen));
  const int per = part_steps(p, all, whole, [&](float inverse) {
    float units = 0;
    each([&](int, const SeqSize& s) { units += (float)s.tiles * parts_at((float)s.steps, inverse); });
    return sum(units);
  });
  int own[3] = {0, 0, 0}, to[3];
  auto add = [&](const SeqSize& s) {
    const int count = parts_of(s.steps, per);
    own[0] += s.tiles * count;
    own[1] += count > 1 ? s.tiles * count : 0;
    own[2] += s.tiles;
  };
  each([&](int, const SeqSize& s) { add(s); });
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    to[i] = scan_lanes(own[i]);
    if (lane == 63) scans[i][wave] = to[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    for (int w = 0; w < wave; ++w) to[i] += scans[i][w];
    own[i] = to[i] - own[i];                    // before this thread's first
  }
  if (threadIdx.x == kLayOutThreads - 1) p.layout[c.seqs] = {to[0], to[1], to[2], per};
  each([&](int b, const SeqSize& s) {
    p.layout[b] = {own[0], own[1], own[2], 0};
    add(s);
  });
}

int padded_dim(int dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : 256; }

// Packed rows of a tile, by the mean of the sequences' rows.  16 sequences of 8192 positions, 8 heads, us:
//   rows per head        16    32    64   128
//   D 128, bf16: 16      41    59   107   182
//                32      48    51    81   134
//               128      87    90    96   113
//   D 128, f32:  16      46    73   125   231   (128: 128, 131, 142, 170)
//   D 256, bf16: 16      88   140   261   503   (128: 269, 275, 284, 302; a 32-row kernel: 280, 285, 469, 861)
// (float32 and 256 channels leave a SIMD one wave of the 32-row kernel).
int tile_rows(int64_t T, int64_t seqs, int group, int dp, bool split) {
  const int64_t rows = T * group;
  if (rows > 64 * seqs) return 128;
  return rows <= 16 * seqs || dp == 256 || split ? 16 : 32;
}

// Workgroups that a compute unit holds, by their registers and LDS (a wave of each on each SIMD).  (Tiles of 128
// rows of 64 channels would fit three times but for MXFP4 in float32; rounds are planned for two.)
int resident(int rows, int dp, bool split) {
  if (rows == 128) return dp == 256 ? 1 : 2;
  if (rows == 32) return dp == 64 ? 3 : 2;
  return dp == 64 ? 4 : dp == 128 ? (split ? 2 : 3) : 1;
}

UnitPlan plan_of(int64_t T, int64_t seqs, int q_heads, int heads, int dp, bool split) {
  UnitPlan p{};
  p.group = q_heads / heads;
  p.rows = tile_rows(T, seqs, p.group, dp, split);
  p.target = std::max(1, resident(p.rows, dp, split) * fp4impl::num_cus() / heads);
  p.max_slots = (int)(T * p.group / p.rows + seqs);
  // Few rows: parts of 4 steps, one for each wave (one token, 32 / 8 heads x 128, replayed: 1000 positions 11.2
  // us against 13.4 with parts of 8; 4096 12.2, 13.6; 16384, 64 parts of 4 or 32 of 8, 16.4, 14.6; with a
  // join 0.3 us shorter than now), joining them for 9 steps' time (32 sequences of 1000, not cut, 18.5 us; cut by a cost
  // of 5 20.1; 1000 positions left whole by a cost of 14 15.0).  Where few tiles can be cut evenly one round is enough, and no
  // workgroups wait for nothing; else 2 (1, 2, 3 rounds: 128 sequences of 1000 to 16000 173, 165, 173 us).
  // Tiles of 128 rows: a round's parts are 34 MB to write and read, 14 steps' time (a prompt of 1024 whole
  // 37 us, in two parts 54).  Up to 4 rounds level batches like two chunks over 16384 and 32768
  // positions (uncut 520 steps, in 3 rounds 3 x 132).
  const bool few = p.rows < 128;
  p.min_per = few ? 4 : 8;
  p.whole = 8;
  p.turn = few ? 4 : 1;
  p.join = few ? 9 : 14;
  p.rounds = few ? (4 * p.max_slots <= p.target ? 1 : 2) : 4;
  p.max_parts = std::max(p.rounds, 2) * p.target + p.target / 8 + 8;
  return p;
}

size_t tiles_bytes(const UnitPlan& p) { return (size_t)(p.max_slots + 1) * sizeof(TileParts); }

size_t layout_bytes(int64_t seqs) { return seqs > fp4impl::kLaneSeqs ? (size_t)(seqs + 1) * sizeof(int4) : 0; }

// The most parts of a tile that the page table has positions for, and units of a head.
int64_t most_parts(const KvCache& c, const UnitPlan& p) {
  const int steps = (c.capacity + 63) / 64;
  return steps <= p.whole ? 1 : (steps + p.min_per - 1) / p.min_per;
}
int64_t most_units(const KvCache& c, const UnitPlan& p) {
  return std::min(p.max_slots * most_parts(c, p),
                  std::max((int64_t)p.max_slots + p.target, (int64_t)p.rounds * p.target) + fp4impl::kSpareUnits);
}

template <int DP, bool MX, bool QBF, bool SPLIT>
void launch(const KvCache& c, const AttendProblem& a, const UnitPlan& p, hipStream_t stream) {
  const dim3 grid = fp4impl::grid_of(most_units(c, p) * c.heads);
  if (p.rows == 16) {
    k_attend_few<DP, MX, QBF, SPLIT, 1><<<grid, 256, 0, stream>>>(c, a, p);
    return;
  }
  if constexpr (DP < 256 && !SPLIT) {
    if (p.rows == 32) {
      k_attend_few<DP, MX, QBF, SPLIT, 2><<<grid, 256, 0, stream>>>(c, a, p);
      return;
    }
  }
  k_attend_tiles<DP, MX, QBF, SPLIT><<<grid, 256, 0, stream>>>(c, a, p);
}

template <int DP>
void launch_dp(const KvCache& c, const AttendProblem& a, const UnitPlan& p, hipStream_t stream) {
  const bool split = !a.q_bf16 || !a.out_bf16;
  auto go = [&](auto mx) {
    if (!a.q_bf16) launch<DP, mx.value, false, true>(c, a, p, stream);
    else if (split) launch<DP, mx.value, true, true>(c, a, p, stream);
    else launch<DP, mx.value, true, false>(c, a, p, stream);
  };
  if (c.mx) go(std::true_type{});
  else go(std::false_type{});
  if (most_parts(c, p) <= 1) return;
  // (25 rows of 8 heads over each of 16 sequences: 6.0 us with 8 workgroups a tile of 32 rows, 7.3 with 4; tiles
  // of 128 rows are bound by the parts' bytes: 264 of them in 2 parts 20 us with 4, 23 with 16)
  const int groups = p.rows < 128 ? p.rows / 4 : 4;
  k_join_parts<DP><<<fp4impl::grid_of((int64_t)p.max_slots * c.heads * groups), 256, 0, stream>>>(c, a, p, groups);
}

}  // namespace

namespace fp4impl {

size_t kv_attention_workspace_bytes(int64_t T, int64_t seqs, int q_heads, int heads, int dim) {
  // (the most that any types of q and out take)
  const int dp = padded_dim(dim);
  size_t most = 0;
  for (bool split : {false, true}) {
    const UnitPlan p = plan_of(T, seqs, q_heads, heads, dp, split);
    most = std::max(most, tiles_bytes(p) + layout_bytes(seqs) + (size_t)p.max_parts * heads * p.rows * (dp + 2) * 4);
  }
  return most;
}

hipError_t launch_kv_attention(const KvCache& c, const AttendProblem& a, hipStream_t stream) {
  const int dp = padded_dim(c.dim);
  UnitPlan p = plan_of(c.rows, c.seqs, a.q_heads, c.heads, dp, !a.q_bf16 || !a.out_bf16);
  p.causal = a.causal;
  p.window = a.window;
  p.tiles = a.workspace;
  p.layout = reinterpret_cast<int4*>(static_cast<char*>(a.workspace) + tiles_bytes(p));
  p.parts = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + tiles_bytes(p) + layout_bytes(c.seqs));
  if (c.seqs > kLaneSeqs) {
    k_lay_out<<<1, kLayOutThreads, 0, stream>>>(c, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (dp == 64) launch_dp<64>(c, a, p, stream);
  else if (dp == 128) launch_dp<128>(c, a, p, stream);
  else launch_dp<256>(c, a, p, stream);
  return hipGetLastError();
}

}  // namespace fp4impl
