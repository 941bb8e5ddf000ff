// Attention over a paged key/value cache in FP4 (include/fp4.h, kv_cache_attention): the
// choice of kernel, and the kernel that joins the parts of long contexts.
#include <type_traits>

#include "fp4_device.h"
#include "fp4_internal.h"
#include "grid.h"
#include "kv_attention.h"
#include "kv_attention_few.h"

using namespace fp4dev;
using fp4impl::AttendProblem;
using fp4impl::KvCache;
using fp4impl::TileParts;
using fp4impl::UnitPlan;

namespace {

// One workgroup per tile and head: rows of tiles cut into parts, 16 threads a row.
__global__ void __launch_bounds__(256) k_join_parts(KvCache c, AttendProblem a, UnitPlan p, int dp, bool out_vec) {
  const int slot = workgroup() / c.heads, head = workgroup() % c.heads;
  const TileParts* tiles = static_cast<const TileParts*>(p.tiles);
  const int slots = tiles[p.max_slots].begin;
  if (slot >= slots || slots > p.max_slots) return;
  const TileParts t = tiles[slot];
  if (t.count <= 1 || t.part0 < 0 || t.part0 + t.count > p.max_parts) return;
  const int c16 = threadIdx.x & 15;
  for (int q = threadIdx.x >> 4; q < t.rows; q += 16) {
    const int rho = t.first_row + q, i = rho / p.group;
    const int64_t at = (int64_t)(t.begin + i) * a.q_heads + head * p.group + (rho - i * p.group);
    float top = -INFINITY, total = 0;
    for (int k = 0; k < t.count; ++k) top = fmaxf(top, part_of(p, c.heads, head, t.part0 + k, dp)[2 * q]);
    const float base = top == -INFINITY ? 0.0f : top;
    f32x4 sum[4] = {};
    for (int k = 0; k < t.count; ++k) {
      const float* left = part_of(p, c.heads, head, t.part0 + k, dp);
      const float w = __builtin_amdgcn_exp2f(left[2 * q] - base);
      total += left[2 * q + 1] * w;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (4 * (c16 + 16 * j) < c.dim) sum[j] += *reinterpret_cast<const f32x4*>(left + 2 * p.rows + q * dp + 4 * (c16 + 16 * j)) * w;
    }
    const float inverse = total > 0 ? 1.0f / total : 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (4 * (c16 + 16 * j) < c.dim) store4(a.out, a.out_bf16, out_vec, at * c.dim + 4 * (c16 + 16 * j), sum[j] * inverse);
    if (c16 == 0 && a.lse != nullptr) a.lse[at] = row_lse(top, total);
  }
}

int padded_dim(int dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : 256; }

// Packed rows of a tile.
int tile_rows(int64_t T, int64_t seqs, int group) { return T * group <= 16 * seqs ? 16 : 32; }

UnitPlan plan_of(int64_t T, int64_t seqs, int q_heads, int heads) {
  UnitPlan p{};
  p.group = q_heads / heads;
  p.rows = tile_rows(T, seqs, p.group);
  p.min_per = 4;
  p.target = (4 * fp4impl::num_cus() + heads - 1) / heads;
  p.max_slots = (int)(T * p.group / p.rows + seqs);
  p.max_parts = 2 * p.target + p.target / 8 + 8;
  return p;
}

size_t tiles_bytes(const UnitPlan& p) { return (size_t)(p.max_slots + 1) * sizeof(TileParts); }

template <int DP, bool MX, bool QBF, bool SPLIT>
void launch(const KvCache& c, const AttendProblem& a, const UnitPlan& p, bool q_vec, bool out_vec, hipStream_t stream) {
  const dim3 grid = fp4impl::grid_of(((int64_t)p.max_slots + p.target + fp4impl::kSpareUnits) * c.heads);
  if (p.rows == 16) k_attend_few<DP, MX, QBF, SPLIT, 1><<<grid, 256, 0, stream>>>(c, a, p, q_vec, out_vec);
  else k_attend_few<DP, MX, QBF, SPLIT, 2><<<grid, 256, 0, stream>>>(c, a, p, q_vec, out_vec);
}

template <int DP>
void launch_dp(const KvCache& c, const AttendProblem& a, const UnitPlan& p, bool q_vec, bool out_vec, hipStream_t stream) {
  const bool split = !a.q_bf16 || !a.out_bf16;
  auto go = [&](auto mx) {
    if (!a.q_bf16) launch<DP, mx.value, false, true>(c, a, p, q_vec, out_vec, stream);
    else if (split) launch<DP, mx.value, true, true>(c, a, p, q_vec, out_vec, stream);
    else launch<DP, mx.value, true, false>(c, a, p, q_vec, out_vec, stream);
  };
  if (c.mx) go(std::true_type{});
  else go(std::false_type{});
}

}  // namespace

namespace fp4impl {

size_t kv_attention_workspace_bytes(int64_t T, int64_t seqs, int q_heads, int heads, int dim) {
  const UnitPlan p = plan_of(T, seqs, q_heads, heads);
  return tiles_bytes(p) + (size_t)p.max_parts * heads * p.rows * (padded_dim(dim) + 2) * 4;
}

hipError_t launch_kv_attention(const KvCache& c, const AttendProblem& a, hipStream_t stream) {
  UnitPlan p = plan_of(c.rows, c.seqs, a.q_heads, c.heads);
  p.causal = a.causal;
  p.window = a.window;
  p.tiles = a.workspace;
  p.parts = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + tiles_bytes(p));
  auto multiple = [](const void* x, int64_t n) { return reinterpret_cast<uintptr_t>(x) % n == 0; };
  const bool q_vec = multiple(a.q, 16) && a.q_stride * (a.q_bf16 ? 2 : 4) % 16 == 0;
  const bool out_vec = multiple(a.out, a.out_bf16 ? 8 : 16);
  const int dp = padded_dim(c.dim);
  if (dp == 64) launch_dp<64>(c, a, p, q_vec, out_vec, stream);
  else if (dp == 128) launch_dp<128>(c, a, p, q_vec, out_vec, stream);
  else launch_dp<256>(c, a, p, q_vec, out_vec, stream);
  k_join_parts<<<grid_of((int64_t)p.max_slots * c.heads), 256, 0, stream>>>(c, a, p, dp, out_vec);
  return hipGetLastError();
}

}  // namespace fp4impl
