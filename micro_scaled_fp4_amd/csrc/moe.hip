// Expert routing for the grouped FP4 GEMM: scores, top-k and their gradient
// (k_route, k_route_grad), the stable sort of token slots by expert
// (k_count, k_place), tokens quantized into sorted order (k_gather_quant), and
// the weighted sum of expert outputs with its gradients (k_combine,
// k_combine_grad).
//
// The "NVIDIA NVFP4 与 Micro-Scaling" article (section 6.1) names MoE expert
// weights as NVFP4's main target and gives no routing; the formulas are those
// stated in include/fp4.h.
#include "epilogue.h"
#include "fp4_device.h"
#include "fp4_internal.h"
#include "grid.h"
#include "scale_bytes.h"

using namespace fp4dev;

namespace {

// ------------------------------------------------------ lane reductions --
// Rotation by R inside each row of 16 lanes (DPP row_ror).
template <int R>
__device__ __forceinline__ uint32_t ror16(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + R, 0xf, 0xf, false);
}
template <int R>
__device__ __forceinline__ float ror16f(float v) {
  return __uint_as_float(ror16<R>(__float_as_uint(v)));
}
// Reductions over the L lanes (16 or 64) of a token, result in every lane; the
// pairing is fixed, so sums do not depend on anything but their inputs.
template <int L>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
  v = umax(v, ror16<8>(v));
  v = umax(v, ror16<4>(v));
  v = umax(v, ror16<2>(v));
  v = umax(v, ror16<1>(v));
  if (L == 64) {
    v = umax(v, (uint32_t)__shfl_xor((int)v, 16, 64));
    v = umax(v, (uint32_t)__shfl_xor((int)v, 32, 64));
  }
  return v;
}
template <int L>
__device__ __forceinline__ float lanes_maxf(float v) {
  v = fmaxf(v, ror16f<8>(v));
  v = fmaxf(v, ror16f<4>(v));
  v = fmaxf(v, ror16f<2>(v));
  v = fmaxf(v, ror16f<1>(v));
  if (L == 64) {
    v = fmaxf(v, __shfl_xor(v, 16, 64));
    v = fmaxf(v, __shfl_xor(v, 32, 64));
  }
  return v;
}
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
  v += ror16f<8>(v);
  v += ror16f<4>(v);
  v += ror16f<2>(v);
  v += ror16f<1>(v);
  if (L == 64) {
    v += __shfl_xor(v, 16, 64);
    v += __shfl_xor(v, 32, 64);
  }
  return v;
}

// e^x, x <= 88, to about 2 ulp: the product x log2 e in two floats, its tail
// applied to the first order after v_exp_f32.  Below e^-104 (-inf included) 0.
__device__ __forceinline__ float exp_accurate(float x) {
  constexpr float kL = 0x1.715476p+0f, kLlo = 0x1.4ae0c0p-26f;
  x = fmaxf(x, -110.0f);
  const float t = x * kL;
  const float r = fmaf(x, kLlo, fmaf(x, kL, -t));
  const float e = __builtin_amdgcn_exp2f(t);
  return fmaf(e * r, 0x1.62e430p-1f, e);
}
// Sigmoid as a selection value (v_rcp_f32: 1 ulp).  Values below 2^-126, float32's
// smallest normal number, tie: from x = -88 down they are the same, at most e^-88.
__device__ __forceinline__ float sigmoid_value(float x) {
  return __builtin_amdgcn_rcpf(1.0f + exp_accurate(fminf(-x, 88.0f)));
}
// sigmoid(x) e^-c (c = 0 where x > 0) and, in rest, 1 - sigmoid(x), which loses no
// digits next to 1.  A common c <= 0 near the largest x of a token keeps scores that
// are all too small for float32 apart.
__device__ __forceinline__ float sigmoid_over(float x, float c, float& rest) {
  const float e = exp_accurate(-fabsf(x)), r = __builtin_amdgcn_rcpf(1.0f + e);
  rest = x > 0.0f ? e * r : r;
  if (x > 0.0f) return r;
  return (c < 0.0f ? exp_accurate(x - c) : e) * r;
}

// Float -> integer that orders like the float (-0 equal to +0).  Masked experts
// have -inf's key, kKeyNone, which every finite value's is above; 0, below it, is
// kept for experts that are taken.
constexpr uint32_t kKeyNone = 0x007fffffu;
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

constexpr float kNegInf = -__builtin_inff();
constexpr float kMaxFloat = 0x1.fffffep+127f;

// A logit as the scores read it: NaN masks the expert like -inf, +inf counts as
// the largest finite value.
__device__ __forceinline__ float clean_logit(float l) {
  return l >= kNegInf ? fminf(l, kMaxFloat) : kNegInf;
}

template <bool BF16>
__device__ __forceinline__ float load_logit(const void* logits, int64_t i) {
  return clean_logit(load1(logits, i, BF16));
}

// A lane's EPL consecutive logits e0 .. e0 + EPL - 1 of a row of E (-inf past
// E).  vec: E is a multiple of EPL and rows are aligned for whole-lane loads.
template <bool BF16, int EPL>
__device__ __forceinline__ void load_logits(const void* logits, int64_t row, int E, int e0, bool vec,
                                            float (&l)[EPL]) {
  const int64_t i = row * E + e0;
  if (EPL >= 4 && vec) {
    if (e0 < E) {
      if constexpr (EPL >= 8 && BF16) {
        const u32x4* p = reinterpret_cast<const u32x4*>(reinterpret_cast<const uint16_t*>(logits) + i);
#pragma unroll
        for (int k = 0; k < EPL / 8; ++k) {
          const u32x4 v = p[k];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            l[8 * k + 2 * q] = bf16_lo(v[q]);
            l[8 * k + 2 * q + 1] = bf16_hi(v[q]);
          }
        }
      } else if constexpr (EPL >= 4) {
#pragma unroll
        for (int k = 0; k < EPL / 4; ++k) {
          const f32x4 v = load4(logits, i + 4 * k, BF16);
          l[4 * k] = v.x; l[4 * k + 1] = v.y; l[4 * k + 2] = v.z; l[4 * k + 3] = v.w;
        }
      }
#pragma unroll
      for (int j = 0; j < EPL; ++j) l[j] = clean_logit(l[j]);
    } else {
#pragma unroll
      for (int j = 0; j < EPL; ++j) l[j] = kNegInf;
    }
  } else {
#pragma unroll
    for (int j = 0; j < EPL; ++j) l[j] = e0 + j < E ? load_logit<BF16>(logits, i + j) : kNegInf;
  }
}

// softmax statistics of a token: its largest logit (0 when all are masked) and
// the sum of e^(l - max)
template <int EPL, int L>
__device__ __forceinline__ void softmax_stats(const float (&l)[EPL], float& top, float& total) {
  float m = l[0];
#pragma unroll
  for (int j = 1; j < EPL; ++j) m = fmaxf(m, l[j]);
  m = lanes_maxf<L>(m);
  top = m > kNegInf ? m : 0.0f;
  float s = 0.0f;
#pragma unroll
  for (int j = 0; j < EPL; ++j) s += l[j] > kNegInf ? exp_accurate(l[j] - top) : 0.0f;
  total = lanes_sum<L>(s);
}

// What a token's selected logits li (-inf: none) are taken relative to when their scores
// are renormalized: only the ratios matter then, and all of the scores can be too
// small for float32 (softmax scores that a bias selects, sigmoid scores of logits far
// below 0).  Sigmoid scores are 0 from about e^-700 down, so that logits of a type's
// lowest value mask an expert.
template <int L>
__device__ __forceinline__ float shared_shift(float li, bool sigmoid) {
  const float m = lanes_maxf<L>(li);
  return sigmoid ? fminf(fmaxf(m, -700.0f), 0.0f) : m > kNegInf ? m : 0.0f;
}

constexpr int kRouteThreads = 256;
constexpr int kMaxGroups = 64;       // FP4_MOE_MAX_GROUPS
constexpr int kMaxTopK = 16;         // FP4_MOE_MAX_TOPK: a token's slots fit its 16 lanes

struct RouteArgs {
  const void* logits;
  const float* bias;
  int64_t T;
  int E, top_k, sigmoid, groups, top_groups, group_top, renorm, vec;
  int bias_vec, lane_groups;   // lanes per group, 0: groups of no whole power of two of lanes
  float scale;
  int32_t* ids;
  float* weights;
};

// Bias of a lane's EPL experts from e0 on (0 without one and past E).
template <int EPL>
__device__ __forceinline__ void load_bias_row(const float* bias, int E, int e0, bool vec, float (&b)[EPL]) {
  if (EPL % 4 == 0 && vec && bias != nullptr && e0 < E) {
    if constexpr (EPL % 4 == 0) {
#pragma unroll
      for (int k = 0; k < EPL / 4; ++k) {
        const f32x4 v = load4(bias, e0 + 4 * k, false);
        b[4 * k] = v.x; b[4 * k + 1] = v.y; b[4 * k + 2] = v.z; b[4 * k + 3] = v.w;
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < EPL; ++j) b[j] = bias != nullptr && e0 + j < E ? bias[e0 + j] : 0.0f;
  }
}

// (m1, m2), the two largest of a set, joined with those of another (p1 >= p2)
__device__ __forceinline__ void top_two(float& m1, float& m2, float p1, float p2) {
  m2 = fmaxf(fminf(m1, p1), fmaxf(m2, p2));
  m1 = fmaxf(m1, p1);
}
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), CTRL, 0xf, 0xf, false));
}
__device__ __forceinline__ float quad_swap1(float v) { return dpp<0xb1>(v); }     // quad_perm [1, 0, 3, 2]
__device__ __forceinline__ float quad_swap2(float v) { return dpp<0x4e>(v); }     // quad_perm [2, 3, 0, 1]
__device__ __forceinline__ float half_mirror(float v) { return dpp<0x141>(v); }   // lane 7 - i of each 8
__device__ __forceinline__ float row_mirror(float v) { return dpp<0x140>(v); }    // lane 15 - i of each 16

// f(k of another lane of the row of 16, that lane) for the lanes STEP, 2 STEP, ...
// away.  Row rotation by R hands lane i the value of lane (i - R) mod 16.
template <int R, int STEP, typename F>
__device__ __forceinline__ void rotations(uint32_t k, int ln, F&& f) {
  if constexpr (R < 16) {
    f(ror16<R>(k), (ln - R) & 15);
    rotations<R + STEP, STEP>(k, ln, f);
  }
}

// ------------------------------------------------------------------ route --
// A token per L lanes (16, so that a wave routes 4 tokens and reductions stay
// in DPP rows; 64 from 513 experts), EPL consecutive experts per lane in
// registers: logits are read once.  Top-k by k rounds of arg-max on
// order-preserving integer keys: a row maximum, a ballot for the lowest lane
// that holds it, and that lane's lowest expert with it -- ties go to the lowest
// index, and selected or masked experts have key 0.
// Bound: vector instructions, most of them in the rounds, where the lane that loses
// its largest key looks through the others.
// 32768 x 256 float32, sigmoid, bias, 4 of 8 groups, top 8: 22.4 us, 1.6 TB/s;
// reading the logits by way of LDS, contiguous over the lanes, took 29.  1 x 64: 3 us.
template <bool BF16, int EPL, int L>
__global__ void __launch_bounds__(kRouteThreads) k_route(RouteArgs a) {
  constexpr int kTokens = kRouteThreads / L;
  __shared__ int ids_s[kTokens][kMaxTopK];
  __shared__ float gs_s[kTokens][kMaxGroups];
  extern __shared__ float v_s[];   // [kTokens][E + 1] selection values (groups only)
  const int tl = threadIdx.x / L, ln = threadIdx.x % L;
  const int64_t t = (int64_t)workgroup() * kTokens + tl;
  const int64_t row = min(t, a.T - 1);   // lanes past the last token repeat it and store nothing
  const int E = a.E, e0 = ln * EPL;
  float l[EPL];
  load_logits<BF16, EPL>(a.logits, row, E, e0, a.vec, l);

  const bool two = a.groups > 1 && a.group_top == 2;
  const bool by_score = a.bias != nullptr || two;
  float top = 0.0f, total = 0.0f;
  if (!a.sigmoid && (by_score || !a.renorm)) softmax_stats<EPL, L>(l, top, total);
  uint32_t key[EPL];
  if (by_score) {
    float b[EPL];
    load_bias_row<EPL>(a.bias, E, e0, a.bias_vec, b);
    const float inv = total > 0.0f ? 1.0f / total : 0.0f;   // one division a token, then 1 ulp
    // the selection values take the logits' place (NaN: masked, like -inf)
    auto select_by = [&](auto score) {
#pragma unroll
      for (int j = 0; j < EPL; ++j) {
        const float v = score(l[j]) + b[j];
        l[j] = l[j] > kNegInf && v > kNegInf ? v : kNegInf;
      }
    };
    if (a.sigmoid)
      select_by([](float x) { return sigmoid_value(x); });
    else
      select_by([&](float x) { return exp_accurate(x - top) * inv; });
  }
#pragma unroll
  for (int j = 0; j < EPL; ++j) key[j] = order_key(l[j]);

  if (a.groups > 1 && a.lane_groups > 0) {
    // a group is lane_groups (1, 2, 4, 8 or 16) whole lanes: its two largest values
    // in registers, then over the lanes, pairs first
    float m1 = kNegInf, m2 = kNegInf;
#pragma unroll
    for (int j = 0; j < EPL; ++j) top_two(m1, m2, l[j], kNegInf);
    if (a.lane_groups > 1) top_two(m1, m2, quad_swap1(m1), quad_swap1(m2));
    if (a.lane_groups > 2) top_two(m1, m2, quad_swap2(m1), quad_swap2(m2));
    if (a.lane_groups > 4) top_two(m1, m2, half_mirror(m1), half_mirror(m2));
    if (a.lane_groups > 8) top_two(m1, m2, row_mirror(m1), row_mirror(m2));
    const float mine_s = a.group_top == 2 && m2 > kNegInf ? m1 + m2 : m1;
    // a group stays when fewer than top_groups are better (equal scores: the lower
    // index is); the scores of the other groups pass by
    const uint32_t mine_k = order_key(mine_s);
    int rank = 0;
    auto pass = [&](uint32_t k, int from) { rank += k > mine_k || (k == mine_k && from < (ln & -a.lane_groups)); };
    switch (a.lane_groups) {
      case 1: rotations<1, 1>(mine_k, ln, pass); break;
      case 2: rotations<2, 2>(mine_k, ln, pass); break;
      case 4: rotations<4, 4>(mine_k, ln, pass); break;
      case 8: rotations<8, 8>(mine_k, ln, pass); break;
      default: break;                  // one group
    }
    if (rank >= a.top_groups) {
#pragma unroll
      for (int j = 0; j < EPL; ++j) key[j] = 0u;
    }
  } else if (a.groups > 1) {
    float* vs = v_s + tl * (E + 1);
    const int size = E / a.groups;
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (e0 + j < E) vs[e0 + j] = l[j];
    wave_lds_order();
    for (int g = ln; g < a.groups; g += L) {
      float m1 = kNegInf, m2 = kNegInf;
      int at = g % size;               // lanes start at different members: fewer bank conflicts
      for (int i = 0; i < size; ++i) {
        const float v = vs[g * size + at];
        at = at + 1 == size ? 0 : at + 1;
        m2 = fmaxf(m2, fminf(m1, v));
        m1 = fmaxf(m1, v);
      }
      gs_s[tl][g] = a.group_top == 2 && m2 > kNegInf ? m1 + m2 : m1;
    }
    wave_lds_order();
    // (kept as above)
    uint32_t keep = 0;                 // bit i: group ln + i L
    for (int g = ln, i = 0; g < a.groups; g += L, ++i) {
      const float mine = gs_s[tl][g];
      int rank = 0;
      for (int o = 0; o < a.groups; ++o) {
        const float s = gs_s[tl][o];
        rank += s > mine || (s == mine && o < g);
      }
      if (rank < a.top_groups && mine > kNegInf) keep |= 1u << i;
    }
    wave_lds_order();                  // every lane has read the scores
    for (int g = ln, i = 0; g < a.groups; g += L, ++i) gs_s[tl][g] = (keep >> i) & 1 ? 1.0f : 0.0f;
    wave_lds_order();
    int g = e0 / size, in = e0 - g * size;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      if (e0 + j >= E || gs_s[tl][min(g, a.groups - 1)] == 0.0f) key[j] = 0u;
      if (++in == size) {
        in = 0;
        ++g;
      }
    }
  }

  uint32_t mine = 0;
#pragma unroll
  for (int j = 0; j < EPL; ++j) mine = umax(mine, key[j]);
  for (int r = 0; r < a.top_k; ++r) {
    const uint32_t best = lanes_max<L>(mine);
    const uint64_t hit = __ballot(mine == best) >> (L == 64 ? 0 : (threadIdx.x & 48));
    const int src = __ffsll((unsigned long long)(L == 64 ? hit : hit & 0xffffu)) - 1;
    if (ln == src) {
      int e = -1;
      if (best > kKeyNone) {
        int at = 0;
        bool taken = false;            // (wave masks: the logic on them is scalar work)
        mine = 0;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
          const bool hit_j = key[j] == best, pick = hit_j && !taken;
          taken |= hit_j;
          key[j] = pick ? 0u : key[j];
          at = pick ? j : at;
          mine = umax(mine, key[j]);
        }
        e = e0 + at;
      }
      ids_s[tl][r] = e;
    }
  }
  wave_lds_order();

  // lane r: slot r's score and weight
  const int id = ln < a.top_k ? ids_s[tl][ln] : -1;
  const float li = id >= 0 ? load_logit<BF16>(a.logits, row * E + id) : kNegInf;
  if (a.renorm) top = shared_shift<L>(li, a.sigmoid);
  float s = 0.0f, rest;
  if (id >= 0) s = a.sigmoid ? sigmoid_over(li, top, rest) : exp_accurate(li - top);
  if (a.renorm) {
    const float sum = lanes_sum<L>(s);
    s = sum > 0.0f ? s / sum : 0.0f;
  } else if (!a.sigmoid) {
    s = total > 0.0f ? s / total : 0.0f;
  }
  if (t < a.T && ln < a.top_k) {
    a.ids[t * a.top_k + ln] = id;
    a.weights[t * a.top_k + ln] = s * a.scale;
  }
}

struct RouteGradArgs {
  const float* dw;
  const void* logits;
  const int32_t* ids;
  int64_t T;
  int E, top_k, sigmoid, renorm, lvec, vec;   // lvec: whole-lane loads; vec: 16-byte stores
  float scale;
  void* dl;
  int dl_bf16;
};

// Gradient of the weights with respect to the logits (ids fixed).  With c the
// scale, p the scores and q = w / c:
//   softmax, renormalized   dl_i = q_i (c dw_i - sum c dw q)      selected i, else 0
//   softmax                 dl_i = p_i (c dw_i [i selected] - sum c dw p)
//   sigmoid, renormalized   dl_i = q_i (c dw_i - sum c dw q) (1 - s_i)
//   sigmoid                 dl_i = c dw_i s_i (1 - s_i)
// Layout as k_route; the row is put together in LDS and written whole, contiguous
// over the lanes (whole-lane stores, 64 bytes apart: 19.5 us against 7.6 at
// 32768 x 256 float32).  HBM bound: 50 MB there, 6.6 TB/s; rows of the sigmoid form
// and of renormalized softmax need no logits but the selected ones.
template <bool BF16, int EPL, int L>
__global__ void __launch_bounds__(kRouteThreads) k_route_grad(RouteGradArgs a) {
  constexpr int kTokens = kRouteThreads / L;
  extern __shared__ float v_s[];   // [kTokens][L * EPL]
  const int tl = threadIdx.x / L, ln = threadIdx.x % L;
  const int64_t t = (int64_t)workgroup() * kTokens + tl;
  const int64_t row = min(t, a.T - 1);
  const int E = a.E, e0 = ln * EPL;
  float* vs = v_s + tl * (L * EPL);
  float top = 0.0f, total = 1.0f;
  const bool dense = !a.sigmoid && !a.renorm;
  int id = ln < a.top_k ? a.ids[row * a.top_k + ln] : -1;
  if (id >= E) id = -1;
  const float dw = id >= 0 ? a.dw[row * a.top_k + ln] * a.scale : 0.0f;
  const float li = id >= 0 ? load_logit<BF16>(a.logits, row * E + id) : kNegInf;
  float l[EPL];
  if (dense) {
    load_logits<BF16, EPL>(a.logits, row, E, e0, a.lvec, l);
    softmax_stats<EPL, L>(l, top, total);
  } else if (a.renorm) {
    top = shared_shift<L>(li, a.sigmoid);
  }
  float s = 0.0f, rest = 0.0f;             // (rest: 1 - s)
  if (li > kNegInf) s = a.sigmoid ? sigmoid_over(li, top, rest) : exp_accurate(li - top);
  float g, mean = 0.0f;
  if (a.renorm) {
    const float sum = lanes_sum<L>(s);
    const float q = sum > 0.0f ? s / sum : 0.0f;
    mean = lanes_sum<L>(dw * q);
    g = q * (dw - mean);
    if (a.sigmoid) g *= rest;
  } else if (a.sigmoid) {
    g = dw * s * rest;
  } else {
    s = total > 0.0f ? s / total : 0.0f;
    mean = lanes_sum<L>(dw * s);
    g = dw * s;
  }
  if (dense) {
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      vs[e0 + j] = l[j] > kNegInf ? -(exp_accurate(l[j] - top) / total) * mean : 0.0f;
  } else {
#pragma unroll
    for (int j = 0; j < EPL; ++j) vs[j * L + ln] = 0.0f;
  }
  wave_lds_order();
  if (id >= 0) vs[id] += g;
  wave_lds_order();
  if (t >= a.T) return;
  // the row in 16-byte pieces, contiguous over the lanes
  if (a.vec && a.dl_bf16) {
    for (int e = 8 * ln; e < E; e += 8 * L) {
      float o[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) o[k] = vs[e + k];
      store_vec<8>(a.dl, t * E + e, true, o);
    }
  } else if (a.vec) {
    for (int e = 4 * ln; e < E; e += 4 * L)
      *reinterpret_cast<f32x4*>(reinterpret_cast<float*>(a.dl) + t * E + e) =
          *reinterpret_cast<const f32x4*>(vs + e);
  } else {
    for (int e = ln; e < E; e += L) store1(a.dl, t * E + e, a.dl_bf16, vs[e]);
  }
}

// ------------------------------------------------------------------- sort --
// Stable counting sort of the n = T top_k slots by expert id.  Workgroup c owns
// the `chunk` slots from c chunk on: k_count writes its histogram, k_place sums
// the histograms before it (and over all, for the offsets) and ranks its own
// slots, kSortThreads at a time: inside a wave by matching ids over their bits
// (a ballot per bit), across waves by per-wave counts in LDS.  One chunk needs
// no histograms from elsewhere: k_place counts for itself.  Ids outside [0, E)
// have no row.  Up to kOneChunk slots go in one chunk (a launch less); more in
// chunks of kSortThreads slots, or of as many as make kMaxChunks chunks, since
// every workgroup reads all histograms (32768 slots: k_place 10.6 us in chunks of
// 4096, 5.1 in chunks of 1024).
constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kOneChunk = 4096;
constexpr int kMaxChunks = 512;
constexpr int kMaxExperts = 1024;    // FP4_MOE_MAX_EXPERTS

inline int64_t sort_chunk(int64_t n) {
  if (n <= kOneChunk) return kOneChunk;
  const int64_t per = (int64_t)kSortThreads * kMaxChunks;
  return (n + per - 1) / per * kSortThreads;
}

__device__ __forceinline__ void count_chunk(const int32_t* __restrict__ ids, int64_t n, int64_t c, int chunk,
                                            int E, int* hist) {
  for (int e = threadIdx.x; e < E; e += blockDim.x) hist[e] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < chunk; i += blockDim.x) {
    const int64_t s = c * chunk + i;
    const int id = s < n ? ids[s] : -1;
    if (id >= 0 && id < E) atomicAdd(&hist[id], 1);   // LDS; a sum of ones has no order
  }
  __syncthreads();
}

// max|x| of the elements of partial `p` of `np`, as a bit pattern
template <bool BF16>
__device__ __forceinline__ uint32_t amax_part(const void* __restrict__ x, int64_t n, int64_t p, int64_t np,
                                              bool vec) {
  uint32_t m = 0;
  constexpr int kPer = BF16 ? 8 : 4;
  if (vec) {
    const u32x4* xv = reinterpret_cast<const u32x4*>(x);
    const int64_t nv = n / kPer, step = np * blockDim.x;
    for (int64_t i = p * blockDim.x + threadIdx.x; i < nv; i += 8 * step) {
      u32x4 v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = i + u * step < nv ? xv[i + u * step] : u32x4{0, 0, 0, 0};
#pragma unroll
      for (int u = 0; u < 8; ++u)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t w = v[u][q];
          if (BF16) {
            const uint32_t b = w & 0x7fff7fffu;
            m = umax(m, umax(b << 16, b & 0xffff0000u));
          } else {
            m = umax(m, w & 0x7fffffffu);
          }
        }
    }
  } else {
    for (int64_t i = p * blockDim.x + threadIdx.x; i < n; i += np * blockDim.x)
      m = umax(m, __float_as_uint(load1(x, i, BF16)) & 0x7fffffffu);
  }
  return m;
}

struct PlaceArgs {
  const int32_t* ids;
  int64_t n;
  int E, chunk, chunks;
  const int* counts;       // [chunks][E] (chunks > 1)
  int32_t* offsets;        // [E + 1]
  int32_t* slot_rows;      // [n]
  int32_t* row_slots;      // [n]
};

// Chunk c of the placement; every thread of the workgroup (kSortThreads) takes
// part.  write: the index arrays are written (else another workgroup does); rows:
// the rows of the chunk's first kSortThreads slots in LDS, or NULL.  Returns the
// number of rows.
__device__ __forceinline__ int place_chunk(const PlaceArgs& a, int64_t c, bool write = true,
                                           int* rows = nullptr) {
  __shared__ int start[kMaxExperts];               // next row of each expert
  __shared__ int wsum[kSortWaves];
  __shared__ uint16_t wave_n[kSortWaves][kMaxExperts];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int E = a.E;
  int mine = 0, before = 0;                        // expert tid: all rows, and those of earlier chunks
  if (a.chunks > 1) {
    if (tid < E) {
#pragma unroll 8
      for (int k = 0; k < a.chunks; ++k) {
        const int v = a.counts[(int64_t)k * E + tid];
        before += k < c ? v : 0;
        mine += v;
      }
    }
  } else {
    count_chunk(a.ids, a.n, 0, a.chunk, E, start);
    if (tid < E) mine = start[tid];
  }
  // exclusive scan of the experts' rows
  int inc = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(inc, d, 64);
    if (lane >= d) inc += v;
  }
  if (lane == 63) wsum[wave] = inc;
  __syncthreads();
  int base = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kSortWaves; ++w) {
    if (w < wave) base += wsum[w];
    all += wsum[w];
  }
  if (tid < E) start[tid] = base + inc - mine + before;
  if (c == 0 && write) {
    if (tid < E) a.offsets[tid] = base + inc - mine;
    if (tid == 0) a.offsets[E] = all;
    for (int64_t r = (int64_t)all + tid; r < a.n; r += kSortThreads) a.row_slots[r] = -1;
  }
  const int bits = 32 - __clz(E);                  // ids 0 .. E (E: no expert)
  for (int i0 = 0; i0 < a.chunk && c * a.chunk + i0 < a.n; i0 += kSortThreads) {
    for (int e = tid; e < kSortWaves * kMaxExperts / 2; e += kSortThreads)
      reinterpret_cast<uint32_t*>(&wave_n[0][0])[e] = 0;
    const int64_t s = c * a.chunk + i0 + tid;
    int id = s < a.n ? a.ids[s] : -1;
    const bool live = id >= 0 && id < E;
    if (!live) id = E;
    uint64_t same = ~0ull;
    for (int b = 0; b < bits; ++b) {
      const uint64_t set = __ballot((id >> b) & 1);
      same &= (id >> b) & 1 ? set : ~set;
    }
    const int rank = __popcll(same & ((1ull << lane) - 1));
    __syncthreads();                               // wave_n is clear, start is ready
    if (live && rank == 0) wave_n[wave][id] = (uint16_t)__popcll(same);
    __syncthreads();
    int r = -1;
    if (live) {
      r = start[id] + rank;
      for (int w = 0; w < wave; ++w) r += wave_n[w][id];
      if (write) a.row_slots[r] = (int32_t)s;
    }
    if (write && s < a.n) a.slot_rows[s] = r;
    if (rows != nullptr && i0 == 0) rows[tid] = r;
    __syncthreads();                               // every rank has read start
    if (tid < E) {
      int sum = 0;
#pragma unroll
      for (int w = 0; w < kSortWaves; ++w) sum += wave_n[w][tid];
      start[tid] += sum;
    }
    __syncthreads();                               // wave_n is read before it is cleared
  }
  return all;
}

// First launch of a dispatch: workgroups [0, sort_wgs) count their chunk (or,
// with one chunk, place it); the others reduce a part of x to its max|x|.
template <bool BF16>
__global__ void __launch_bounds__(kSortThreads)
    k_count(PlaceArgs a, int* __restrict__ counts, int sort_wgs, const void* __restrict__ x, int64_t nx,
            bool vec, uint32_t* __restrict__ partials, int npart) {
  __shared__ int hist[kMaxExperts];
  if ((int)blockIdx.x < sort_wgs) {
    if (a.chunks == 1) {
      place_chunk(a, 0);
    } else {
      count_chunk(a.ids, a.n, blockIdx.x, a.chunk, a.E, hist);
      for (int e = threadIdx.x; e < a.E; e += kSortThreads) counts[(int64_t)blockIdx.x * a.E + e] = hist[e];
    }
    return;
  }
  const int p = blockIdx.x - sort_wgs;
  uint32_t m = wave_max_u32(amax_part<BF16>(x, nx, p, npart, vec));
  if ((threadIdx.x & 63) == 0) hist[threadIdx.x >> 6] = (int)m;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < kSortWaves; ++i) m = umax(m, (uint32_t)hist[i]);
    partials[p] = m;
  }
}

__global__ void __launch_bounds__(kSortThreads) k_place(PlaceArgs a) { place_chunk(a, blockIdx.x); }

__global__ void k_empty_dispatch(int32_t* offsets, int E, float* amax_out, float* scale_out) {
  for (int e = threadIdx.x; e <= E; e += blockDim.x) offsets[e] = 0;
  if (threadIdx.x == 0) {
    if (amax_out != nullptr) *amax_out = 0.0f;
    if (scale_out != nullptr) *scale_out = 1.0f;
  }
}

// ------------------------------------------------------- gather + quantize --
struct GatherArgs {
  const void* x;
  int64_t T;
  int H, top_k, E;
  const int32_t* slot_rows;
  const int32_t* offsets;
  uint8_t* q;
  uint8_t* scales;
  const float* amax_in;          // NVFP4: the given amax, or NULL with the partials below
  const uint32_t* partials;
  int npart;
  float* amax_out;
  float* scale_out;
  int vec;                       // x is 16-byte aligned, H a multiple of 32 always
};

constexpr int kGatherThreads = 256;

// Quantizes block blk (16 values, MXFP4 32) of token t exactly as nvfp4_quantize /
// mxfp4_quantize do and writes it to each of the token's rows (row_of(j)), so a
// token is read and encoded once however many experts take it.
template <bool MX, bool BF16, typename F>
__device__ __forceinline__ void quantize_to_rows(const GatherArgs& a, int64_t t, int blk, float s_global,
                                                 F&& row_of) {
  constexpr int BS = MX ? 32 : 16;
  const int nb = a.H / BS;
  float v[BS];
  const int64_t src = t * a.H + (int64_t)blk * BS;
  if (a.vec) {
    if (BF16) {
      const u32x4* p = reinterpret_cast<const u32x4*>(reinterpret_cast<const uint16_t*>(a.x) + src);
#pragma unroll
      for (int k = 0; k < BS / 8; ++k) {
        const u32x4 w = p[k];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          v[8 * k + 2 * q] = bf16_lo(w[q]);
          v[8 * k + 2 * q + 1] = bf16_hi(w[q]);
        }
      }
    } else {
      const f32x4* p = reinterpret_cast<const f32x4*>(reinterpret_cast<const float*>(a.x) + src);
#pragma unroll
      for (int k = 0; k < BS / 4; ++k) {
        const f32x4 w = p[k];
        v[4 * k] = w.x; v[4 * k + 1] = w.y; v[4 * k + 2] = w.z; v[4 * k + 3] = w.w;
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < BS; ++k) v[k] = load1(a.x, src + k, BF16);
  }
  uint32_t am = 0;
#pragma unroll
  for (int k = 0; k < BS; ++k) am = umax(am, __float_as_uint(v[k]) & 0x7fffffffu);
  uint32_t sc;
  float r;
  if (MX) {
    sc = e8m0_code(am);
    r = e8m0_inv(sc);
  } else {
    nv_block_scale(__uint_as_float(am), s_global, sc, r);
  }
  uint32_t c[BS / 8];
#pragma unroll
  for (int k = 0; k < BS / 8; ++k) {
#pragma unroll
    for (int q = 0; q < 8; ++q) v[8 * k + q] *= r;
    c[k] = e2m1_pack8(v + 8 * k);
  }
  for (int j = 0; j < a.top_k; ++j) {
    const int row = row_of(j);
    if (row < 0) continue;
    uint8_t* dst = a.q + (int64_t)row * (a.H / 2) + blk * (BS / 2);
    if constexpr (MX)
      *reinterpret_cast<u32x4*>(dst) = u32x4{c[0], c[1], c[2], c[3]};
    else
      *reinterpret_cast<u32x2*>(dst) = u32x2{c[0], c[1]};
    a.scales[(int64_t)row * nb + blk] = (uint8_t)sc;
  }
}

// Codes and scales of the rows of dropped slots (from `first` on): zeros.
template <bool MX>
__device__ __forceinline__ void zero_rows(const GatherArgs& a, int64_t first) {
  constexpr int BS = MX ? 32 : 16;
  const int nb = a.H / BS;
  const int64_t end = a.T * a.top_k * nb, step = (int64_t)gridDim.x * blockDim.x;
  for (int64_t i = first * nb + (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < end; i += step) {
    uint8_t* dst = a.q + i * (BS / 2);
    if constexpr (MX)
      *reinterpret_cast<u32x4*>(dst) = u32x4{0, 0, 0, 0};
    else
      *reinterpret_cast<u32x2*>(dst) = u32x2{0, 0};
    a.scales[i] = 0;
  }
}

// The tensor scale of max|x| = G, written once.
__device__ __forceinline__ float tensor_scale(const GatherArgs& a, float G) {
  const float s = nv_global_scale(G);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    if (a.amax_out != nullptr) *a.amax_out = G;
    *a.scale_out = s;
  }
  return s;
}

// A thread per block.  HBM bound: 4096 x 7168 bf16 to 8 rows each, 191 MB in 32 us.
template <bool MX, bool BF16>
__global__ void __launch_bounds__(kGatherThreads) k_gather_quant(GatherArgs a) {
  __shared__ uint32_t red[kGatherThreads / 64];
  const int nb = a.H / (MX ? 32 : 16);
  float s_global = 1.0f;
  if (!MX) {
    float G;
    if (a.amax_in != nullptr) {
      G = *a.amax_in;
    } else {
      uint32_t m = 0;
      for (int i = threadIdx.x; i < a.npart; i += kGatherThreads) m = umax(m, a.partials[i]);
      m = wave_max_u32(m);
      if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kGatherThreads / 64; ++i) m = umax(m, red[i]);
      G = __uint_as_float(m);
    }
    s_global = tensor_scale(a, G);
  }
  const int64_t n = a.T * nb, step = (int64_t)gridDim.x * kGatherThreads;
  for (int64_t i = (int64_t)blockIdx.x * kGatherThreads + threadIdx.x; i < n; i += step) {
    const int64_t t = i / nb;
    quantize_to_rows<MX, BF16>(a, t, (int)(i - t * nb), s_global,
                               [&](int j) { return a.slot_rows[t * a.top_k + j]; });
  }
  zero_rows<MX>(a, a.offsets[a.E]);
}

// A small dispatch in one launch: every workgroup sorts all slots (at most
// kSortThreads) and reduces all of x (at most kSmallX values) for itself, and
// workgroup 0 writes the index arrays.  Bound by latency, of x's loads and of a
// chain of barriers: 16 tokens x 7168 to 8 of 64 experts in 10.8 us, the call 18 us
// from the host (23 in the two launches of the general form).
constexpr int64_t kSmallX = (int64_t)1 << 17;
template <bool MX, bool BF16>
__global__ void __launch_bounds__(kSortThreads) k_dispatch_small(PlaceArgs p, GatherArgs a) {
  __shared__ int rows[kSortThreads];
  __shared__ uint32_t red[kSortWaves];
  const int nb = a.H / (MX ? 32 : 16);
  float s_global = 1.0f;
  if (!MX) {
    float G;
    if (a.amax_in != nullptr) {
      G = *a.amax_in;
    } else {
      uint32_t m = wave_max_u32(amax_part<BF16>(a.x, a.T * a.H, 0, 1, a.vec));
      if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kSortWaves; ++i) m = umax(m, red[i]);
      G = __uint_as_float(m);
    }
    s_global = tensor_scale(a, G);
  }
  const int all = place_chunk(p, 0, blockIdx.x == 0, rows);   // (ends with a barrier)
  const int n = (int)a.T * nb;
  for (int i = blockIdx.x * kSortThreads + threadIdx.x; i < n; i += gridDim.x * kSortThreads) {
    const int t = i / nb;
    quantize_to_rows<MX, BF16>(a, t, i - t * nb, s_global, [&](int j) { return rows[t * a.top_k + j]; });
  }
  zero_rows<MX>(a, all);
}

// ---------------------------------------------------------------- combine --
struct CombineArgs {
  const void* rows;
  int64_t M;
  const float* weights;
  const int32_t* slot_rows;
  int64_t T;
  int H, top_k, rows_bf16, res_bf16, y_bf16;
  const void* residual;
  void* y;
};

// V consecutive values as float32 (V 8: 16-byte loads; V 1: one element)
template <int V>
__device__ __forceinline__ void load_vals(const void* p, int64_t i, bool bf16, float (&v)[V]) {
  if constexpr (V == 8) {
    if (bf16) {
      const u32x4 w = *reinterpret_cast<const u32x4*>(reinterpret_cast<const uint16_t*>(p) + i);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        v[2 * q] = bf16_lo(w[q]);
        v[2 * q + 1] = bf16_hi(w[q]);
      }
    } else {
      const f32x4 a = load4(p, i, false), b = load4(p, i + 4, false);
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
  } else {
    v[0] = load1(p, i, bf16);
  }
}
template <int V>
__device__ __forceinline__ void store_vals(void* p, int64_t i, bool bf16, const float (&v)[V]) {
  if constexpr (V == 8)
    store_vec<8>(p, i, bf16, v);
  else
    store1(p, i, bf16, v[0]);
}

// the same past the caches, for what nothing reads soon
template <int V>
__device__ __forceinline__ void stream_vals(void* p, int64_t i, bool bf16, const float (&v)[V]) {
  if constexpr (V == 8) {
    if (bf16) {
      __builtin_nontemporal_store(u32x4{bf16_pack2(v[0], v[1]), bf16_pack2(v[2], v[3]), bf16_pack2(v[4], v[5]),
                                        bf16_pack2(v[6], v[7])},
                                  reinterpret_cast<u32x4*>(reinterpret_cast<uint16_t*>(p) + i));
    } else {
      f32x4* q = reinterpret_cast<f32x4*>(reinterpret_cast<float*>(p) + i);
      __builtin_nontemporal_store(f32x4{v[0], v[1], v[2], v[3]}, q);
      __builtin_nontemporal_store(f32x4{v[4], v[5], v[6], v[7]}, q + 1);
    }
  } else {
    store1(p, i, bf16, v[0]);
  }
}

constexpr int kCombineThreads = 256;
constexpr int kSlotBatch = 8;        // slots whose rows are in flight together

// One slot's row: a descriptor of its H values, empty for a dropped slot (loads
// through it read zeros, with no branch around them), and its weight, 0 then.
struct SlotRow {
  __amdgpu_buffer_rsrc_t rsrc;
  float w;
  int row;                           // -1: dropped
};
__device__ __forceinline__ SlotRow slot_row(const void* rows, bool bf16, int64_t M, int H,
                                            const int32_t* slot_rows, const float* weights, int64_t slot,
                                            bool exists) {
  int row = exists ? slot_rows[slot] : -1;
  if (row >= M) row = -1;
  const int bytes = H * (bf16 ? 2 : 4);
  const uint8_t* p = reinterpret_cast<const uint8_t*>(rows) + (int64_t)max(row, 0) * bytes;
  return {__builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p), 0, row >= 0 ? bytes : 0, kBufferWord3),
          row >= 0 ? weights[slot] : 0.0f, row};
}
// V values from column h on, as loaded (V 8: 16 or 32 bytes; V 1: one element)
template <int V>
struct RowRaw {
  u32x4 v[V == 8 ? 2 : 1];
};
constexpr int kLoadNT = 2;           // buffer load cache policy: nontemporal
template <int V>
__device__ __forceinline__ void load_row(RowRaw<V>& r, const SlotRow& s, int h, bool bf16) {
  if constexpr (V == 8) {
    r.v[0] = __builtin_amdgcn_raw_buffer_load_b128(s.rsrc, h * (bf16 ? 2 : 4), 0, kLoadNT);
    if (!bf16) r.v[1] = __builtin_amdgcn_raw_buffer_load_b128(s.rsrc, h * 4 + 16, 0, kLoadNT);
  } else {
    r.v[0].x = bf16 ? (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(s.rsrc, h * 2, 0, 0) << 16
                    : __builtin_amdgcn_raw_buffer_load_b32(s.rsrc, h * 4, 0, 0);
  }
}
template <int V>
__device__ __forceinline__ void row_values(float (&v)[V], const RowRaw<V>& r, bool bf16) {
  if constexpr (V == 8) {
    if (bf16) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        v[2 * q] = bf16_lo(r.v[0][q]);
        v[2 * q + 1] = bf16_hi(r.v[0][q]);
      }
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] = __uint_as_float(r.v[q >> 2][q & 3]);
    }
  } else {
    v[0] = __uint_as_float(r.v[0].x);
  }
}

// y[t] = sum over slots of weight * row (+ residual), float32 in slot order; a
// workgroup per piece of a token's columns, so the slots' rows and weights are
// uniform and the rows of kSlotBatch slots are in flight together.  HBM bound:
// 4096 tokens x 8 rows of 7168 bf16, 533 MB in 93 us, 5.7 TB/s (a slot's loads
// after the sum of the one before it: 128 us).
template <int V, bool ROWS_BF16>
__global__ void __launch_bounds__(kCombineThreads) k_combine(CombineArgs a, int pieces) {
  const uint32_t wg = workgroup();
  const int64_t t = wg / (uint32_t)pieces;
  const int h = ((int)(wg - t * pieces) * kCombineThreads + (int)threadIdx.x) * V;
  if (t >= a.T || h >= a.H) return;
  float acc[V], res[V];
#pragma unroll
  for (int q = 0; q < V; ++q) acc[q] = res[q] = 0.0f;
  if (a.residual != nullptr) load_vals<V>(a.residual, t * a.H + h, a.res_bf16, res);
  for (int j0 = 0; j0 < a.top_k; j0 += kSlotBatch) {
    float w[kSlotBatch];
    RowRaw<V> raw[kSlotBatch];
#pragma unroll
    for (int j = 0; j < kSlotBatch; ++j) {
      const SlotRow s = slot_row(a.rows, ROWS_BF16, a.M, a.H, a.slot_rows, a.weights,
                                 t * a.top_k + j0 + j, j0 + j < a.top_k);
      w[j] = s.w;
      load_row<V>(raw[j], s, h, ROWS_BF16);
    }
#pragma unroll
    for (int j = 0; j < kSlotBatch; ++j) {
      float v[V];
      row_values<V>(v, raw[j], ROWS_BF16);
#pragma unroll
      for (int q = 0; q < V; ++q) acc[q] = fmaf(w[j], v[q], acc[q]);
    }
  }
#pragma unroll
  for (int q = 0; q < V; ++q) acc[q] += res[q];
  store_vals<V>(a.y, t * a.H + h, a.y_bf16, acc);
}

struct CombineGradArgs {
  const void* dy;
  const void* rows;
  const float* weights;
  const int32_t* slot_rows;
  const int32_t* row_slots;
  int64_t T, M;
  int H, top_k, dy_bf16, rows_bf16, dr_bf16;
  void* d_rows;
  float* d_weights;
};

// d_rows[row] = weight * dy[t] and d_weight = <dy[t], row>: a workgroup per
// token reads dy once for all its slots; the dot products are summed per thread
// over its columns, then over lanes and waves in a fixed order.  Rows of no
// slot get zeros.  HBM bound: the same 4096 tokens, 1.0 GB in 216 us, 4.6 TB/s (the
// copy rate: as much is written as read).
template <int V, bool ROWS_BF16>
__global__ void __launch_bounds__(kCombineThreads) k_combine_grad(CombineGradArgs a) {
  __shared__ float red[kCombineThreads / 64][kMaxTopK];
  const int64_t t = workgroup();
  if (t >= a.T) return;
  const int k = a.top_k, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  float dot[kMaxTopK];
#pragma unroll
  for (int j = 0; j < kMaxTopK; ++j) dot[j] = 0.0f;
  for (int h = threadIdx.x * V; h < a.H; h += kCombineThreads * V) {
    float dy[V];
    load_vals<V>(a.dy, t * a.H + h, a.dy_bf16, dy);
#pragma unroll
    for (int j0 = 0; j0 < kMaxTopK; j0 += kSlotBatch) {
      if (j0 >= k) continue;
      SlotRow s[kSlotBatch];
      RowRaw<V> raw[kSlotBatch];
#pragma unroll
      for (int j = 0; j < kSlotBatch; ++j) {
        s[j] = slot_row(a.rows, ROWS_BF16, a.M, a.H, a.slot_rows, a.weights, t * k + j0 + j, j0 + j < k);
        load_row<V>(raw[j], s[j], h, ROWS_BF16);
      }
#pragma unroll
      for (int j = 0; j < kSlotBatch; ++j) {
        float v[V], d[V];
        row_values<V>(v, raw[j], ROWS_BF16);
#pragma unroll
        for (int q = 0; q < V; ++q) {
          dot[j0 + j] = fmaf(dy[q], v[q], dot[j0 + j]);
          d[q] = s[j].w * dy[q];
        }
        if (s[j].row >= 0) stream_vals<V>(a.d_rows, (int64_t)s[j].row * a.H + h, a.dr_bf16, d);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < kMaxTopK; ++j)
    if (j < k) {
      const float s = lanes_sum<64>(dot[j]);
      if (lane == 0) red[wave][j] = s;
    }
  __syncthreads();
  if ((int)threadIdx.x < k) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kCombineThreads / 64; ++w) s += red[w][threadIdx.x];
    // (a slot without a row: 0 also where dy times the zeros read for it is NaN)
    const int row = a.slot_rows[t * k + threadIdx.x];
    a.d_weights[t * k + threadIdx.x] = row >= 0 && row < a.M ? s : 0.0f;
  }
  // this workgroup's share of the rows: those of no slot
  const int64_t per = (a.M + a.T - 1) / a.T;
  for (int64_t r = t * per; r < min((t + 1) * per, a.M); ++r) {
    const int s = a.row_slots[r];
    if (s >= 0) continue;
    float z[V];
#pragma unroll
    for (int q = 0; q < V; ++q) z[q] = 0.0f;
    for (int h = threadIdx.x * V; h < a.H; h += kCombineThreads * V)
      store_vals<V>(a.d_rows, r * a.H + h, a.dr_bf16, z);
  }
}

bool ok16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace

namespace fp4impl {

// Lanes per token and experts per lane by E.
#define FP4_ROUTE_SIZES(CALL)                 \
  if (E <= 16) { CALL(1, 16); }               \
  else if (E <= 64) { CALL(4, 16); }          \
  else if (E <= 128) { CALL(8, 16); }         \
  else if (E <= 256) { CALL(16, 16); }        \
  else if (E <= 512) { CALL(32, 16); }        \
  else { CALL(16, 64); }

hipError_t launch_route(const RouteProblem& p, const float* bias, int groups, int top_groups,
                        int group_top, int32_t* ids, float* weights, hipStream_t stream) {
  const int E = (int)p.E;
  RouteArgs a{p.logits, bias, p.T, E, p.top_k, p.sigmoid, groups, top_groups, group_top, p.renorm, 0,
              0, 0, p.scale, ids, weights};
  const int size = E / groups;
#define FP4_CALL(EPL, L)                                                                              \
  a.vec = E % EPL == 0 && ok16(p.logits);                                                             \
  a.bias_vec = E % EPL == 0 && ok16(bias);                                                            \
  /* (16-lane tokens: rows of DPP; groups of whole lanes, a power of two of them) */                 \
  const int lg = L == 16 && size % EPL == 0 ? size / EPL : 0;                                         \
  a.lane_groups = lg > 0 && (lg & (lg - 1)) == 0 ? lg : 0;                                            \
  const int64_t grid = (p.T + kRouteThreads / L - 1) / (kRouteThreads / L);                           \
  const size_t lds = groups > 1 && a.lane_groups == 0 ? sizeof(float) * (kRouteThreads / L) * (E + 1) : 0;                  \
  if (p.bf16)                                                                                         \
    hipLaunchKernelGGL((k_route<true, EPL, L>), grid_of(grid), dim3(kRouteThreads), lds, stream, a);     \
  else                                                                                                \
    hipLaunchKernelGGL((k_route<false, EPL, L>), grid_of(grid), dim3(kRouteThreads), lds, stream, a)
  FP4_ROUTE_SIZES(FP4_CALL)
#undef FP4_CALL
  return hipGetLastError();
}

hipError_t launch_route_grad(const RouteProblem& p, const float* dw, const int32_t* ids, void* dl,
                             bool dl_bf16, hipStream_t stream) {
  const int E = (int)p.E;
  RouteGradArgs a{dw, p.logits, ids, p.T, E, p.top_k, p.sigmoid, p.renorm, 0, 0, p.scale, dl, dl_bf16};
#define FP4_CALL(EPL, L)                                                                              \
  a.lvec = E % EPL == 0 && ok16(p.logits);                                                            \
  a.vec = E % 8 == 0 && ok16(dl);                                                                     \
  const int64_t grid = (p.T + kRouteThreads / L - 1) / (kRouteThreads / L);                           \
  const size_t lds = sizeof(float) * kRouteThreads * EPL;                                             \
  if (p.bf16)                                                                                         \
    hipLaunchKernelGGL((k_route_grad<true, EPL, L>), grid_of(grid), dim3(kRouteThreads), lds, stream, a); \
  else                                                                                                \
    hipLaunchKernelGGL((k_route_grad<false, EPL, L>), grid_of(grid), dim3(kRouteThreads), lds, stream, a)
  FP4_ROUTE_SIZES(FP4_CALL)
#undef FP4_CALL
  return hipGetLastError();
}

// Workspace: kAmaxPartials partial maxima of x | histograms [chunks][E].
size_t dispatch_workspace_bytes(int64_t n, int64_t E) {
  const int64_t chunk = sort_chunk(n), chunks = (n + chunk - 1) / chunk;
  return (size_t)kAmaxPartials * 4 + (chunks > 1 ? (size_t)chunks * E * 4 : 0);
}

hipError_t launch_dispatch(const DispatchProblem& p, hipStream_t stream) {
  const int64_t n = p.T * p.top_k;
  if (n == 0) {
    hipLaunchKernelGGL(k_empty_dispatch, dim3(1), dim3(256), 0, stream, p.offsets, (int)p.E,
                       p.mx || p.amax_in != nullptr ? nullptr : p.amax_out, p.mx ? nullptr : p.scale_out);
    return hipGetLastError();
  }
  const int64_t chunk = sort_chunk(n), chunks = (n + chunk - 1) / chunk;
  uint32_t* partials = static_cast<uint32_t*>(p.workspace);
  int* counts = reinterpret_cast<int*>(partials + kAmaxPartials);
  const bool need_amax = !p.mx && p.amax_in == nullptr;
  const int64_t nx = p.T * p.H;
  const bool vec = ok16(p.x);
  const PlaceArgs a{p.ids, n, (int)p.E, (int)chunk, (int)chunks, counts, p.offsets, p.slot_rows, p.row_slots};
  GatherArgs ga{p.x, p.T, (int)p.H, p.top_k, (int)p.E, p.slot_rows, p.offsets, p.q, p.scales,
                p.amax_in, partials, 0, need_amax ? p.amax_out : nullptr, p.scale_out, vec};
  const int64_t blocks = p.T * (p.H / (p.mx ? 32 : 16));
  // (blocks < 2^30: 32-bit indexes there)
  if (n <= kSortThreads && p.H > 0 && blocks < (1 << 30) && (!need_amax || nx <= kSmallX)) {
    const int64_t wgs = (blocks + kSortThreads - 1) / kSortThreads;
    const dim3 gs((unsigned)(wgs < num_cus() ? wgs : num_cus()));
#define FP4_SMALL(MXV, BFV) \
  hipLaunchKernelGGL((k_dispatch_small<MXV, BFV>), gs, dim3(kSortThreads), 0, stream, a, ga)
    if (p.mx) {
      if (p.bf16) FP4_SMALL(true, true); else FP4_SMALL(true, false);
    } else {
      if (p.bf16) FP4_SMALL(false, true); else FP4_SMALL(false, false);
    }
#undef FP4_SMALL
    return hipGetLastError();
  }
  // one partial per 32 KB of x, at most two workgroups per CU
  int npart = 0;
  if (need_amax) {
    const int64_t want = (nx * (p.bf16 ? 2 : 4) + (1 << 15) - 1) >> 15;
    const int64_t most = min((int64_t)kAmaxPartials, (int64_t)2 * num_cus());
    npart = (int)(want < most ? want : most);
  }
  ga.npart = npart;
  const dim3 grid((unsigned)(chunks + npart));
  if (p.bf16)
    hipLaunchKernelGGL((k_count<true>), grid, dim3(kSortThreads), 0, stream, a, counts, (int)chunks, p.x,
                       nx, vec, partials, npart);
  else
    hipLaunchKernelGGL((k_count<false>), grid, dim3(kSortThreads), 0, stream, a, counts, (int)chunks, p.x,
                       nx, vec, partials, npart);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (chunks > 1) {
    hipLaunchKernelGGL(k_place, dim3((unsigned)chunks), dim3(kSortThreads), 0, stream, a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (p.H == 0) {
    if (!p.mx) return launch_empty_scales(p.amax_in != nullptr ? nullptr : p.amax_out, p.scale_out, stream);
    return hipSuccess;
  }
  const int64_t want = (blocks + kGatherThreads - 1) / kGatherThreads, most = (int64_t)16 * num_cus();
  const dim3 gg((unsigned)(want < most ? want : most));
#define FP4_GATHER(MXV, BFV) \
  hipLaunchKernelGGL((k_gather_quant<MXV, BFV>), gg, dim3(kGatherThreads), 0, stream, ga)
  if (p.mx) {
    if (p.bf16) FP4_GATHER(true, true); else FP4_GATHER(true, false);
  } else {
    if (p.bf16) FP4_GATHER(false, true); else FP4_GATHER(false, false);
  }
#undef FP4_GATHER
  return hipGetLastError();
}

hipError_t launch_combine(const void* rows, bool rows_bf16, int64_t M, int64_t H, const float* weights,
                          const int32_t* slot_rows, int64_t T, int top_k, const void* residual,
                          bool res_bf16, void* y, bool y_bf16, hipStream_t stream) {
  const CombineArgs a{rows, M, weights, slot_rows, T, (int)H, top_k, rows_bf16, res_bf16, y_bf16,
                      residual, y};
  const bool vec = H % 8 == 0 && ok16(rows) && ok16(residual) && ok16(y);
  const int64_t per = (int64_t)kCombineThreads * (vec ? 8 : 1);
  const int64_t pieces = (H + per - 1) / per;
  if (T * pieces >= (int64_t)1 << 31) return hipErrorInvalidValue;
#define FP4_COMBINE(VV, BF) \
  hipLaunchKernelGGL((k_combine<VV, BF>), grid_of(T * pieces), dim3(kCombineThreads), 0, stream, a, (int)pieces)
  if (vec) {
    if (rows_bf16) FP4_COMBINE(8, true); else FP4_COMBINE(8, false);
  } else {
    if (rows_bf16) FP4_COMBINE(1, true); else FP4_COMBINE(1, false);
  }
#undef FP4_COMBINE
  return hipGetLastError();
}

hipError_t launch_combine_grad(const void* dy, bool dy_bf16, const void* rows, bool rows_bf16, int64_t M,
                               int64_t H, const float* weights, const int32_t* slot_rows,
                               const int32_t* row_slots, int64_t T, int top_k, void* d_rows, bool dr_bf16,
                               float* d_weights, hipStream_t stream) {
  const CombineGradArgs a{dy, rows, weights, slot_rows, row_slots, T, M, (int)H, top_k, dy_bf16,
                          rows_bf16, dr_bf16, d_rows, d_weights};
  const bool vec = H % 8 == 0 && ok16(dy) && ok16(rows) && ok16(d_rows);
#define FP4_COMBINE(VV, BF) hipLaunchKernelGGL((k_combine_grad<VV, BF>), grid_of(T), dim3(kCombineThreads), 0, stream, a)
  if (vec) {
    if (rows_bf16) FP4_COMBINE(8, true); else FP4_COMBINE(8, false);
  } else {
    if (rows_bf16) FP4_COMBINE(1, true); else FP4_COMBINE(1, false);
  }
#undef FP4_COMBINE
  return hipGetLastError();
}

}  // namespace fp4impl
