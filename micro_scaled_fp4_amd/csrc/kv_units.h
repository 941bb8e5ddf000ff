// Units of work of the attention over a paged cache: row tiles x parts of their
// positions, laid out from the sequences' sizes on the device.
//
// The query rows of a sequence and key/value head are packed as rho = row * group + (query
// head within the group), so that all heads of a group share what is read; kRows of them make a
// row tile.  A tile's positions are cut into parts of `per` steps (of 64 positions), `per`
// being the same for all sequences: the length that makes whole rounds of resident workgroups
// fastest (unit_of).  So long sequences are cut into many parts and short ones into one, whatever
// the batch holds, and the host needs to know no length.  A tile of one part writes its output;
// the parts of a cut one leave theirs in the workspace, and k_join_parts joins them.
//
// Up to 64 sequences every wave lays them out by itself, a lane for each (part of the 2.6 us until a
// unit is known, and no launch); more are laid out once, by k_lay_out, and a wave searches that.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kv_cache.h"

namespace fp4impl {

// What the unit layout depends on besides the sequences.
struct UnitPlan {
  int rows;                      // query rows of a tile (packed)
  int group;
  int min_per;                   // least steps of a part
  int whole;                     // tiles of up to so many steps are never cut, if no tile has more
  int turn;                      // steps that a workgroup takes at a time
  int join;                      // what joining parts costs, in steps (tiles of 128 rows: for each round)
  int target;                    // parts per key/value head that fill the card
  int rounds;                    // at most that many rounds of such parts are looked at
  int max_slots, max_parts;      // most tiles, and most parts of cut tiles (per head)
  bool causal;
  int window;
  // workspace: per tile (slot) a TileParts, then the layout of more than kLaneSeqs sequences, then
  // the parts' results
  void* tiles;
  int4* layout;                  // [seqs + 1]: units, parts of cut tiles and tiles before each; the last: of all, and `per`
  float* parts;
};

// A tile as k_join_parts needs it.
struct TileParts {
  int begin, first_row, rows, part0, count, pad[3];
};

// Units past the tiles and parts that the layout can give (the total of the steps is a sum of
// float32 values).
constexpr int kSpareUnits = 8;
// Sequences that a wave lays out by itself.
constexpr int kLaneSeqs = 64;
// `slots` where offsets decrease and give more tiles than there are rows: nothing is done then.
constexpr int kNoLayout = 0x7fffffff;

}  // namespace fp4impl

namespace fp4dev {

using fp4impl::KvCache;
using fp4impl::TileParts;
using fp4impl::UnitPlan;

// Sums over lanes 0 .. lane.
__device__ __forceinline__ int scan_lanes(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);   // row_shr:1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);   // row_bcast:15 into rows 1 and 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);   // row_bcast:31 into rows 2 and 3
  return v;
}

// The sum over all lanes, the same in all.
__device__ __forceinline__ float sum_lanes(float v) {
  auto moved = [&](int x) { return __uint_as_float((uint32_t)x); };
  auto bits = [&]() { return (int)__float_as_uint(v); };
  v += moved(__builtin_amdgcn_update_dpp(0, bits(), 0x111, 0xf, 0xf, false));
  v += moved(__builtin_amdgcn_update_dpp(0, bits(), 0x112, 0xf, 0xf, false));
  v += moved(__builtin_amdgcn_update_dpp(0, bits(), 0x114, 0xf, 0xf, false));
  v += moved(__builtin_amdgcn_update_dpp(0, bits(), 0x118, 0xf, 0xf, false));
  v += moved(__builtin_amdgcn_update_dpp(0, bits(), 0x142, 0xa, 0xf, false));
  v += moved(__builtin_amdgcn_update_dpp(0, bits(), 0x143, 0xc, 0xf, false));
  return moved(__builtin_amdgcn_readlane(bits(), 63));
}

__device__ __forceinline__ float max_lanes(float v) {   // v >= 0
  auto at = [&](int x) { return __uint_as_float((uint32_t)x); };
  auto bits = [&]() { return (int)__float_as_uint(v); };
  v = fmaxf(v, at(__builtin_amdgcn_update_dpp(0, bits(), 0x111, 0xf, 0xf, false)));
  v = fmaxf(v, at(__builtin_amdgcn_update_dpp(0, bits(), 0x112, 0xf, 0xf, false)));
  v = fmaxf(v, at(__builtin_amdgcn_update_dpp(0, bits(), 0x114, 0xf, 0xf, false)));
  v = fmaxf(v, at(__builtin_amdgcn_update_dpp(0, bits(), 0x118, 0xf, 0xf, false)));
  v = fmaxf(v, at(__builtin_amdgcn_update_dpp(0, bits(), 0x142, 0xa, 0xf, false)));
  v = fmaxf(v, at(__builtin_amdgcn_update_dpp(0, bits(), 0x143, 0xc, 0xf, false)));
  return at(__builtin_amdgcn_readlane(bits(), 63));
}

struct Unit {
  int b, begin, n, length;       // the sequence: its first row, rows, positions
  int tile, slot;                // its row tile, and that among all sequences' tiles
  int part, count, per;          // this part of count, per steps each
  int part0;                     // the tile's first among all cut tiles' parts
  int slots;                     // all tiles
  bool any;                      // there is such a unit
};

struct SeqSize {
  int begin, n, length, tiles, steps;
};

// Tiles of sequence b and the steps of each, at most (a window bounds what a tile sees).
__device__ __forceinline__ SeqSize seq_size(const KvCache& c, const UnitPlan& p, int b) {
  SeqSize s;
  s.begin = seq_begin(c, b);
  s.n = seq_end(c, b, s.begin) - s.begin;
  s.length = seq_length(c, b);
  s.tiles = (int)(((int64_t)s.n * p.group + p.rows - 1) / p.rows);
  s.steps = (s.length + 63) >> 6;
  if (p.window > 0) s.steps = (int)min((int64_t)s.steps, ((int64_t)p.window + (p.rows - 1) / p.group + 127) >> 6);
  s.steps = max(s.steps, 1);
  return s;
}

// The sequences' totals: steps of all tiles, tiles, and the most steps of a tile.
struct Totals {
  float work, tiles, longest;
};

// Whether the layout of so many tiles holds (false: offsets decrease).
__device__ __forceinline__ bool fits(const UnitPlan& p, const Totals& all) { return all.tiles <= 1.01f * (float)p.max_slots; }

// Parts of 1 / inverse steps each that `steps` steps make, inverse being 2^-21 too large: as many up to
// 2^20 steps, never too few beyond.
__device__ __forceinline__ float parts_at(float steps, float inverse) { return ceilf((steps - 0.5f) * inverse); }

constexpr float kStart = 4;      // a part's beginning and end, in steps

// Steps of all tiles of a sequence, about, as far as causal rows see: the first tile sees `least`, each
// further one as many positions more as it has rows, up to s.steps.
__device__ __forceinline__ float seen_steps(const UnitPlan& p, const SeqSize& s) {
  const float tiles = (float)s.tiles, steps = (float)s.steps;
  if (!p.causal) return tiles * steps;
  const float rows = fmaxf((float)(p.rows / p.group), 1.0f);
  const float least = fminf(fmaxf(((float)(s.length - s.n) + rows) * (1.0f / 64), 1.0f), steps);
  return tiles * steps - 0.5f * (steps - least) * fminf(tiles, (steps - least) * 64 / rows);
}

// Time of all tiles without parts, in steps: whole rounds of the longest where tiles are alike.  Causal
// tiles of a prompt are not: longest first, they fill each other's gaps, and the mean load of a workgroup
// counts.  `seen` steps (the sum of seen_steps) say how far they differ.
__device__ __forceinline__ float whole_time(const UnitPlan& p, const Totals& all) {
  return ceilf(all.tiles / (float)p.target) * (all.longest + kStart);
}
__device__ __forceinline__ float whole_time(const UnitPlan& p, const Totals& all, float seen) {
  const float alike = fmaxf(2 * seen / all.work - 1, 0.0f);
  return alike * whole_time(p, all) +
         (1 - alike) * fmaxf(all.longest + kStart, (seen + all.tiles * kStart) / (float)p.target);
}

// Steps of a part: a multiple of p.turn.  Parts of the same length run in rounds of `target`: the
// shortest length that needs no more than k rounds, for the k with the least time, or no parts at all
// (`whole`, whole_time).  Time in steps: kStart for a part, p.join for joining.  units_at(inverse): all
// units of parts of 1 / inverse steps.
template <typename UnitsAt>
__device__ __forceinline__ int part_steps(const UnitPlan& p, const Totals& all, float whole, UnitsAt units_at) {
  const float target = (float)p.target, turn = (float)p.turn;
  if (!(all.tiles < p.rounds * target && all.longest > (float)p.whole)) return max(p.whole, (int)fminf(ceilf(all.work / target), 1.0e9f));
  // (more than 32 parts of a tile: twice as long ones, since each is a step of the join's)
  const float shortest = (float)(all.longest > 32.0f * (float)p.min_per ? p.whole : p.min_per);
  float best = whole;
  float per = all.longest;
  for (int k = 1; k <= p.rounds; ++k) {
    const float room = k * target;
    if (all.tiles > room) continue;
    const float least = fmaxf(ceilf(all.work / room), shortest);
    // in turns
    float lo = ceilf(least / turn);
    float hi = fmaxf(lo, ceilf((all.tiles < room ? fminf(all.longest, ceilf(all.work / (room - all.tiles))) : all.longest) / turn));
    for (int i = 0; i < 6 && lo < hi; ++i) {
      const float mid = floorf(0.5f * (lo + hi));
      if (units_at((1.0f + 0x1p-21f) / (mid * turn)) <= room) hi = mid;
      else lo = mid + 1;
    }
    const float time = k * (hi * turn + kStart) + (p.turn > 1 ? p.join : k * p.join);
    if (time < best) {
      best = time;
      per = hi * turn;
    }
    if (hi * turn <= 1.125f * least + 1) break;   // a round more has nothing left to fill
  }
  return max((int)per, p.min_per);
}

__device__ __forceinline__ int parts_of(int steps, int per) { return (steps + per - 1) / per; }

// Unit u of this head, for one wave (all 64 lanes call; the result is the same in all).  ALIKE: a
// sequence's tiles see the same steps, but for one or two (few rows).
template <bool ALIKE>
__device__ __forceinline__ Unit unit_of(const KvCache& c, const UnitPlan& p, int u) {
  const int lane = threadIdx.x & 63;
  Unit r{};
  r.slots = fp4impl::kNoLayout;
  SeqSize s;
  int left, part0, slot;         // u among the sequence's units; parts and tiles before the sequence
  if (c.seqs <= fp4impl::kLaneSeqs) {
    const SeqSize mine = lane < c.seqs ? seq_size(c, p, lane) : SeqSize{0, 0, 0, 0, 1};
    const float tiles = (float)mine.tiles, steps = (float)mine.steps;
    const Totals all{sum_lanes(tiles * steps), sum_lanes(tiles), max_lanes(mine.tiles > 0 ? steps : 0.0f)};
    if (!fits(p, all)) return r;
    float whole;
    if constexpr (ALIKE) whole = whole_time(p, all);
    else whole = whole_time(p, all, sum_lanes(seen_steps(p, mine)));
    r.per = __builtin_amdgcn_readfirstlane(
        part_steps(p, all, whole, [&](float inverse) { return sum_lanes(tiles * parts_at(steps, inverse)); }));
    const int count = parts_of(mine.steps, r.per), units = mine.tiles * count, parts = count > 1 ? units : 0;
    const int units_to = scan_lanes(units), parts_to = scan_lanes(parts), tiles_to = scan_lanes(mine.tiles);
    r.slots = __builtin_amdgcn_readlane(tiles_to, 63);
    r.any = u < __builtin_amdgcn_readlane(units_to, 63);
    if (!r.any) return r;
    r.b = __builtin_amdgcn_readfirstlane((int)__ffsll((unsigned long long)__ballot(units_to > u)) - 1);
    s = {__builtin_amdgcn_readlane(mine.begin, r.b), __builtin_amdgcn_readlane(mine.n, r.b),
         __builtin_amdgcn_readlane(mine.length, r.b), __builtin_amdgcn_readlane(mine.tiles, r.b),
         __builtin_amdgcn_readlane(mine.steps, r.b)};
    left = u - __builtin_amdgcn_readlane(units_to - units, r.b);
    part0 = __builtin_amdgcn_readlane(parts_to - parts, r.b);
    slot = __builtin_amdgcn_readlane(tiles_to - mine.tiles, r.b);
  } else {
    const int4 all = p.layout[c.seqs];
    r.per = __builtin_amdgcn_readfirstlane(all.w);
    r.slots = __builtin_amdgcn_readfirstlane(all.z);
    r.any = u < __builtin_amdgcn_readfirstlane(all.x);
    if (!r.any) return r;
    r.b = __builtin_amdgcn_readfirstlane(last_at_most(c.seqs, u, [&](int b) { return p.layout[b].x; }));
    const int4 before = p.layout[r.b];
    left = u - __builtin_amdgcn_readfirstlane(before.x);
    part0 = __builtin_amdgcn_readfirstlane(before.y);
    slot = __builtin_amdgcn_readfirstlane(before.z);
    const SeqSize mine = seq_size(c, p, r.b);
    s = {__builtin_amdgcn_readfirstlane(mine.begin), __builtin_amdgcn_readfirstlane(mine.n),
         __builtin_amdgcn_readfirstlane(mine.length), __builtin_amdgcn_readfirstlane(mine.tiles),
         __builtin_amdgcn_readfirstlane(mine.steps)};
  }
  const int count = __builtin_amdgcn_readfirstlane(parts_of(s.steps, r.per)), k = left / count;
  r.begin = s.begin;
  r.n = s.n;
  r.length = s.length;
  r.tile = s.tiles - 1 - k;                     // later rows see more positions and start first
  r.slot = slot + r.tile;
  r.part = left - k * count;
  r.count = count;
  r.per = __builtin_amdgcn_readfirstlane(parts_of(s.steps, count));   // parts of equal length
  r.part0 = part0 + r.tile * count;
  return r;
}

// The page table of a sequence as a wave walks along it in steps of 64 positions: lane i holds
// entry base + i (-1: a hole or past the table), and the next 64 entries are on their way, so that
// no page number is waited for.  A step's entries (1, 2 or 4, and 64 is a multiple of them) are
// among the 64.
struct PageWalk {
  const int32_t* table;
  int max_pages, num_pages, shift, base, now, next;
  uint64_t holes;                // of `now`

  __device__ __forceinline__ int entries(int from) const {
    const int i = from + (int)(threadIdx.x & 63);
    const int p = i < max_pages ? table[i] : -1;
    return p >= 0 && p < num_pages ? p : -1;
  }
  // from step t on (a multiple of 64)
  __device__ __forceinline__ PageWalk(const KvCache& c, int b, int t)
      : table(c.pages + b * c.max_pages), max_pages((int)c.max_pages), num_pages((int)c.num_pages),
        shift(c.page_shift), base(t >> c.page_shift) {
    now = entries(base);
    next = entries(base + 64);
    holes = __ballot(now < 0);
  }
  // To step t, the same in all lanes, not before the last one.
  __device__ __forceinline__ void reach(int t) {
    while ((t >> shift) - base >= 64) {
      base += 64;
      now = next;
      next = entries(base + 64);
      holes = __ballot(now < 0);
    }
  }
  // The page of a position of the step reached.
  __device__ __forceinline__ int at(int t) const { return __builtin_amdgcn_readlane(now, (t >> shift) - base); }
  // Bit i: positions t + 16 i .. of the step t reached are in a hole.
  __device__ __forceinline__ uint32_t holes_at(int t) const {
    if (holes == 0) return 0;
    uint32_t h = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) h |= (uint32_t)(holes >> (((t + 16 * i) >> shift) - base) & 1) << i;
    return h;
  }
};

// Positions of a unit: [t0, t1), t0 a multiple of 64 unless the unit is empty.  Positions before lo
// are seen by no row of the tile.
struct Span {
  int t0, t1, lo;
};

__device__ __forceinline__ Span span_of(const UnitPlan& p, const Unit& u, int rows) {
  const int first = u.length - u.n + u.tile * p.rows / p.group;
  const int last = u.length - u.n + (u.tile * p.rows + rows - 1) / p.group;
  const int hi = p.causal ? max(0, min(u.length, last + 1)) : u.length;   // (rows may sit before position 0)
  const int lo = p.window > 0 ? max(0, first - p.window + 1) : 0;
  const int64_t t0 = (lo & ~63) + (int64_t)u.part * u.per * 64;
  const int64_t t1 = u.part == u.count - 1 ? hi : min((int64_t)hi, t0 + (int64_t)u.per * 64);
  return {(int)min(t0, (int64_t)hi), (int)t1, lo};
}

}  // namespace fp4dev
