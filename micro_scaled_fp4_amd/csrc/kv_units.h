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
  int target;                    // parts per key/value head that fill the card
  int rounds;                    // at most that many rounds of such parts are looked at
  int max_slots, max_parts;      // most tiles, and most parts of cut tiles (per head)
  bool causal;
  int window;
  // workspace: per tile (slot) a TileParts, then the parts' results
  void* tiles;
  float* parts;
};

// A tile as k_join_parts needs it.
struct TileParts {
  int begin, first_row, rows, part0, count, pad[3];
};

// Units past the tiles and parts that the layout can give (the total of the steps is a sum of
// float32 values).
constexpr int kSpareUnits = 8;

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

// Unit u of this head, for one wave (all 64 lanes call; the result is the same in all).  Each
// lane takes a run of sequences; sums and scans over the lanes give the totals and u's lane.
__device__ __forceinline__ Unit unit_of(const KvCache& c, const UnitPlan& p, int u) {
  const int lane = threadIdx.x & 63, run = (c.seqs + 63) >> 6;
  const int b0 = min(lane * run, c.seqs), b1 = min(b0 + run, c.seqs);
  // (up to 64 sequences: one a lane, read once)
  const SeqSize mine = b0 < b1 ? seq_size(c, p, b0) : SeqSize{0, 0, 0, 0, 1};
  auto each = [&](auto f) {
    f(mine);
    for (int b = b0 + 1; b < b1; ++b) f(seq_size(c, p, b));
  };
  float work = 0, all = 0, longest = 0;         // steps of all tiles, tiles, the most steps of one
  each([&](const SeqSize& s) {
    work += (float)s.tiles * (float)s.steps;
    all += (float)s.tiles;
    longest = fmaxf(longest, s.tiles > 0 ? (float)s.steps : 0.0f);
  });
  work = sum_lanes(work);
  all = sum_lanes(all);
  Unit r{};
  // offsets that decrease can give more tiles than there are rows: nothing is done then
  r.slots = 0x7fffffff;
  if (!(all <= 1.01f * (float)p.max_slots)) return r;
  const float target = (float)p.target;
  r.per = max(p.min_per, (int)fminf(ceilf(work / target), 1.0e9f));
  if (all < p.rounds * target && work > 0) {
    // Parts of the same length run in rounds of `target`: the shortest length that needs no more
    // than k rounds, for the k with the least time (kStart steps for a part's beginning and end).
    constexpr float kStart = 4;
    longest = max_lanes(longest);
    float best = INFINITY;
    for (int k = 1; k <= p.rounds; ++k) {
      const float room = k * target;
      if (all > room) continue;
      const float least = fmaxf(ceilf(work / room), (float)p.min_per);
      float lo = least, hi = fmaxf(lo, all < room ? fminf(longest, ceilf(work / (room - all))) : longest);
      for (int i = 0; i < 6 && lo < hi; ++i) {
        const float mid = floorf(0.5f * (lo + hi)), inverse = (1.0f + 0x1p-21f) / mid;   // never too few
        float units = 0;
        each([&](const SeqSize& s) { units += (float)s.tiles * ceilf((float)s.steps * inverse); });
        if (sum_lanes(units) <= room) hi = mid;
        else lo = mid + 1;
      }
      const float time = k * (hi + kStart);
      if (time < best) {
        best = time;
        r.per = (int)hi;
      }
      if (hi <= 1.125f * least + 1) break;      // a round more has nothing left to fill
    }
  }
  r.per = __builtin_amdgcn_readfirstlane(r.per);
  int units = 0, parts = 0, tiles = 0;
  each([&](const SeqSize& s) {
    const int count = (s.steps + r.per - 1) / r.per;
    units += s.tiles * count;
    parts += count > 1 ? s.tiles * count : 0;
    tiles += s.tiles;
  });
  const int units_to = scan_lanes(units), parts_to = scan_lanes(parts), tiles_to = scan_lanes(tiles);
  r.slots = __builtin_amdgcn_readlane(tiles_to, 63);
  r.any = u < __builtin_amdgcn_readlane(units_to, 63);
  if (!r.any) return r;
  const int at = __builtin_amdgcn_readfirstlane((int)__ffsll((unsigned long long)__ballot(units_to > u)) - 1);
  int left = u - __builtin_amdgcn_readlane(units_to - units, at);
  int part0 = __builtin_amdgcn_readlane(parts_to - parts, at), slot = __builtin_amdgcn_readlane(tiles_to - tiles, at);
  for (int b = at * run; b < c.seqs; ++b) {
    SeqSize s;
    if (b == at * run) {
      s = {__builtin_amdgcn_readlane(mine.begin, at), __builtin_amdgcn_readlane(mine.n, at),
           __builtin_amdgcn_readlane(mine.length, at), __builtin_amdgcn_readlane(mine.tiles, at),
           __builtin_amdgcn_readlane(mine.steps, at)};
    } else {
      s = seq_size(c, p, b);
    }
    const int tiles_b = __builtin_amdgcn_readfirstlane(s.tiles);
    const int count = __builtin_amdgcn_readfirstlane((s.steps + r.per - 1) / r.per);
    if (left < tiles_b * count) {
      // later rows see more positions and start first
      const int k = left / count;
      r.b = b;
      r.begin = __builtin_amdgcn_readfirstlane(s.begin);
      r.n = __builtin_amdgcn_readfirstlane(s.n);
      r.length = __builtin_amdgcn_readfirstlane(s.length);
      r.tile = tiles_b - 1 - k;
      r.slot = slot + r.tile;
      r.part = left - k * count;
      r.count = count;
      r.per = __builtin_amdgcn_readfirstlane((s.steps + count - 1) / count);   // parts of equal length
      r.part0 = part0 + r.tile * count;
      return r;
    }
    left -= tiles_b * count;
    part0 += count > 1 ? tiles_b * count : 0;
    slot += tiles_b;
  }
  r.any = false;
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
