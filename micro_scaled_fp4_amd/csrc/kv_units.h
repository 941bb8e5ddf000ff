// Units of work of the attention over a paged cache: row tiles x parts of their
// positions, laid out from the sequences' sizes on the device.
//
// The query rows of a sequence and key/value head are packed as rho = row * group + (query
// head within the group), so that all heads of a group share what is read; kRows of them make a
// row tile.  A tile's positions are cut into parts of `per` steps (of 64 positions), `per`
// being the same for all sequences: the total of all tiles' steps over the number of parts that
// fill the card.  So long sequences are cut into many parts and short ones into one, whatever
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
  bool fit;                      // no more than those, for kernels whose workgroups are all resident
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
// The most workgroups on a compute unit that any of the kernels reaches.
constexpr int kMostResident = 4;

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
  float work = 0, all = 0;       // steps of all tiles, and tiles
  for (int b = b0; b < b1; ++b) {
    const SeqSize s = seq_size(c, p, b);
    work += (float)s.tiles * (float)s.steps;
    all += (float)s.tiles;
  }
  work = sum_lanes(work);
  all = sum_lanes(all);
  Unit r{};
  // offsets that decrease can give more tiles than there are rows: nothing is done then
  r.slots = 0x7fffffff;
  if (!(all <= 1.01f * (float)p.max_slots)) return r;
  const float share = ceilf(work / (float)p.target);
  r.per = max(p.min_per, (int)fminf(share, 1.0e9f));
  if (p.fit && 2.0f * all < (float)p.target) {
    // the shortest parts that are no more than `target`: each tile's last part is shorter than the
    // others, so share gives up to a part more for each tile, and work / (target - all) never does
    int lo = r.per, hi = max(p.min_per, (int)ceilf(work / ((float)p.target - all)));
    for (int i = 0; i < 4 && lo < hi; ++i) {
      const int mid = (lo + hi) >> 1;
      float units = 0;
      for (int b = b0; b < b1; ++b) {
        const SeqSize s = seq_size(c, p, b);
        units += (float)(s.tiles * ((s.steps + mid - 1) / mid));
      }
      if (sum_lanes(units) <= (float)p.target) hi = mid;
      else lo = mid + 1;
    }
    r.per = hi;
  }
  int units = 0, parts = 0, tiles = 0;
  for (int b = b0; b < b1; ++b) {
    const SeqSize s = seq_size(c, p, b);
    const int count = (s.steps + r.per - 1) / r.per;
    units += s.tiles * count;
    parts += count > 1 ? s.tiles * count : 0;
    tiles += s.tiles;
  }
  const int units_to = scan_lanes(units), parts_to = scan_lanes(parts), tiles_to = scan_lanes(tiles);
  r.slots = __builtin_amdgcn_readlane(tiles_to, 63);
  r.any = u < __builtin_amdgcn_readlane(units_to, 63);
  if (!r.any) return r;
  const int at = __builtin_amdgcn_readfirstlane((int)__ffsll((unsigned long long)__ballot(units_to > u)) - 1);
  int left = u - __builtin_amdgcn_readlane(units_to - units, at);
  int part0 = __builtin_amdgcn_readlane(parts_to - parts, at), slot = __builtin_amdgcn_readlane(tiles_to - tiles, at);
  for (int b = at * run; b < c.seqs; ++b) {
    const SeqSize s = seq_size(c, p, b);
    const int count = __builtin_amdgcn_readfirstlane((s.steps + r.per - 1) / r.per);
    const int tiles_b = __builtin_amdgcn_readfirstlane(s.tiles);
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

// The page table of a sequence as a wave walks along it: lane i holds entry base + i (-1: a hole
// or past the table), and the next 64 entries are on their way, so that no page number is waited
// for.
struct PageWalk {
  const int32_t* table;
  int max_pages, num_pages, shift, base, now, next;

  __device__ __forceinline__ int entries(int from) const {
    const int i = from + (int)(threadIdx.x & 63);
    const int p = i < max_pages ? table[i] : -1;
    return p >= 0 && p < num_pages ? p : -1;
  }
  // from position t on
  __device__ __forceinline__ PageWalk(const KvCache& c, int b, int t)
      : table(c.pages + b * c.max_pages), max_pages((int)c.max_pages), num_pages((int)c.num_pages),
        shift(c.page_shift), base(t >> c.page_shift) {
    now = entries(base);
    next = entries(base + 64);
  }
  // Makes at() valid for the 64 positions from t on (t is the same in all lanes and does not decrease).
  __device__ __forceinline__ void reach(int t) {
    while ((t >> shift) - base >= 64) {
      base += 64;
      now = next;
      next = entries(base + 64);
    }
  }
  __device__ __forceinline__ int at(int t) const {
    const int i = (t >> shift) - base;
    return i < 64 ? __builtin_amdgcn_readlane(now, i) : __builtin_amdgcn_readlane(next, i - 64);
  }
};

// Positions of a unit: [t0, t1), t0 a multiple of 64 (positions before `lo` are masked).
struct Span {
  int t0, t1;
};

__device__ __forceinline__ Span span_of(const UnitPlan& p, const Unit& u, int rows) {
  const int first = u.length - u.n + u.tile * p.rows / p.group;
  const int last = u.length - u.n + (u.tile * p.rows + rows - 1) / p.group;
  const int hi = p.causal ? min(u.length, last + 1) : u.length;
  const int lo = p.window > 0 ? max(0, first - p.window + 1) : 0;
  const int64_t t0 = (lo & ~63) + (int64_t)u.part * u.per * 64;
  const int64_t t1 = u.part == u.count - 1 ? hi : min((int64_t)hi, t0 + (int64_t)u.per * 64);
  return {(int)min(t0, (int64_t)hi), (int)t1};
}

}  // namespace fp4dev
