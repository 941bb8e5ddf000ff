// Rows, sequences and positions of a paged FP4 cache, for its kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp4_internal.h"

namespace fp4dev {

// Rows of sequence b, as far as the T rows go.
__device__ __forceinline__ int seq_begin(const fp4impl::KvCache& c, int b) { return min(max(c.offsets[b], 0), c.rows); }
__device__ __forceinline__ int seq_end(const fp4impl::KvCache& c, int b, int begin) {
  return min(max(c.offsets[b + 1], begin), c.rows);
}
__device__ __forceinline__ int seq_length(const fp4impl::KvCache& c, int b) {
  return min(max(c.lengths[b], 0), c.capacity);
}

// The page of position t of sequence b, or -1 in a hole (0 <= t < capacity).
__device__ __forceinline__ int page_of(const fp4impl::KvCache& c, int b, int t) {
  const int p = c.pages[b * c.max_pages + (t >> c.page_shift)];
  return p >= 0 && p < c.num_pages ? p : -1;
}

// The row (page, head, slot) of a position among all rows of the cache: its codes start
// at byte row * dim / 2, its scale bytes at row * dim / bs.
__device__ __forceinline__ int64_t cache_row(const fp4impl::KvCache& c, int page, int head, int t) {
  return (((int64_t)page * c.heads + head) << c.page_shift) + (t & ((1 << c.page_shift) - 1));
}

// The sequence of row r (the same in all 64 lanes, which all call): the last b with
// offsets[b] <= r, or -1.  64 probes a round, so one round up to 64 sequences.
__device__ __forceinline__ int seq_of_row(const fp4impl::KvCache& c, int r) {
  const int lane = threadIdx.x & 63;
  int lo = 0, n = c.seqs;
  while (true) {
    const int step = (n + 63) >> 6;
    const int i = lo + lane * step;
    const bool at = lane * step < n && c.offsets[i] <= r;
    const int hits = __popcll(__ballot(at));
    if (hits == 0) return -1;
    lo += (hits - 1) * step;
    n = min(step, n - (hits - 1) * step);
    if (step == 1) return lo;
  }
}

}  // namespace fp4dev
