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

// The last i < n with at(i) <= x for ascending at(i), or -1; the same in all 64 lanes, which all
// call.  64 probes a round, so one round up to 64.
template <typename At>
__device__ __forceinline__ int last_at_most(int n, int x, At at) {
  const int lane = threadIdx.x & 63;
  int lo = 0;
  while (true) {
    const int step = (n + 63) >> 6;
    const bool reached = lane * step < n && at(lo + lane * step) <= x;
    const int hits = __popcll(__ballot(reached));
    if (hits == 0) return -1;
    lo += (hits - 1) * step;
    n = min(step, n - (hits - 1) * step);
    if (step == 1) return lo;
  }
}

// The sequence of row r: the last b with offsets[b] <= r, or -1.
__device__ __forceinline__ int seq_of_row(const fp4impl::KvCache& c, int r) {
  return last_at_most(c.seqs, r, [&](int b) { return c.offsets[b]; });
}

}  // namespace fp4dev
