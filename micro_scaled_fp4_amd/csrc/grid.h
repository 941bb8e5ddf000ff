// Grids of up to 2^31 workgroups.  A dispatch counts work-items in 32 bits per
// dimension, so a one-dimensional grid of 256 threads ends below 2^24 workgroups (past
// them the count wraps, without an error): more go in rows of kGridRow, the last of
// which may run past the count.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp4impl {

constexpr int64_t kGridRow = 1 << 20;           // a multiple of the XCD count

inline dim3 grid_of(int64_t workgroups) {
  if (workgroups <= kGridRow) return dim3((unsigned)workgroups);
  return dim3((unsigned)kGridRow, (unsigned)((workgroups + kGridRow - 1) / kGridRow));
}

}  // namespace fp4impl

namespace fp4dev {

// This workgroup's number in a grid_of launch, and their count.
__device__ __forceinline__ uint32_t workgroup() { return blockIdx.y * gridDim.x + blockIdx.x; }
__device__ __forceinline__ uint32_t workgroups() { return gridDim.y * gridDim.x; }

}  // namespace fp4dev
